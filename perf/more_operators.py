"""Operators of a decode step whose cache is held in 8 bits, as they are measured: norms and
rotation of queries and keys on their way into the cache, folding full blocks of a bf16 cache into
the 8-bit one, and attention over the 8-bit cache with the bf16 positions behind it.

``run`` computes a case in plain torch (``own`` false) or through the library (``own`` true);
``exact`` is the definition in 64 bits.  Lengths follow from the case alone, values from the
seed.
"""
import math
import random

import torch

own = False

D = 64                      # head dimension of the library's caches
SCALE = 1.0 / math.sqrt(D)
THETA = 150000.0
FACTOR, CONTEXT, TURNS_LOW, TURNS_HIGH = 32.0, 4096.0, 1.0, 32.0
EPS = 1e-5
SMALLEST = 2.0 ** -110      # a block's largest magnitude counts as at least this
TAIL = 37                   # room of a bf16 cache beside its blocks, positions


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # one request, one step: latency
        dict(name="rope_one", op="rope", tokens=1, seqs=1, q_heads=64, kv_heads=8, room=63, rot=64,
             layout="half", norm=False, scaling="index", append=True, far=9000),
        # a full batch of one token each, with head norms, into the caches
        dict(name="rope_batch", op="rope", tokens=512, seqs=512, q_heads=64, kv_heads=8, room=127,
             rot=64, layout="half", norm=True, scaling="index", append=True, far=30000),
        # four prompts behind the fused projection
        dict(name="rope_prompts", op="rope", tokens=16384, seqs=4, q_heads=64, kv_heads=8, room=4096,
             rot=64, layout="half", norm=False, scaling="turns", append=True, far=0),
        # half of the head rotated, neighbouring pairs, no cache
        dict(name="rope_partial", op="rope", tokens=3001, seqs=1, q_heads=32, kv_heads=4, room=0,
             rot=32, layout="interleaved", norm=True, scaling="none", append=False, far=100000),
        # a batch between two steps: the bf16 positions of 64 requests, some with a full block
        dict(name="fold_tails", op="fold", seqs=64, kv_heads=8, length=127, held=1024, block=64,
             format="e4m3"),
        # the prompts of a batch on their way into the 8-bit cache
        dict(name="fold_prompts", op="fold", seqs=64, kv_heads=8, length=8192, held=0, block=64,
             format="e4m3"),
        # three requests of odd lengths, short blocks, behind what the cache holds already
        dict(name="fold_odd", op="fold", seqs=3, kv_heads=3, length=5003, held=1000, block=16,
             format="int8"),
        # two requests on short caches: latency
        dict(name="kvq_pair", op="kvq", seqs=2, q_heads=64, kv_heads=8, length=512, tail=40,
             block=64, format="e4m3", window=0),
        # one request on a long document
        dict(name="kvq_document", op="kvq", seqs=1, q_heads=64, kv_heads=8, length=131072, tail=64,
             block=64, format="e4m3", window=0),
        # a batch of long caches
        dict(name="kvq_gptoss", op="kvq", seqs=64, q_heads=64, kv_heads=8, length=8192, tail=64,
             block=64, format="e4m3", window=0),
        # odd head groups, short blocks, 8-bit integers
        dict(name="kvq_odd", op="kvq", seqs=37, q_heads=20, kv_heads=4, length=3001, tail=33,
             block=16, format="int8", window=0),
        # a full batch of the longest caches, 8 query heads on one KV head
        dict(name="kvq_32k", op="kvq", seqs=512, q_heads=8, kv_heads=1, length=32768, tail=128,
             block=128, format="int8", window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _draw(rng)
    most = dict(rope=3.3e8, fold=7.5e8, kvq=1.2e9)[case["op"]]
    while work(case)["bytes"] > most or _scores(case) > 512 * 8 * 32768:
        for k in ("length", "tokens", "held", "seqs"):
            if case.get(k, 0) > 8:
                case[k] -= case[k] // 3
        if case["op"] == "rope":
            case["seqs"] = min(case["seqs"], case["tokens"])
    return case


def _scores(case):
    return case["seqs"] * case.get("q_heads", 0) * (case.get("length", 0) + case.get("tail", 0))


def _draw(rng):
    op = rng.choice(["rope", "fold", "kvq", "kvq"])
    seqs = _log(rng, 1, 512)
    kv_heads = rng.choice([1, 2, 3, 4, 8, 8])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 8, 12, 16])
    if op == "rope":
        tokens = rng.choice([seqs, max(seqs, _log(rng, 1, 16384))])
        return dict(op=op, tokens=tokens, seqs=seqs, q_heads=q_heads, kv_heads=kv_heads,
                    room=rng.randint(1, 100), rot=rng.choice([16, 32, 48, 64, 64, 64]),
                    layout=rng.choice(["half", "half", "interleaved"]), norm=rng.choice([False, True]),
                    scaling=rng.choice(["none", "linear", "turns", "index"]),
                    append=rng.choice([False, True, True]),
                    far=rng.choice([0, 1000, 30000, 1000000]))
    block = rng.choice([16, 32, 64, 64, 128])
    fmt = rng.choice(["e4m3", "int8"])
    if op == "fold":
        tails = rng.choice([False, True])
        return dict(op=op, seqs=seqs, kv_heads=kv_heads,
                    length=rng.randint(block, 3 * block) if tails else _log(rng, 1, 32768),
                    held=rng.choice([0, 100, 1000, 5000]), block=block, format=fmt)
    return dict(op=op, seqs=seqs, q_heads=q_heads, kv_heads=kv_heads, length=_log(rng, 1, 65536),
                tail=rng.randint(1, 2 * block), block=block, format=fmt,
                window=rng.choice([0, 0, 0, 0, 128, 1000]))


# ---------------------------------------------------------------------------------------
# lengths and indices: functions of the case, so that work() can count them
# ---------------------------------------------------------------------------------------
def _spread(case, what, n, lo, hi):
    rng = random.Random("%s %s" % (what, sorted((k, v) for k, v in case.items() if k != "name")))
    got = [rng.randint(lo, hi) for _ in range(n)]
    got[0] = hi
    return got


def _rope_places(case):
    """Sequence and slot of every token: the tokens in equal runs, each behind what the sequence
    holds already."""
    n, T = case["seqs"], case["tokens"]
    seq = [t * n // T for t in range(T)]
    first, slot = {}, []
    start = _spread(case, "start", n, 0, case["room"])
    for t, s in enumerate(seq):
        slot.append(start[s] + t - first.setdefault(s, t))
    return seq, slot


def _rope_cap(case):
    return case["room"] + -(-case["tokens"] // case["seqs"])


def _fold_lengths(case):
    """bf16 positions and 8-bit positions of every request."""
    n, B = case["seqs"], case["block"]
    kv = _spread(case, "length", n, 0 if n > 4 else (case["length"] + 1) // 2, case["length"])
    held = [B * b for b in _spread(case, "held", n, 0, case["held"] // B)]
    return kv, held


def _fold_cap(case):
    B = case["block"]
    return (case["held"] // B + case["length"] // B + 1) * B


def _kvq_lengths(case):
    """8-bit positions (whole blocks) and bf16 positions of every request."""
    n, B = case["seqs"], case["block"]
    most = case["length"] // B
    held = [B * b for b in _spread(case, "length", n, 0 if n > 4 else (most + 1) // 2, most)]
    return held, _spread(case, "tail", n, 1, case["tail"])


def _kvq_cap(case):
    return (case["length"] // case["block"] + 1) * case["block"]


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _quantise(x, block, fmt):
    """Codes and scales of bf16 values [..., positions, D], positions a multiple of block."""
    y = x.float().unflatten(-2, (-1, block))
    amax = y.abs().amax((-1, -2)).clamp(min=SMALLEST)
    if fmt == "int8":
        s = amax / torch.full_like(amax, 127.0)     # 32-bit quotients, here and below
    else:
        m, e = torch.frexp(amax)                    # amax <= 448 2^(e - 9) when m <= 0.875
        s = ((torch.where(m <= 0.875, e - 9, e - 8) + 127) << 23).view(torch.float32)
    z = y / s[..., None, None]
    code = z.round().to(torch.int8) if fmt == "int8" else z.to(torch.float8_e4m3fn)
    return code.flatten(-3, -2), s


def _values(code, scale, block):
    return (code.float().unflatten(-2, (-1, block)) * scale[..., None, None]).flatten(-3, -2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        return t.normal_(0.0, scale, generator=g)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def held(n, heads, cap, block, fmt):
        """An 8-bit cache: keys and values whose size changes from head to head and along it."""
        code = torch.empty(n, heads, cap, D, device="cuda",
                           dtype=torch.int8 if fmt == "int8" else torch.float8_e4m3fn)
        scale = torch.empty(n, heads, cap // block, device="cuda")
        step = max(1, (1 << 21) // (heads * cap))
        for i in range(0, n, step):
            x = normal(min(step, n - i), heads, cap, D)
            size = torch.empty(x.shape[0], heads, cap // block, 1, 1, device="cuda")
            size = size.uniform_(-1.0, 1.0, generator=g).exp2_()
            x = (x.unflatten(2, (-1, block)) * size).bfloat16().flatten(2, 3)
            c, s = _quantise(x, block, fmt)
            code.view(torch.uint8)[i:i + step] = c.view(torch.uint8)
            scale[i:i + step] = s
        return code, scale

    st = dict(case=case, n=case["seqs"])
    if own:
        from intra_spatial_pipelining_gb300 import sgp
        st["sgp"] = sgp
    nkv = case["kv_heads"]
    if case["op"] == "rope":
        T, nq = case["tokens"], case["q_heads"]
        seq, slot = _rope_places(case)
        qkv = normal(T, (nq + 2 * nkv) * D)         # a fused projection's rows
        st.update(q=qkv[:, :nq * D], k=qkv[:, nq * D:(nq + nkv) * D], v=qkv[:, (nq + nkv) * D:],
                  pos=ints([s + case["far"] for s in slot]), freq=_frequencies(case),
                  q_out=torch.zeros(T, nq * D, dtype=torch.bfloat16, device="cuda"))
        st["gq"] = (1 + normal(D, scale=0.2)).bfloat16() if case["norm"] else None
        st["gk"] = (1 + normal(D, scale=0.2)).bfloat16() if case["norm"] else None
        if case["append"]:
            st.update(seq=ints(seq), slot=ints(slot), kc=normal(case["seqs"], nkv, _rope_cap(case), D),
                      vc=normal(case["seqs"], nkv, _rope_cap(case), D))
        else:
            st["k_out"] = torch.zeros(T, nkv * D, dtype=torch.bfloat16, device="cuda")
        if own:
            st["dims"] = sgp.make_heads(nq, nkv, D)
            st["rope"] = sgp.make_rope(case["rot"], THETA, layout=case["layout"],
                                       scaling=case["scaling"], factor=FACTOR, context=CONTEXT,
                                       turns_low=TURNS_LOW, turns_high=TURNS_HIGH,
                                       amplitude=_amplitude(case))
            st["ws"] = torch.zeros(64, dtype=torch.uint8, device="cuda")
            if case["append"]:
                st["cache"] = sgp.make_cache(st["kc"], st["vc"])
    elif case["op"] == "fold":
        n, L, B, cap = case["seqs"], case["length"], case["block"], _fold_cap(case)
        kv, at = _fold_lengths(case)
        st.update(k=normal(n, nkv, L, D), v=normal(n, nkv, L, D, scale=0.5), len=ints(kv),
                  held=ints(at), len_out=ints(kv), held_out=ints(at),
                  rk=torch.zeros(n, nkv, B + TAIL, D, dtype=torch.bfloat16, device="cuda"))
        st["rv"] = torch.zeros_like(st["rk"])
        st["kq"], st["ks"] = held(n, nkv, cap, B, case["format"])
        st["vq"], st["vs"] = held(n, nkv, cap, B, case["format"])
        if own:
            st["dims"] = sgp.make_heads(nkv, nkv, D)
            st["from"] = sgp.make_cache(st["k"], st["v"])
            st["rest"] = sgp.make_cache(st["rk"], st["rv"])
            st["to"] = sgp.make_kvq(st["kq"], st["vq"], st["ks"], st["vs"])
            st["ws"] = torch.zeros(64, dtype=torch.uint8, device="cuda")
    else:
        n, nq, cap, B = case["seqs"], case["q_heads"], _kvq_cap(case), case["block"]
        at, tail = _kvq_lengths(case)
        st.update(held=ints(at), len=ints(tail), q=normal(n, nq, D, scale=2.0),
                  k=normal(n, nkv, case["tail"], D), v=normal(n, nkv, case["tail"], D))
        st["kq"], st["ks"] = held(n, nkv, cap, B, case["format"])
        st["vq"], st["vs"] = held(n, nkv, cap, B, case["format"])
        if own:
            st["dims"] = sgp.make_heads(nq, nkv, D)
            st["cache"] = sgp.make_cache(st["k"], st["v"], case["window"])
            st["kvq"] = sgp.make_kvq(st["kq"], st["vq"], st["ks"], st["vs"])
            nbytes = sgp.sgp_kvq_attention_workspace_bytes(st["dims"], n)
            st["ws"] = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
            st["o"] = torch.empty_like(st["q"])
            st["lse"] = torch.empty(n, nq, dtype=torch.float32, device="cuda")
    return st


def _amplitude(case):
    return 0.1 * math.log(FACTOR) + 1.0 if case["scaling"] in ("turns", "index") else 1.0


def _frequencies(case):
    """Radians per position of every pair, [rot / 2], 64 bits."""
    i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
    f = THETA ** (-2.0 * i / case["rot"])
    if case["scaling"] == "linear":
        return f / FACTOR
    if case["scaling"] == "turns":                  # turns within the context trained on
        keep = (CONTEXT * f / (2 * math.pi) - TURNS_LOW) / (TURNS_HIGH - TURNS_LOW)
    elif case["scaling"] == "index":                # the same bounds, linear in the pair's index
        lo, hi = (case["rot"] / 2 * math.log(CONTEXT / (2 * math.pi * t)) / math.log(THETA)
                  for t in (TURNS_HIGH, TURNS_LOW))
        keep = 1.0 - (i - lo) / (hi - lo)
    else:
        return f
    keep = keep.clamp(0.0, 1.0)
    return f * keep + f / FACTOR * (1.0 - keep)


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        sgp = st["sgp"]
        if op == "rope" and case["append"]:
            sgp.sgp_qk_rope_append(st["dims"], st["rope"], st["gq"], st["gk"], EPS, st["pos"],
                                   st["q"], st["q_out"], st["k"], st["v"], st["cache"], st["n"],
                                   st["seq"], st["slot"], case["tokens"], st["ws"])
            return st["q_out"], st["kc"], st["vc"]
        if op == "rope":
            sgp.sgp_qk_rope(st["dims"], st["rope"], st["gq"], st["gk"], EPS, st["pos"], st["q"],
                            st["q_out"], st["k"], st["k_out"], case["tokens"], st["ws"])
            return st["q_out"], st["k_out"]
        if op == "fold":
            sgp.sgp_kvq_fold(st["dims"], st["from"], st["to"], st["rest"], st["len"], st["held"],
                             st["len_out"], st["held_out"], st["n"], st["ws"])
            return (st["kq"], st["vq"], st["ks"], st["vs"], st["rk"], st["rv"], st["len_out"],
                    st["held_out"])
        sgp.sgp_kvq_attention(st["dims"], st["kvq"], st["held"], st["cache"], st["len"], st["q"],
                              st["o"], st["lse"], st["n"], st["ws"])
        return st["o"], st["lse"]
    if op == "rope":
        return _rope_plain(st)
    if op == "fold":
        return _fold_plain(st)
    return _kvq_plain(st)


def _rope_plain(st):
    case = st["case"]
    # far positions: the angle in 64 bits
    angle = st["pos"].double()[:, None] * st["freq"]
    cos, sin = ((f(angle) * _amplitude(case)).float()[:, None] for f in (torch.cos, torch.sin))

    def rotate(x, gain):
        x = x.float().unflatten(-1, (-1, D))
        if gain is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain.float()
        rot, rest = x[..., :case["rot"]], x[..., case["rot"]:]
        if case["layout"] == "half":
            a, b = rot.chunk(2, -1)
            rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = rot[..., 0::2], rot[..., 1::2]
            rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([rot, rest], -1).bfloat16()

    q, k = rotate(st["q"], st["gq"]), rotate(st["k"], st["gk"])
    if not case["append"]:
        return q.flatten(1), k.flatten(1)
    seq, slot = st["seq"].long(), st["slot"].long()
    st["kc"][seq, :, slot] = k
    st["vc"][seq, :, slot] = st["v"].unflatten(-1, (-1, D))
    return q.flatten(1), st["kc"], st["vc"]


def _fold_plain(st):
    case = st["case"]
    B, cap, L = case["block"], _fold_cap(case), case["length"]
    kv, held = st["len"].long(), st["held"].long()
    full = kv // B * B
    # where every position of the 8-bit cache comes from, and every position behind the blocks
    src = torch.arange(cap, device="cuda") - held[:, None]
    new = (src >= 0) & (src < full[:, None])
    behind = torch.arange(B + TAIL, device="cuda") + full[:, None]
    left = behind < kv[:, None]
    out = []
    for x, code, scale in ((st["k"], st["kq"], st["ks"]), (st["v"], st["vq"], st["vs"])):
        pad = torch.nn.functional.pad(x, (0, 0, 0, -L % B))
        c, s = _quantise(pad, B, case["format"])
        at = src.clamp(0, c.shape[2] - 1)[:, None].expand(-1, code.shape[1], -1)
        c = c.view(torch.uint8).gather(2, at[..., None].expand(-1, -1, -1, D))
        c = torch.where(new[:, None, :, None], c, code.view(torch.uint8)).view(code.dtype)
        s = torch.where(new[:, None, ::B], s.gather(2, at[..., ::B] // B), scale)
        out.append((c, s))
    rest = []
    for x, r in ((st["k"], st["rk"]), (st["v"], st["rv"])):
        at = behind.clamp(max=L - 1)[:, None, :, None].expand(-1, x.shape[1], -1, D)
        rest.append(torch.where(left[:, None, :, None], x.gather(2, at), r))
    return (out[0][0], out[1][0], out[0][1], out[1][1], rest[0], rest[1], (kv - full).int(),
            (held + full).int())


def _kvq_plain(st):
    case = st["case"]
    n, nkv, nq, B = case["seqs"], case["kv_heads"], case["q_heads"], case["block"]
    q = st["q"].float().view(n, nkv, nq // nkv, D) * SCALE
    held, tail = st["held"].long(), st["len"].long()
    low = (held + tail - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(held)
    sq = torch.einsum("tjgd,tjpd->tjgp", q, _values(st["kq"], st["ks"], B))
    sb = torch.einsum("tjgd,tjpd->tjgp", q, st["k"].float())
    at = torch.arange(sq.shape[-1], device="cuda")
    sq.masked_fill_(~((at >= low[:, None]) & (at < held[:, None]))[:, None, None], -math.inf)
    at = torch.arange(sb.shape[-1], device="cuda")
    sees = (at + held[:, None] >= low[:, None]) & (at < tail[:, None])
    sb.masked_fill_(~sees[:, None, None], -math.inf)
    m = torch.maximum(sq.amax(-1, keepdim=True), sb.amax(-1, keepdim=True))
    sq, sb = (sq - m).exp_(), (sb - m).exp_()
    l = sq.sum(-1, keepdim=True) + sb.sum(-1, keepdim=True)
    o = torch.einsum("tjgp,tjpd->tjgd", sq, _values(st["vq"], st["vs"], B))
    o = (o + torch.einsum("tjgp,tjpd->tjgd", sb, st["v"].float())) / l
    return o.reshape(n, nq, D).bfloat16(), (m + l.log()).reshape(n, nq)


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------
def work(case):
    nkv, n = case["kv_heads"], case["seqs"]
    if case["op"] == "rope":
        T, nq = case["tokens"], case["q_heads"]
        rows = T * (nq + (2 if case["append"] else 1) * nkv)
        return dict(bytes=rows * D * 4 + T * (12 if case["append"] else 4),
                    flops=T * (nq + nkv) * (3.0 * case["rot"] + (4.0 * D if case["norm"] else 0.0)))
    B = case["block"]
    if case["op"] == "fold":
        kv, _ = _fold_lengths(case)
        full = sum(m // B for m in kv) * nkv
        rest = sum(m % B for m in kv) * nkv
        return dict(bytes=full * (B * D * 6 + 8) + rest * D * 8 + 16 * n, flops=full * B * D * 4.0)
    held, tail = _kvq_lengths(case)
    nq, W = case["q_heads"], case["window"]
    coded = plain = 0
    for h, t in zip(held, tail):
        low = max(0, h + t - W) if W else 0
        coded += max(0, h - low)
        plain += t - max(0, low - h)
    return dict(bytes=nkv * (coded * D * 2 + coded // B * 8 + plain * D * 4) + n * nq * (D * 4 + 4) + 8 * n,
                flops=4.0 * D * nq * (coded + plain))


# ---------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _rope_exact(case, st)
    if case["op"] == "fold":
        return _fold_exact(case, st)
    return _kvq_exact(case, st)


def _rope_exact(case, st):
    half = case["rot"] // 2
    turn = torch.polar(torch.full((case["tokens"], half), _amplitude(case), dtype=torch.float64,
                                  device="cuda"), st["pos"].double()[:, None] * st["freq"])

    def rotate(x, gain):
        x = x.double().reshape(case["tokens"], -1, D)
        if gain is not None:
            x = x / (x.pow(2).mean(2, keepdim=True) + EPS).sqrt() * gain.double()
        y = x.clone()
        i = torch.arange(half, device="cuda")
        re, im = (i, i + half) if case["layout"] == "half" else (2 * i, 2 * i + 1)
        z = torch.complex(x[..., re], x[..., im]) * turn[:, None]
        y[..., re], y[..., im] = z.real, z.imag
        return y

    q, k = rotate(st["q"], st["gq"]).flatten(1), rotate(st["k"], st["gk"])
    if not case["append"]:
        return q, k.flatten(1)
    kc, vc = st["kc"].double(), st["vc"].double()
    v = st["v"].double().reshape(case["tokens"], -1, D)
    seq, slot = st["seq"].tolist(), st["slot"].tolist()
    first = 0
    for t in range(1, len(seq) + 1):                # a run of tokens goes to a run of slots
        if t == len(seq) or seq[t] != seq[first]:
            a, b = slot[first], slot[first] + t - first
            kc[seq[first], :, a:b] = k[first:t].transpose(0, 1)
            vc[seq[first], :, a:b] = v[first:t].transpose(0, 1)
            first = t
    return q, kc, vc


def _code64(y, fmt):
    """The nearest code's value (halves to even) of values already divided by the scale."""
    if fmt == "int8":
        return y.round()
    power = torch.tensor([2.0 ** e for e in range(-5, 10)], dtype=torch.float64, device=y.device)
    step = power[torch.bucketize(y.abs(), power, right=True)] / 16  # eight from a power to the next
    return (y / step).round() * step


def _fold_exact(case, st):
    B, fmt = case["block"], case["format"]
    kv, held = _fold_lengths(case)
    kq, vq, ks, vs, rk, rv = (st[k].double() for k in ("kq", "vq", "ks", "vs", "rk", "rv"))
    for t, (m, h) in enumerate(zip(kv, held)):
        f = m // B * B
        for x, code, scale, rest in ((st["k"], kq, ks, rk), (st["v"], vq, vs, rv)):
            y = x[t, :, :f].double().reshape(-1, f // B, B * D) if f else x[t, :, :0].double()
            amax = y.abs().amax(2).clamp(min=SMALLEST)
            if fmt == "int8":
                # the scale is a 32-bit number and so is the quotient that is rounded
                s = (amax / torch.full_like(amax, 127.0)).float().double()
                z = (y / s[..., None]).float().double()
            else:
                s = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
                z = y / s[..., None]
            code[t, :, h:h + f] = _code64(z, fmt).reshape(z.shape[0], f, D)
            scale[t, :, h // B:(h + f) // B] = s
            rest[t, :, :m - f] = x[t, :, f:m].double()
    full = torch.tensor([m // B * B for m in kv])
    return (kq, vq, ks, vs, rk, rv, (torch.tensor(kv) - full).int(), (torch.tensor(held) + full).int())


def _kvq_exact(case, st):
    nkv, nq, B = case["kv_heads"], case["q_heads"], case["block"]
    outs, lses = [], []
    for t, (h, m) in enumerate(zip(*_kvq_lengths(case))):
        low = max(0, h + m - case["window"]) if case["window"] else 0
        keys, vals = (torch.cat([c[t, :, :h].double() * s[t, :, :h // B].double().repeat_interleave(B, 1)[..., None],
                                 x[t, :, :m].double()], 1)[:, low:]
                      for c, s, x in ((st["kq"], st["ks"], st["k"]), (st["vq"], st["vs"], st["v"])))
        s = st["q"][t].double().view(nkv, -1, D) @ keys.mT / math.sqrt(D)
        outs.append((torch.softmax(s, -1) @ vals).reshape(nq, D))
        lses.append(torch.logsumexp(s, -1).reshape(nq))
    return torch.stack(outs), torch.stack(lses)
