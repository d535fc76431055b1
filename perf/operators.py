"""The serving operators beside the decode layer, as they are measured: attention over a
prefix that a batch shares, the accumulated attention weight of cached positions, eviction
from the cache by that weight, and the low-rank adapters of many requests at once.

``run`` computes a case in plain torch (``own`` false) or through the library (``own`` true);
``exact`` is the definition in 64 bits.  Lengths follow from the case alone, values from the
seed.
"""
import math
import random

import numpy as np
import torch

own = False

D = 64                      # head dimension of the library's caches
SCALE = 1.0 / math.sqrt(D)


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # two requests on a short system prompt, a few own tokens: launch latency
        dict(name="prefix_pair", op="prefix", seqs=2, q_heads=64, kv_heads=8, prefixes=1,
             prefix=500, own=40, window=0, alone=0),
        # 64 requests on one long system prompt, ragged own contexts
        dict(name="prefix_gptoss", op="prefix", seqs=64, q_heads=64, kv_heads=8, prefixes=1,
             prefix=8192, own=1024, window=0, alone=0),
        # several tenants: prompts of different lengths, some requests without one
        dict(name="prefix_tenants", op="prefix", seqs=251, q_heads=32, kv_heads=4, prefixes=6,
             prefix=3001, own=611, window=0, alone=9),
        # a sliding-window layer of the same service: most of the prompt is out of reach
        dict(name="prefix_sliding", op="prefix", seqs=64, q_heads=64, kv_heads=8, prefixes=1,
             prefix=8192, own=200, window=128, alone=0),
        # a whole batch on one document, 8 query heads on one KV head
        dict(name="prefix_32k", op="prefix", seqs=512, q_heads=8, kv_heads=1, prefixes=1,
             prefix=32768, own=512, window=0, alone=0),
        # the weights of a few short caches
        dict(name="weights_small", op="weights", seqs=3, q_heads=64, kv_heads=8, length=577),
        # the weights of a full batch of long caches
        dict(name="weights_gptoss", op="weights", seqs=64, q_heads=64, kv_heads=8, length=8192),
        # two caches a block over their budget
        dict(name="evict_pair", op="evict", seqs=2, kv_heads=8, length=640, budget=512, sinks=4,
             recent=64),
        # prompts of up to 8192 positions cut to 4096 on their way into the decode cache
        dict(name="evict_gptoss", op="evict", seqs=64, kv_heads=8, length=8192, budget=4096,
             sinks=4, recent=512),
        # one request, one adapter, query projection
        dict(name="lora_one", op="lora", seqs=1, inputs=2880, outputs=4096, adapters=1, rank=16,
             alone=0),
        # 64 requests of 24 tenants, output projection, ranks up to 64
        dict(name="lora_tenants", op="lora", seqs=64, inputs=4096, outputs=2880, adapters=24,
             rank=64, alone=5),
        # a full batch on a few adapters, fused query/key/value projection
        dict(name="lora_batch", op="lora", seqs=512, inputs=2880, outputs=5120, adapters=8,
             rank=32, alone=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _draw(rng)
    while not _fits(case):
        for k in ("length", "prefix", "own", "budget", "recent", "seqs"):
            if case.get(k, 0) > 8:
                case[k] -= case[k] // 3
        if "prefixes" in case:
            case["prefixes"] = min(case["prefixes"], case["seqs"])
    return case


def _fits(case):
    """Whether a drawn case stays below the largest listed ones, in what it does and holds."""
    held = case["seqs"] * case.get("kv_heads", 0) * max(case.get("length", 0), case.get("own", 0))
    scores = case["seqs"] * case.get("q_heads", 0) * (case.get("prefix", 0) + case.get("own", 0))
    w = work(case)
    return (held <= 64 * 8 * 8192 and scores <= 512 * 8 * 32768 and w["bytes"] < 8e8
            and w["flops"] < 34e9)


def _draw(rng):
    op = rng.choice(["prefix", "prefix", "weights", "evict", "lora"])
    seqs = _log(rng, 1, 512)
    if op == "lora":
        return dict(op=op, seqs=seqs, inputs=64 * rng.randint(4, 64),
                    outputs=64 * rng.randint(4, 80), adapters=_log(rng, 1, 64),
                    rank=rng.choice([8, 16, 24, 32, 48, 64]), alone=rng.choice([0, 0, 3, 7]))
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "evict":
        length = _log(rng, 64, 32768)
        budget = max(16, int(length * rng.uniform(0.1, 0.9)))
        return dict(op=op, seqs=seqs, kv_heads=kv_heads, length=length, budget=budget,
                    sinks=rng.randint(0, 8), recent=int((budget - 8) * rng.uniform(0.0, 0.6)))
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 8, 12, 16])
    if op == "weights":
        return dict(op=op, seqs=seqs, q_heads=group * kv_heads, kv_heads=kv_heads,
                    length=_log(rng, 1, 32768))
    return dict(op=op, seqs=seqs, q_heads=group * kv_heads, kv_heads=kv_heads,
                prefixes=min(seqs, rng.choice([1, 1, 1, 2, 5, 8])), prefix=_log(rng, 1, 32768),
                own=_log(rng, 1, 4096), window=rng.choice([0, 0, 0, 128, 1000]),
                alone=rng.choice([0, 0, 4, 9]))


# ---------------------------------------------------------------------------------------
# lengths and indices: functions of the case, so that work() can count them
# ---------------------------------------------------------------------------------------
def _spread(case, what, n, lo, hi):
    rng = random.Random("%s %s" % (what, sorted((k, v) for k, v in case.items() if k != "name")))
    got = [rng.randint(lo, hi) for _ in range(n)]
    got[0] = hi
    return got


def _none(case, i):
    """Whether request i has no prefix or no adapter (every `alone`-th has none)."""
    return case["alone"] > 0 and i % case["alone"] == case["alone"] - 1


def _prefix_lists(case):
    """Prefix of every request (-1: none), prefix lengths, own lengths."""
    n = case["seqs"]
    of = [-1 if _none(case, i) else p
          for i, p in enumerate(_spread(case, "of", n, 0, case["prefixes"] - 1))]
    plen = _spread(case, "prefix", case["prefixes"], (case["prefix"] + 1) // 2, case["prefix"])
    olen = _spread(case, "own", n, 0 if n > 2 else 1, case["own"])
    return of, plen, olen


def _lengths(case):
    n = case["seqs"]
    return _spread(case, "length", n, 0 if n > 4 else (case["length"] + 1) // 2, case["length"])


def _evict_cap(case):
    return case["budget"] + 33      # the decode cache: the budget and room for new tokens


def _lora_lists(case):
    """Adapter of every request (-1: none) and the rank of every adapter."""
    of = [-1 if _none(case, i) else a
          for i, a in enumerate(_spread(case, "of", case["seqs"], 0, case["adapters"] - 1))]
    steps = case["rank"] // 8
    return of, [8 * r for r in _spread(case, "rank", case["adapters"], (steps + 1) // 2, steps)]


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        return t.normal_(0.0, scale, generator=g)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    st = dict(case=case, n=case["seqs"])
    if own:
        from intra_spatial_pipelining_gb300 import sgp
        st["sgp"] = sgp
    if case["op"] == "prefix":
        n, nkv, nq = case["seqs"], case["kv_heads"], case["q_heads"]
        of, plen, olen = _prefix_lists(case)
        st.update(of=ints(of), plen=ints(plen), olen=ints(olen), q=normal(n, nq, D),
                  pk=normal(case["prefixes"], nkv, case["prefix"], D),
                  pv=normal(case["prefixes"], nkv, case["prefix"], D),
                  k=normal(n, nkv, case["own"], D), v=normal(n, nkv, case["own"], D))
        if own:
            st["dims"] = sgp.make_heads(nq, nkv, D)
            st["cache"] = sgp.make_cache(st["k"], st["v"], case["window"])
            st["prefix"] = sgp.make_prefix(st["pk"], st["pv"], st["plen"], st["of"])
            nbytes = sgp.sgp_prefix_attention_workspace_bytes(
                st["dims"], n, case["own"], case["prefixes"])
            st["ws"] = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
            st["o"] = torch.empty_like(st["q"])
            st["lse"] = torch.empty(n, nq, dtype=torch.float32, device="cuda")
    elif case["op"] == "weights":
        n, nkv, nq, L = case["seqs"], case["kv_heads"], case["q_heads"], case["length"]
        st.update(olen=ints(_lengths(case)), q=normal(n, nq, D), k=normal(n, nkv, L, D))
        # what a few earlier steps added up, and this step's log-sum-exp of every query head
        acc = torch.empty(n, nkv, L, device="cuda").exponential_(1.0, generator=g)
        acc *= 4.0 * nq / nkv / L
        pos = torch.arange(L, device="cuda")
        st["acc"] = acc * (pos < st["olen"][:, None, None])
        st["lse"] = torch.cat([_lse64(st["q"][i], st["k"][i], int(m)).float()[None]
                               for i, m in enumerate(_lengths(case))])
        if own:
            st["dims"] = sgp.make_heads(nq, nkv, D)
            st["cache"] = sgp.make_cache(st["k"], st["k"])
            st["ws"] = torch.zeros(64, dtype=torch.uint8, device="cuda")
    elif case["op"] == "evict":
        n, nkv, L, cap = case["seqs"], case["kv_heads"], case["length"], _evict_cap(case)
        acc = torch.empty(n, nkv, L, device="cuda").exponential_(1.0, generator=g)
        # positions that no query has looked at yet carry no weight: ties
        acc *= torch.rand(n, nkv, L, device="cuda", generator=g) < 0.8
        st.update(olen=ints(_lengths(case)), k=normal(n, nkv, L, D), v=normal(n, nkv, L, D),
                  acc=acc, k_out=torch.zeros(n, nkv, cap, D, dtype=torch.bfloat16, device="cuda"))
        st.update(v_out=torch.zeros_like(st["k_out"]),
                  acc_out=torch.zeros(n, nkv, cap, device="cuda"), olen_out=torch.zeros_like(st["olen"]),
                  kept=torch.zeros(n, nkv, case["budget"], dtype=torch.int32, device="cuda"))
        if own:
            st["dims"] = sgp.make_heads(nkv, nkv, D)
            st["cache"] = sgp.make_cache(st["k"], st["v"])
            st["out"] = sgp.make_cache(st["k_out"], st["v_out"])
            st["policy"] = sgp.make_evict(case["budget"], case["sinks"], case["recent"])
            nbytes = sgp.sgp_kv_evict_workspace_bytes(st["dims"], n, case["budget"])
            st["ws"] = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    else:
        n, i, o, r = case["seqs"], case["inputs"], case["outputs"], case["rank"]
        of, ranks = _lora_lists(case)
        st.update(of=ints(of), ranks=ints(ranks), x=normal(n, i), y=normal(n, o),
                  a=normal(case["adapters"], r, i, scale=1.0 / math.sqrt(i)),
                  b=normal(case["adapters"], o, r, scale=1.0 / math.sqrt(r)),
                  scale=torch.rand(case["adapters"], device="cuda", generator=g) + 0.5)
        if own:
            st["lora"] = sgp.make_lora(st["a"], st["b"], st["scale"], st["ranks"])
            st["out"] = torch.empty_like(st["y"])
            st["ws"] = torch.zeros(64, dtype=torch.uint8, device="cuda")
    return st


def _lse64(q, k, length):
    """log sum exp of one request's scaled scores, [q_heads], from 64-bit sums."""
    nkv = k.shape[0]
    s = torch.einsum("jgd,jpd->jgp", q.double().view(nkv, -1, D), k[:, :length].double()) * SCALE
    return torch.logsumexp(s, -1).flatten()


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    if own:
        sgp = st["sgp"]
        if op == "prefix":
            sgp.sgp_prefix_attention(st["dims"], st["cache"], st["prefix"], st["olen"], st["q"],
                                     st["o"], st["lse"], st["n"], st["ws"])
            return st["o"], st["lse"]
        if op == "weights":
            sgp.sgp_attention_weights(st["dims"], st["cache"], st["olen"], st["q"], st["lse"],
                                      st["acc"], st["n"], st["ws"])
            return st["acc"]
        if op == "evict":
            sgp.sgp_kv_evict(st["dims"], st["cache"], st["out"], st["policy"], st["olen"],
                             st["olen_out"], st["acc"], st["acc_out"], st["kept"], st["n"],
                             st["ws"])
            return st["k_out"], st["v_out"], st["acc_out"], st["olen_out"], st["kept"]
        sgp.sgp_lora_apply(st["lora"], st["of"], st["x"], st["y"], st["out"], st["n"], st["ws"])
        return st["out"]
    if op == "prefix":
        return _prefix_plain(st)
    if op == "weights":
        return _weights_plain(st)
    if op == "evict":
        return _evict_plain(st)
    return _lora_plain(st)


def _prefix_plain(st):
    case = st["case"]
    n, nkv, nq = case["seqs"], case["kv_heads"], case["q_heads"]
    q = st["q"].float().view(n, nkv, nq // nkv, D) * SCALE
    of, olen = st["of"], st["olen"]
    plen = torch.where(of >= 0, st["plen"][of.clamp(min=0)], 0)
    total = plen + olen
    low = (total - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(total)
    # one prefix is read in place, several are gathered for each request
    if case["prefixes"] == 1:
        pk, pv = st["pk"][0].float(), st["pv"][0].float()
        sp = torch.einsum("tjgd,jpd->tjgp", q, pk)
    else:
        pk, pv = (t[of.clamp(min=0)].float() for t in (st["pk"], st["pv"]))
        sp = torch.einsum("tjgd,tjpd->tjgp", q, pk)
    so = torch.einsum("tjgd,tjpd->tjgp", q, st["k"].float())
    at = torch.arange(sp.shape[-1], device="cuda")
    sp.masked_fill_(~((at >= low[:, None]) & (at < plen[:, None]))[:, None, None], -math.inf)
    at = torch.arange(so.shape[-1], device="cuda")
    sees = (at + plen[:, None] >= low[:, None]) & (at < olen[:, None])
    so.masked_fill_(~sees[:, None, None], -math.inf)
    m = torch.maximum(sp.amax(-1, keepdim=True), so.amax(-1, keepdim=True))
    m = torch.where(m == -math.inf, 0.0, m)
    sp, so = (sp - m).exp_(), (so - m).exp_()
    l = sp.sum(-1, keepdim=True) + so.sum(-1, keepdim=True)
    if case["prefixes"] == 1:
        o = torch.einsum("tjgp,jpd->tjgd", sp, pv)
    else:
        o = torch.einsum("tjgp,tjpd->tjgd", sp, pv)
    o = (o + torch.einsum("tjgp,tjpd->tjgd", so, st["v"].float())) / torch.where(l == 0, 1.0, l)
    return o.reshape(n, nq, D).bfloat16(), (m + l.log()).reshape(n, nq)


def _weights_plain(st):
    case = st["case"]
    n, nkv, nq = case["seqs"], case["kv_heads"], case["q_heads"]
    q = st["q"].float().view(n, nkv, nq // nkv, D) * SCALE
    s = torch.einsum("tjgd,tjpd->tjgp", q, st["k"].float())
    p = (s - st["lse"].view(n, nkv, -1, 1)).exp_()
    sees = torch.arange(case["length"], device="cuda") < st["olen"][:, None]
    st["acc"] += torch.where(sees[:, None, None], p, 0.0).sum(2)
    return st["acc"]


def _evict_plain(st):
    case = st["case"]
    n, nkv, L, B, cap = (case["seqs"], case["kv_heads"], case["length"], case["budget"],
                         _evict_cap(case))
    olen = st["olen"].long()[:, None]
    at = torch.arange(L, device="cuda")
    key = st["acc"].masked_fill((at >= olen)[:, None], -math.inf)
    safe = (at < case["sinks"]) | ((at >= olen - case["recent"]) & (at < olen))
    key.masked_fill_(safe[:, None], math.inf)
    # heaviest first, ties to the lower position; within the budget nothing is dropped
    order = key.sort(dim=-1, descending=True, stable=True).indices[..., :min(B, L)]
    count = olen.clamp(max=B)
    kept = torch.where(torch.arange(order.shape[-1], device="cuda") < count[:, None], order, L)
    kept = kept.sort(dim=-1).values
    kept = torch.nn.functional.pad(kept, (0, cap - kept.shape[-1]), value=L)
    live = kept < L
    src = kept.clamp(max=L - 1)
    k, v = (torch.where(live[..., None], t.gather(2, src[..., None].expand(-1, -1, -1, D)), u)
            for t, u in ((st["k"], st["k_out"]), (st["v"], st["v_out"])))
    acc = torch.where(live, st["acc"].gather(2, src), 0.0)
    return k, v, acc, count[:, 0].int(), torch.where(live, kept, -1)[..., :B].int()


def _lora_plain(st):
    case = st["case"]
    of = st["of"].long()
    a = of.clamp(min=0)
    v = torch.einsum("ti,tri->tr", st["x"].float(), st["a"][a].float())
    live = torch.arange(case["rank"], device="cuda") < st["ranks"][a][:, None]
    v = torch.where(live & (of >= 0)[:, None], v, 0.0) * st["scale"][a][:, None]
    return (st["y"].float() + torch.einsum("tr,tor->to", v, st["b"][a].float())).bfloat16()


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------
def work(case):
    n = case["seqs"]
    if case["op"] == "prefix":
        nkv, nq, W = case["kv_heads"], case["q_heads"], case["window"]
        of, plen, olen = _prefix_lists(case)
        seen, first, rows = 0, {}, 0
        for p, o in zip(of, olen):
            P = plen[p] if p >= 0 else 0
            low = max(0, P + o - W) if W else 0
            seen += P + o - low
            rows += o - max(0, low - P)
            if low < P:
                first[p] = min(first.get(p, P), low)
        rows += sum(plen[p] - low for p, low in first.items())
        return dict(bytes=rows * nkv * D * 4 + n * nq * (D * 4 + 4) + 8 * n,
                    flops=4.0 * D * nq * seen)
    if case["op"] == "weights":
        nkv, nq, rows = case["kv_heads"], case["q_heads"], sum(_lengths(case))
        return dict(bytes=rows * nkv * (D * 2 + 8) + n * nq * (D * 2 + 4) + 4 * n,
                    flops=2.0 * D * nq * rows)
    if case["op"] == "evict":
        nkv, L = case["kv_heads"], _lengths(case)
        kept = sum(min(m, case["budget"]) for m in L)
        return dict(bytes=nkv * (4 * sum(L) + kept * D * 8 + 4 * n * (_evict_cap(case) + case["budget"]))
                    + 8 * n, flops=float(nkv * sum(L)))
    i, o = case["inputs"], case["outputs"]
    of, ranks = _lora_lists(case)
    return dict(bytes=2 * n * (i + 2 * o) + 4 * n + sum(2 * ranks[a] * (i + o) for a in set(of) if a >= 0),
                flops=sum(2.0 * ranks[a] * (i + o) for a in of if a >= 0))


# ---------------------------------------------------------------------------------------
# the definitions, in 64 bits, request by request
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    n = case["seqs"]
    if case["op"] == "prefix":
        of, plen, olen = _prefix_lists(case)
        nkv, nq = case["kv_heads"], case["q_heads"]
        outs, lses = [], []
        for t in range(n):
            P = plen[of[t]] if of[t] >= 0 else 0
            keys = torch.cat([st["pk"][max(of[t], 0), :, :P], st["k"][t, :, :olen[t]]], 1).double()
            vals = torch.cat([st["pv"][max(of[t], 0), :, :P], st["v"][t, :, :olen[t]]], 1).double()
            low = max(0, keys.shape[1] - case["window"]) if case["window"] else 0
            keys, vals = keys[:, low:], vals[:, low:]
            if keys.shape[1] == 0:
                outs.append(torch.zeros(nq, D, dtype=torch.float64, device="cuda"))
                lses.append(torch.full((nq,), -math.inf, dtype=torch.float64, device="cuda"))
                continue
            s = st["q"][t].double().view(nkv, -1, D) @ keys.mT / math.sqrt(D)
            outs.append((torch.softmax(s, -1) @ vals).reshape(nq, D))
            lses.append(torch.logsumexp(s, -1).reshape(nq))
        return torch.stack(outs), torch.stack(lses)
    if case["op"] == "weights":
        acc = st["acc"].double()
        for t, L in enumerate(_lengths(case)):
            keys = st["k"][t, :, :L].double()
            s = st["q"][t].double().view(case["kv_heads"], -1, D) @ keys.mT / math.sqrt(D)
            acc[t, :, :L] += (s - st["lse"][t].double().view(case["kv_heads"], -1, 1)).exp().sum(1)
        return acc
    if case["op"] == "evict":
        nkv, B, cap = case["kv_heads"], case["budget"], _evict_cap(case)
        acc = st["acc"].cpu().numpy()
        outs = [torch.zeros(n, nkv, cap, D, dtype=torch.float64, device="cuda") for _ in range(2)]
        w = np.zeros((n, nkv, cap))
        kept = np.full((n, nkv, B), -1, dtype=np.int32)
        count = []
        for t, L in enumerate(_lengths(case)):
            count.append(min(L, B))
            for j in range(nkv):
                if L <= B:
                    keep = np.arange(L)
                else:
                    a, z = case["sinks"], L - case["recent"]
                    mid = np.argsort(-acc[t, j, a:z], kind="stable")[:B - a - case["recent"]] + a
                    keep = np.concatenate([np.arange(a), np.sort(mid), np.arange(z, L)])
                kept[t, j, :len(keep)] = keep
                w[t, j, :len(keep)] = acc[t, j, keep]
                at = torch.from_numpy(keep).cuda()
                for u, src in zip(outs, (st["k"], st["v"])):
                    u[t, j, :len(keep)] = src[t, j, at].double()
        return outs[0], outs[1], w, np.array(count, dtype=np.int32), kept
    of, ranks = _lora_lists(case)
    y = st["y"].double()
    for t, a in enumerate(of):
        if a >= 0:
            r = ranks[a]
            v = st["a"][a, :r].double() @ st["x"][t].double()
            y[t] += st["scale"][a].double() * (st["b"][a, :, :r].double() @ v)
    return y
