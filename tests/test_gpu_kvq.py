"""GPU parity of norms and rotation, of folding into an 8-bit cache and of attention over it, against
their 64-bit definitions.  Tolerances are the bounds of oracle/kvq.py, which count the roundings; a fold
is exact.  What lies behind a length or before a window is NaN, and outputs start as NaN."""
import math

import numpy as np
import pytest
import torch

from intra_spatial_pipelining_gb300 import sgp, synth
from oracle import kvq as Q
from tests import harness as H
from tests.test_gpu_serving import bf16, f64, ints, within

pytestmark = pytest.mark.gpu

NAN = float("nan")
D = 64
DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def status(ws):
    return sgp.sgp_status_from_workspace(ws)


def word():
    return torch.zeros(64, dtype=torch.uint8, device="cuda")


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


# ---------------------------------------------------------------------------------------
# norms and rotation
# ---------------------------------------------------------------------------------------
ROPES = [
    # T, nq, nkv, rot, layout, scaling, norm, far
    (1, 64, 8, 64, "half", "none", False, 0),
    (1, 1, 1, 16, "interleaved", "linear", True, 5),
    (7, 8, 8, 32, "half", "turns", True, 131072),
    (33, 12, 4, 48, "half", "index", False, 1000000),
    (130, 15, 3, 48, "interleaved", "index", True, 2 ** 31 - 200),
    (515, 64, 8, 64, "interleaved", "turns", False, -300),
    (2500, 7, 7, 64, "half", "index", True, -2 ** 31),
    (2500, 48, 3, 16, "half", "none", False, 77),
    (700, 2048, 128, 64, "half", "none", True, 3),
]


class Rope:
    def __init__(self, T, nq, nkv, rot, layout, scaling, norm, far):
        rng = np.random.default_rng(T * 131 + nq)
        self.T, self.nq, self.nkv, self.eps = T, nq, nkv, 1e-5
        amp = 1.0 if scaling in ("none", "linear") else 1.3466
        kw = dict(factor=32.0, context=4096.0, turns_low=1.0, turns_high=32.0)
        self.rope = sgp.make_rope(rot, 150000.0, layout=layout, scaling=scaling, amplitude=amp, **kw)
        freq = Q.frequencies(rot, 150000.0, scaling, 32.0, 4096.0)
        assert np.allclose(np.array(self.rope.freq[:rot // 2]), freq, rtol=1e-14, atol=0)
        self.kw = dict(freq=freq, layout=layout, amplitude=np.float64(np.float32(amp)), eps=self.eps)
        self.dims = sgp.make_heads(nq, nkv)
        self.gq = (1 + bf16(rng, D, scale=0.3)).bfloat16() if norm else None
        self.gk = (1 + bf16(rng, D, scale=0.3)).bfloat16() if norm else None
        self.pos_list = [far + int(p) for p in rng.integers(0, 150, T)]
        self.pos = ints(self.pos_list)
        # rows of a projection with a gap behind them that nobody may touch
        self.width = (nq + 2 * nkv) * D
        self.qkv = bf16(rng, T + 1, self.width + 16, scale=2.0)
        self.q, self.k, self.v = (self.qkv[:, a * D:b * D] for a, b in
                                  ((0, nq), (nq, nq + nkv), (nq + nkv, nq + 2 * nkv)))
        self.ws = word()

    def want(self, x, gain):
        x = f64(x[:self.T]).reshape(self.T, -1, D)
        return Q.rope(x, self.pos_list, gain=None if gain is None else f64(gain), **self.kw)

    def check(self, name, got, x, gain):
        y, err = self.want(x, gain)
        within(name, got.reshape(y.shape), y, err)


@pytest.mark.parametrize("T,nq,nkv,rot,layout,scaling,norm,far", ROPES)
def test_qk_rope(T, nq, nkv, rot, layout, scaling, norm, far):
    x = Rope(T, nq, nkv, rot, layout, scaling, norm, far)
    qo = torch.full((T + 1, nq * D + 8), NAN, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((T + 1, nkv * D), NAN, dtype=torch.bfloat16, device="cuda")
    sgp.sgp_qk_rope(x.dims, x.rope, x.gq, x.gk, x.eps, x.pos, x.q, qo[:, :nq * D], x.k, ko, T, x.ws)
    assert status(x.ws) == sgp.SGP_OK
    x.check("q", qo[:T, :nq * D], x.q, x.gq)
    x.check("k", ko[:T], x.k, x.gk)
    assert qo[T].isnan().all() and qo[:, nq * D:].isnan().all() and ko[T].isnan().all()
    # in place, one side at a time
    was = x.qkv.clone()
    want = [qo[:T, :nq * D].clone(), ko[:T].clone()]
    sgp.sgp_qk_rope(x.dims, x.rope, x.gq, None, x.eps, x.pos, x.q, x.q, None, None, T, x.ws)
    sgp.sgp_qk_rope(x.dims, x.rope, None, x.gk, x.eps, x.pos, None, None, x.k, x.k, T, x.ws)
    assert torch.equal(x.q[:T], want[0]) and torch.equal(x.k[:T], want[1])
    assert torch.equal(x.v, was[:, (nq + nkv) * D:x.width]) and torch.equal(x.qkv[T], was[T])
    assert torch.equal(x.qkv[:, x.width:], was[:, x.width:])


@pytest.mark.parametrize("n,cap", [(1, 5000), (5, 700), (40, 130)])
@pytest.mark.parametrize("T,nq,nkv,rot,layout,scaling,norm,far", [ROPES[i] for i in (0, 2, 3, 5, 6)])
def test_qk_rope_append(T, nq, nkv, rot, layout, scaling, norm, far, n, cap):
    x = Rope(T, nq, nkv, rot, layout, scaling, norm, far)
    rng = np.random.default_rng(n)
    places = rng.choice(n * cap, T, replace=False)
    seq, slot = places // cap, places % cap
    lost = set(range(3, T, 7))                                # tokens without a place
    seq_in = ints([-1 - t if t in lost else int(s) for t, s in enumerate(seq)])
    kc, vc = (torch.full((n, nkv, cap, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = sgp.make_cache(kc, vc)
    qo = torch.full((T, nq * D), NAN, dtype=torch.bfloat16, device="cuda")
    sgp.sgp_qk_rope_append(x.dims, x.rope, x.gq, x.gk, x.eps, x.pos, x.q, qo, x.k, x.v, cache, n, seq_in,
                           ints(slot), T, x.ws)
    assert status(x.ws) == sgp.SGP_OK
    x.check("q", qo, x.q, x.gq)
    y, err = x.want(x.k, x.gk)
    stay = np.ones((n, cap), dtype=bool)
    for t in range(T):
        if t not in lost:
            stay[seq[t], slot[t]] = False
    live = [t for t in range(T) if t not in lost]
    at = torch.from_numpy(seq[live]).cuda(), torch.from_numpy(slot[live]).cuda()
    within("k", kc[at[0], :, at[1]], y[live], err[live])
    assert torch.equal(vc[at[0], :, at[1]].reshape(len(live), -1), x.v[:T][live])
    stay = torch.from_numpy(stay).cuda()
    for c in (kc, vc):
        assert (c.transpose(1, 2)[stay] == 5.0).all()
    # keys that stand in the cache already, and no queries: the same bits
    before, values = kc.clone(), vc.clone()
    kc.fill_(5.0)
    kc[at[0], :, at[1]] = x.k[:T][live].reshape(len(live), nkv, D)
    sgp.sgp_qk_rope_append(x.dims, x.rope, None, x.gk, x.eps, x.pos, None, None, None, None, cache, n, seq_in,
                           ints(slot), T, x.ws)
    assert status(x.ws) == sgp.SGP_OK
    assert torch.equal(kc, before) and torch.equal(vc, values)


@pytest.mark.parametrize("nkv", [15, 16, 17, 33, 100])
def test_qk_rope_append_of_many_kv_heads(nkv):
    """More rows of a token than a stage holds, from rows and in their slots."""
    T, n, cap = 300, 20, 16
    x = Rope(T, nkv, nkv, 64, "half", "none", True, 5)
    place = np.random.default_rng(nkv).permutation(n * cap)[:T]
    seq, slot = ints(place // cap), ints(place % cap)
    at = seq.long(), slot.long()
    kc, vc = (torch.full((n, nkv, cap, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qo = torch.full((T, nkv * D), NAN, dtype=torch.bfloat16, device="cuda")
    sgp.sgp_qk_rope_append(x.dims, x.rope, x.gq, x.gk, x.eps, x.pos, x.q, qo, x.k, x.v, sgp.make_cache(kc, vc), n, seq, slot, T, x.ws)
    x.check("q", qo, x.q, x.gq)
    x.check("k", kc[at[0], :, at[1]], x.k, x.gk)
    assert torch.equal(vc[at[0], :, at[1]].reshape(T, -1), x.v[:T])
    before, values = kc.clone(), vc.clone()
    kc[at[0], :, at[1]] = x.k[:T].reshape(T, nkv, D)
    qa = torch.full_like(qo, NAN)
    sgp.sgp_qk_rope_append(x.dims, x.rope, x.gq, x.gk, x.eps, x.pos, x.q, qa, None, None, sgp.make_cache(kc, vc), n, seq, slot, T, x.ws)
    assert torch.equal(qa, qo) and torch.equal(kc, before) and torch.equal(vc, values)
    assert status(x.ws) == sgp.SGP_OK


@pytest.mark.parametrize("T,nq,nkv,rot,layout,scaling,norm,far", [
    (9800, 36, 18, 64, "half", "none", True, 0),
    (9801, 2, 1, 48, "interleaved", "turns", False, 77),
    (100003, 1, 1, 64, "half", "none", True, 0)])
def test_qk_rope_of_many_tokens(T, nq, nkv, rot, layout, scaling, norm, far):
    """So many that they go round the warps, in the end more than 32 to a warp: into rows, into caches, and in
    the caches, the last two with tokens that have no place."""
    x = Rope(T, nq, nkv, rot, layout, scaling, norm, far)
    qo, ko = (torch.full((T, n * D), NAN, dtype=torch.bfloat16, device="cuda") for n in (nq, nkv))
    sgp.sgp_qk_rope(x.dims, x.rope, x.gq, x.gk, x.eps, x.pos, x.q, qo, x.k, ko, T, x.ws)
    some = np.unique(np.r_[0:T:97, T - 40:T])
    x.pos_list = [x.pos_list[t] for t in some]
    for name, got, rows, gain in (("q", qo, x.q, x.gq), ("k", ko, x.k, x.gk)):
        y, err = Q.rope(f64(rows[some]).reshape(len(some), -1, D), x.pos_list, gain=None if gain is None else f64(gain), **x.kw)
        within(name, got[some].view(y.shape), y, err)
    n, cap = 7, T // 7 + 1
    place = np.random.default_rng(T).permutation(n * cap)[:T]
    lost = np.arange(T) % 11 == 3
    seq, slot = ints([-1 if no else int(a) for a, no in zip(place // cap, lost)]), ints(place % cap)
    live = torch.from_numpy(np.flatnonzero(~lost)).cuda()
    at = seq[live].long(), slot[live].long()
    kc, vc = (torch.full((n, nkv, cap, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qa = torch.full_like(qo, NAN)
    sgp.sgp_qk_rope_append(x.dims, x.rope, x.gq, x.gk, x.eps, x.pos, x.q, qa, x.k, x.v, sgp.make_cache(kc, vc), n, seq, slot, T, x.ws)
    assert torch.equal(qa, qo)
    assert torch.equal(kc[at[0], :, at[1]].reshape(len(live), -1), ko[live])
    assert torch.equal(vc[at[0], :, at[1]].reshape(len(live), -1), x.v[live])
    assert (kc == 5.0).all(3).sum() == (n * cap - len(live)) * nkv
    before = kc.clone()
    kc[at[0], :, at[1]] = x.k[live].reshape(len(live), nkv, D)
    sgp.sgp_qk_rope_append(x.dims, x.rope, None, x.gk, x.eps, x.pos, None, None, None, None, sgp.make_cache(kc, vc), n, seq, slot, T, x.ws)
    assert torch.equal(kc, before) and status(x.ws) == sgp.SGP_OK


@pytest.mark.parametrize("T", [5, 700, 9900])
@pytest.mark.parametrize("rows_of_k", [False, True])
@pytest.mark.parametrize("with_q", [False, True])
@pytest.mark.parametrize("with_v", [False, True])
def test_qk_rope_append_of_any_parts(T, rows_of_k, with_q, with_v):
    """q or not, keys from rows or in their slots, values or not: what is there is as with all of them."""
    nq, nkv, n = 6, 3, 5
    cap = T // n + 2
    x = Rope(T, nq, nkv, 32, "interleaved", "none", True, 5)
    place = np.random.default_rng(T).permutation(n * cap)[:T]
    seq, slot = ints(place // cap), ints(place % cap)
    at = seq.long(), slot.long()
    caches = [torch.full((n, nkv, cap, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    qo, qa = (torch.full((T, nq * D), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sgp.sgp_qk_rope_append(x.dims, x.rope, x.gq, x.gk, x.eps, x.pos, x.q, qo, x.k, x.v, sgp.make_cache(*caches[:2]), n, seq, slot, T, x.ws)
    x.check("q", qo, x.q, x.gq)
    if not rows_of_k:
        caches[2][at[0], :, at[1]] = x.k[:T].reshape(T, nkv, D)
    sgp.sgp_qk_rope_append(x.dims, x.rope, x.gq, x.gk, x.eps, x.pos, x.q if with_q else None, qa if with_q else None,
                           x.k if rows_of_k else None, x.v if with_v else None, sgp.make_cache(*caches[2:]), n, seq, slot, T, x.ws)
    assert torch.equal(caches[2], caches[0])
    assert torch.equal(caches[3], caches[1]) if with_v else (caches[3] == 5.0).all()
    assert torch.equal(qa, qo) if with_q else qa.isnan().all()
    assert status(x.ws) == sgp.SGP_OK


def test_qk_rope_append_without_sequences_and_with_bad_places():
    """Token t goes to sequence t; a place out of range is reported, its caches stay, its q is turned."""
    T, nq, nkv, cap = 6, 8, 2, 9
    x = Rope(T, nq, nkv, 64, "half", "none", False, 0)
    kc, vc = (torch.full((T - 1, nkv, cap, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = sgp.make_cache(kc, vc)
    qo = torch.full((T, nq * D), NAN, dtype=torch.bfloat16, device="cuda")
    slot = ints([0, cap - 1, cap, -1, 4, 2])                  # the last one has no sequence
    sgp.sgp_qk_rope_append(x.dims, x.rope, None, None, 0.0, x.pos, x.q, qo, x.k, x.v, cache, T - 1, None, slot, T, x.ws)
    assert status(x.ws) == sgp.SGP_ERR_DEVICE_BOUNDS
    x.check("q", qo, x.q, None)
    y, err = x.want(x.k, None)
    put = [(0, 0), (1, cap - 1), (4, 4)]
    for t, s in put:
        within("k", kc[t, :, s], y[t], err[t])
        kc[t, :, s] = 5.0
    assert (kc == 5.0).all()


def test_qk_rope_values_of_every_size():
    """Rows of zeros, of small and of large numbers, infinities and NaN: only their own rows."""
    T, nq = 5, 2
    x = Rope(T, nq, 1, 64, "half", "none", True, 9)
    x.q[0] = 0.0
    x.q[1] = 2.0 ** -110
    x.q[2] *= 2.0 ** 54
    x.q[3, 5] = math.inf
    x.q[3, D + 7] = NAN
    qo = torch.empty(T, nq * D, dtype=torch.bfloat16, device="cuda")
    sgp.sgp_qk_rope(x.dims, x.rope, x.gq, None, x.eps, x.pos, x.q, qo, None, None, T, x.ws)
    y, err = x.want(torch.nan_to_num(x.q, 0.0, 0.0, 0.0), x.gq)
    for t in (0, 1, 2, 4):
        within("q", qo[t].view(nq, D), y[t], err[t])
    assert qo[3].view(nq, D).isnan().any(1).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [16, 32, 48])
def test_qk_rope_leaves_what_it_does_not_rotate(rot, layout):
    """Bit by bit without a norm: infinities, NaN with a payload, zeros of both signs, subnormals.  With one an
    infinity makes the numbers that are not rotated 0, with their signs, and itself NaN; a zero keeps its sign."""
    T, nq, nkv = 37, 6, 2
    x = Rope(T, nq, nkv, rot, layout, "none", True, 9)
    words = torch.from_numpy(np.random.default_rng(rot).integers(-2 ** 15, 2 ** 15, (T + 1, nq, D)).astype(np.int16))
    words[0, 0, rot:] = torch.tensor([0x7f80, -0x80, 0x7f81, -0x8000, 0, 1, -0x7fff, 0x7fff] * ((D - rot) // 8), dtype=torch.int16)
    q = words.cuda().view(torch.bfloat16).reshape(T + 1, nq * D)
    kc, vc = (torch.zeros(T, nkv, 3, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qo = torch.empty_like(q)
    sgp.sgp_qk_rope_append(x.dims, x.rope, None, None, 0.0, x.pos, q, qo, q[:, :nkv * D], None, sgp.make_cache(kc, vc), T,
                           None, ints([t % 3 for t in range(T)]), T, x.ws)
    assert status(x.ws) == sgp.SGP_OK
    assert torch.equal(qo[:T].view(torch.int16).view(T, nq, D)[..., rot:].cpu(), words[:T, :, rot:])
    t = torch.arange(T, device="cuda")
    assert torch.equal(kc[t, :, t % 3].view(torch.int16)[..., rot:].cpu(), words[:T, :nkv, rot:])
    # normed: one infinity to a head, in the part that is not rotated
    q = bf16(np.random.default_rng(1), T, nq, D)
    q[..., D - 6] = -0.0
    at = rot + (torch.arange(T * nq, device="cuda").view(T, nq) * 7) % (D - rot - 8)
    q.scatter_(2, at[..., None], math.inf)
    qo = torch.full_like(q, 5.0)
    sgp.sgp_qk_rope(x.dims, x.rope, x.gq, None, x.eps, x.pos, q.view(T, -1), qo.view(T, -1), None, None, T, x.ws)
    hit = torch.zeros_like(q, dtype=torch.bool).scatter_(2, at[..., None], True)
    assert torch.equal(qo.isnan(), hit)
    assert (qo[~hit] == 0).all()
    sign = q.signbit() ^ x.gq.signbit()
    assert torch.equal(qo.signbit()[..., rot:][~hit[..., rot:]], sign[..., rot:][~hit[..., rot:]])
    q.masked_fill_(hit, 1.0)
    sgp.sgp_qk_rope(x.dims, x.rope, x.gq, None, x.eps, x.pos, q.view(T, -1), qo.view(T, -1), None, None, T, x.ws)
    zero = qo[..., D - 6]
    assert (zero == 0).all() and torch.equal(zero.signbit(), sign[..., D - 6])


# ---------------------------------------------------------------------------------------
# fold
# ---------------------------------------------------------------------------------------
class Fold:
    """bf16 caches with lens, codes with held; NaN behind."""

    def __init__(self, seed, nkv, lens, held, block, fmt, cap=None, cap_q=None, scale=1.0):
        rng = np.random.default_rng(seed)
        self.T, self.nkv, self.lens, self.held, self.block, self.fmt = len(lens), nkv, list(lens), list(held), block, fmt
        T = self.T
        cap = cap or max(1, max(lens))
        cap_q = cap_q or (max(held) // block + max(lens) // block + 1) * block
        size = 2.0 ** rng.integers(-4, 5, (T, nkv, cap, 1))
        self.k = torch.from_numpy(rng.standard_normal((T, nkv, cap, D)) * size * scale).bfloat16().cuda()
        self.v = bf16(rng, T, nkv, cap, D, scale=scale)
        for t, n in enumerate(lens):
            if 0 <= n <= cap:
                self.k[t, :, n:], self.v[t, :, n:] = NAN, NAN
        raw = torch.from_numpy(rng.integers(0, 256, (2, T, nkv, cap_q, D)).astype(np.uint8)).cuda()
        self.kq, self.vq = (c.contiguous().view(DTYPE[fmt]) for c in raw)
        self.ks, self.vs = (torch.from_numpy(rng.standard_normal((T, nkv, cap_q // block))).float().cuda() for _ in range(2))
        self.dims = sgp.make_heads(nkv, nkv)
        self.ws = word()
        self.n, self.h = ints(lens), ints(held)
        self.before = [t.clone() for t in (self.kq, self.vq, self.ks, self.vs)]

    def run(self, in_place, stream=None, lengths="apart"):
        """The fold, and what its bf16 caches have to hold afterwards."""
        self.k0, self.v0 = self.k.clone(), self.v.clone()
        if in_place:
            rk, rv = self.k, self.v
        else:
            room = max(1, self.block - 1)
            rk, rv = (torch.full((len(self.lens), self.nkv, room, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.rest0 = [rk.clone(), rv.clone()]
        self.rest = [rk, rv]
        if lengths == "apart":
            self.n_out, self.h_out = torch.full_like(self.n, -5), torch.full_like(self.h, -5)
        else:
            self.n_out, self.h_out = self.n, self.h
        sgp.sgp_kvq_fold(self.dims, sgp.make_cache(self.k, self.v),
                         sgp.make_kvq(self.kq, self.vq, self.ks, self.vs), sgp.make_cache(rk, rv), self.n, self.h,
                         self.n_out, self.h_out, self.T, self.ws, stream)

    def check(self, left=()):
        """left: sequences that have to be as they were."""
        B = self.block
        want = [bits(t) for t in self.before[:2]], [t.cpu().numpy().copy() for t in self.before[2:]]
        rest = [bits(t) for t in self.rest0]
        for t in range(self.T):
            n, h = self.lens[t], self.held[t]
            if t in left:
                assert (int(self.n_out[t]), int(self.h_out[t])) == (n, h)
                continue
            f = n // B * B
            assert (int(self.n_out[t]), int(self.h_out[t])) == (n - f, h + f)
            for j in range(self.nkv):
                for i, x in enumerate((self.k0, self.v0)):
                    c, s = Q.quantise(f64(x[t, j, :f]), B, self.fmt)
                    want[0][i][t, j, h:h + f] = c
                    want[1][i][t, j, h // B:(h + f) // B] = s
                    rest[i][t, j, :n - f] = bits(x[t, j, f:n])
        for got, w in zip((self.kq, self.vq), want[0]):
            assert np.array_equal(bits(got), w)
        for got, w in zip((self.ks, self.vs), want[1]):
            assert np.array_equal(got.cpu().numpy(), w, equal_nan=True)
        for got, w in zip(self.rest, rest):
            assert np.array_equal(bits(got), w)


FOLDS = [
    (1, [0], [0]), (1, [1], [0]), (2, [127, 128, 129, 15, 16, 17], [0, 128, 256, 0, 128, 0]),
    (3, [5, 300, 31, 32, 33, 64, 257, 0], [128, 0, 0, 384, 128, 0, 0, 256]), (8, [1000, 777], [128, 0]),
    (1, [3001], [1280]),
]


@pytest.mark.parametrize("lengths", ["apart", "same"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_kvq_fold(block, fmt, in_place, lengths):
    for i, (nkv, lens, held) in enumerate(FOLDS):
        x = Fold(i + block, nkv, lens, held, block, fmt)
        x.run(in_place, lengths=lengths)
        assert status(x.ws) == sgp.SGP_OK
        x.check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_kvq_fold_of_many(fmt):
    lens = [(t * 37) % 130 for t in range(512)]
    x = Fold(5, 2, lens, [64 * (t % 5) for t in range(512)], 64, fmt)
    x.run(True, lengths="same")
    assert status(x.ws) == sgp.SGP_OK
    x.check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("block", [16, 64])
def test_kvq_fold_values(fmt, block):
    """Halves between codes, powers of two, the smallest and largest magnitudes, zeros, blocks of one
    sign; every bf16 number below 448 and a few blocks of one huge or tiny number among others."""
    n = 256
    x = Fold(1, 1, [n] * 6, [0] * 6, block, fmt, cap=n)
    every = torch.arange(0, 0x7f80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    some = every[(every <= 448) & (every > 2.0 ** -12)].cuda()
    pick = torch.from_numpy(np.random.default_rng(2).integers(0, len(some), n * D)).cuda()
    sign = torch.where(torch.arange(n * D, device="cuda") % 3 == 0, -1.0, 1.0)
    x.k[0, 0] = (some[pick] * sign).view(n, D).bfloat16()
    x.k[0, 0, ::block, 0] = 448.0                             # e4m3: scale 1
    x.v[0, 0] = torch.arange(n * D, device="cuda").view(n, D).remainder(255).sub(127).mul(0.5).bfloat16()
    x.v[0, 0, ::block, 0] = 127.0                             # int8: scale 1, every half a tie
    x.k[1], x.v[1] = 0.0, -0.0
    x.k[2] = every[torch.arange(n * D) % 200].view(n, D).cuda()   # below the smallest normal numbers
    x.v[2] = 3.3895e38
    x.k[3], x.v[3] = -448.0, 449.0
    x.k[4] *= 1e-30
    x.k[4, 0, 3::block, 5] = 1e30
    x.v[4] = 2.0 ** -112
    x.run(False)
    assert status(x.ws) == sgp.SGP_OK
    x.check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_kvq_fold_infinities_mark_their_block(fmt, block):
    x = Fold(3, 2, [2 * 128, 128], [0, 0], block, fmt)
    x.k[0, 0, block, 3] = math.inf                            # second block
    x.v[0, 1, 0, 0] = -math.inf
    x.k[1, 1, 127, 63] = NAN
    x.run(True)
    assert status(x.ws) == sgp.SGP_OK
    assert x.ks[0, 0, 1].isnan() and x.vs[0, 1, 0].isnan() and x.ks[1, 1, 128 // block - 1].isnan()
    x.check()


@pytest.mark.parametrize("in_place", [False, True])
def test_kvq_fold_bad_lengths_leave_the_sequence(in_place):
    x = Fold(4, 2, [64, -1, 65, 64, 100, 64, 130], [0, 0, 0, 16, 256, -32, 160], 32, "int8", cap=140, cap_q=256)
    x.lens[2] = 141
    x.n = ints(x.lens)
    x.run(in_place)
    assert status(x.ws) == sgp.SGP_ERR_DEVICE_BOUNDS
    # no room: 96 behind 256, 128 behind 160 of 256; 16 and -32 are no places
    x.check(left=(1, 2, 3, 4, 5, 6))
    assert torch.equal(x.k[1:].view(torch.int16), x.k0[1:].view(torch.int16))


# ---------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------
class Kvq:
    """Inputs of one attention over an 8-bit cache; what lies behind a length is NaN (codes that are NaN
    for e4m3, any for integers), and so are the scales there."""

    def __init__(self, seed, nq, nkv, held, tail, block, fmt, window=0, scale=1.0, cap=None, spread=3, tail_cap=None):
        rng = np.random.default_rng(seed)
        self.T, self.nq, self.nkv, self.block, self.fmt, self.window = len(held), nq, nkv, block, fmt, window
        self.held, self.tail = list(held), list(tail)
        T, cap = self.T, cap or max(held) + block
        code = rng.integers(0, 256, (2, T, nkv, cap, D)).astype(np.uint8)
        # values of about unit size: integers / 64; e4m3 numbers about 1, some of any size below 2
        unit = 1 / 64 if fmt == "int8" else 1.0
        if fmt == "e4m3":
            code = np.where(rng.random(code.shape) < 0.9, (code & 0x87) | (rng.integers(4, 8, code.shape) << 3),
                            code & 0xbf).astype(np.uint8)
        scales = (unit * 2.0 ** rng.uniform(-spread, 0, (2, T, nkv, cap // block))).astype(np.float32)
        total = np.array(held) + np.array(tail)
        self.low = [max(0, int(n) - window) if window else 0 for n in total]
        for t, n in enumerate(held):
            code[:, t, :, n:] = 0x7f
            scales[:, t, :, n // block:] = NAN
            b = min(self.low[t], n) // block                  # blocks that no query sees
            code[:, t, :, :b * block] = 0x7f
            scales[:, t, :, :b] = NAN
        self.kq, self.vq = (torch.from_numpy(c).cuda().view(DTYPE[fmt]) for c in code)
        self.ks, self.vs = (torch.from_numpy(s).cuda() for s in scales)
        tail_cap = tail_cap or max(1, max(tail) + 3)
        self.q = bf16(rng, T, nq, D, scale=scale)
        self.k, self.v = (bf16(rng, T, nkv, tail_cap, D) for _ in range(2))
        for t, n in enumerate(tail):
            hid = max(0, self.low[t] - held[t])
            for x in (self.k, self.v):
                x[t, :, n:], x[t, :, :hid] = NAN, NAN
        self.n, self.h = ints(tail), ints(held)
        self.dims = sgp.make_heads(nq, nkv)
        self.ws = torch.full((sgp.sgp_kvq_attention_workspace_bytes(self.dims, T),), 255, dtype=torch.uint8, device="cuda")
        self.ws[:64] = 0
        self.o = torch.full((T, nq, D), NAN, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((T, nq), NAN, device="cuda")
        self.kvq = sgp.make_kvq(self.kq, self.vq, self.ks, self.vs)
        self.cache = sgp.make_cache(self.k, self.v, window)

    def run(self, stream=None, lse=True, tail=True):
        sgp.sgp_kvq_attention(self.dims, self.kvq, self.h, self.cache if tail else None, self.n if tail else None,
                              self.q, self.o, self.lse if lse else None, self.T, self.ws, stream)

    def check(self, seqs=None):
        assert status(self.ws) == sgp.SGP_OK
        self.compare(seqs)

    def compare(self, seqs=None):
        G, B = self.nq // self.nkv, self.block
        q = f64(self.q)
        k, v = (np.nan_to_num(f64(x)) for x in (self.k, self.v))
        ks, vs = (np.nan_to_num(f64(s)) for s in (self.ks, self.vs))
        kc, vc = bits(self.kq), bits(self.vq)
        for t in range(self.T) if seqs is None else seqs:
            h, n = self.held[t], self.tail[t]
            for j in range(self.nkv):
                keys, vals = (np.concatenate([np.nan_to_num(Q.values(c[t, j, :h], s[t, j, :h // B], B, self.fmt)), x[t, j, :n]])
                              for c, s, x in ((kc, ks, k), (vc, vs, v)))
                at = slice(j * G, (j + 1) * G)
                sv = np.repeat(vs[t, j, :h // B], B)
                o, lse, eo, el = Q.attention(q[t, at], keys, vals, sv, self.low[t], h)
                within(f"o[{t},{j}]", self.o[t, at], o, eo)
                within(f"lse[{t},{j}]", self.lse[t, at], lse, el)


KVQ = {
    # nq, nkv, held, tail, window
    "one": (1, 1, [0], [1], 0),
    "one_block": (8, 1, [128], [0], 0),
    "empty_among_others": (16, 2, [0, 128, 0, 256], [0, 0, 5, 1], 0),
    "all_empty": (8, 2, [0, 0], [0, 0], 0),
    "groups_of_8": (64, 8, [512, 384], [40, 17], 0),
    "group_3": (9, 3, [128 * (t % 4) for t in range(20)], [t * 7 % 60 for t in range(20)], 0),
    "group_5": (10, 2, [1280, 0, 128], [33, 31, 32], 0),
    "group_12": (24, 2, [640, 256], [64, 65], 0),
    "group_16": (32, 2, [1024, 0, 384], [1, 130, 0], 0),
    "batch_512": (8, 1, [128 * (t % 9) for t in range(512)], [t % 40 for t in range(512)], 0),
    "more_tiles_than_shares": (4, 4, [1280 + 128 * (t % 7) for t in range(40)], [t % 70 for t in range(40)], 0),
    "long": (8, 1, [40960], [7], 0),
    "long_tail": (16, 2, [128, 0], [1030, 2000], 0),
    "window_in_tail": (8, 2, [256, 128, 0], [200, 130, 300], 100),
    "window_across": (16, 2, [1024, 128, 256], [40, 1, 64], 128),
    "window_of_one": (8, 1, [256, 0, 128], [3, 1, 0], 1),
    "window_odd": (8, 1, [640, 1152], [21, 2], 333),
    "window_wide": (8, 1, [256, 0], [9, 1], 100000),
}


# Short caches and caches with much room take different ways to the same sums.
ROOM = 4096


@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("name", KVQ)
def test_kvq_attention(name, fmt, room):
    nq, nkv, held, tail, window = KVQ[name]
    if room and len(held) > 100:
        pytest.skip("many sequences go one way in any case")
    for block in (16, 64, 128):
        x = Kvq(sum(map(ord, name)) + block, nq, nkv, held, tail, block, fmt, window, cap=max(held) + 128 + room if room else None)
        x.run()
        x.check()
        first = x.o.clone()
        x.run(lse=False)                                      # without lse, and again: the same bits
        assert torch.equal(first, x.o)


@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_kvq_attention_lengths_around_blocks_and_tiles(block, fmt, room):
    held = [block * i for i in range(0, 10)] * 2
    for window in (0, 1, 15, 16, 17, 63, 64, 65, 130):
        x = Kvq(block + window, 8, 1, held, [(t * 5) % 67 for t in range(20)], block, fmt, window,
                cap=1280 + room if room else None)
        x.run()
        x.check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_kvq_attention_without_a_bf16_cache(fmt):
    x = Kvq(3, 16, 2, [256, 0, 1024], [0, 0, 0], 32, fmt)
    x.run(tail=False)
    x.check()


@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("scale", [0.0, 1e-30, 40.0, 1e30])
def test_kvq_attention_query_sizes(fmt, scale, room):
    """Weights all alike, one position that takes all, queries near the ends of the range."""
    x = Kvq(9, 16, 2, [768, 256], [30, 0], 64, fmt, scale=min(scale, 1e3), cap=832 + room)
    if scale > 1e3:                                           # large queries on small keys
        x.q *= 1e27
        x.ks *= 2.0 ** -95
        x.k *= 2.0 ** -95
    x.run()
    x.check()


@pytest.mark.parametrize("room", [0, ROOM])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_kvq_attention_value_scales_far_apart(fmt, room):
    """Blocks whose values are 2^60 times others', where the weights make up for it: the small weights
    of the large values count as much as the large weights of the small ones."""
    x = Kvq(4, 8, 1, [512, 512], [20, 20], 64, fmt, spread=0, cap=576 + room)
    x.q[:] = 0
    x.q[:, :, 0] = 16.0                                       # the score: 2 k[0]
    unit = 0x40 if fmt == "e4m3" else 64                      # 2, and 64
    x.kq.view(torch.uint8).fill_(0)
    x.kq.view(torch.uint8)[..., 0] = unit
    x.ks[:, 0, :8] = 0
    x.ks[:, 0, 0] = 21.0 / (2 if fmt == "e4m3" else 64)       # weights differ by exp(42), about 2^60
    x.vs[:, 0, 0] *= 2.0 ** -60
    x.k[:, :, :, 0] = 0
    x.run()
    x.check()


@pytest.mark.parametrize("block", [32, 64])
@pytest.mark.parametrize("room", [0, ROOM])
def test_kvq_attention_scales_of_zero_and_nan(room, block):
    """A value scale of 0 gives values of 0; NaN in a scale that is seen shows in that head alone."""
    x = Kvq(5, 16, 2, [256, 256, 256], [5, 5, 5], block, "int8", cap=320 + room)
    x.vs[0, 0, 1] = 0
    x.vs[0, 1, :256 // block] = 0
    x.ks[1, 1, 2] = NAN
    x.vs[2, 0, 0] = NAN
    x.run()
    G = 8
    assert status(x.ws) == sgp.SGP_OK
    assert x.o[1, G:].isnan().all() and x.lse[1, G:].isnan().all() and x.o[2, :G].isnan().all()
    assert not x.o[0].isnan().any() and not x.o[1, :G].isnan().any() and not x.o[2, G:].isnan().any()
    x.compare(seqs=[0])


@pytest.mark.parametrize("room", [0, ROOM])
def test_kvq_attention_infinities_stay_with_their_sequence(room):
    """Infinite keys of one sequence and a NaN query head of another."""
    x = Kvq(6, 16, 2, [256, 128, 0, 128], [9, 40, 33, 7], 64, "e4m3", cap=320 + room)
    x.k[1, :, 3] = math.inf
    x.q[2, 5] = NAN
    x.q[3, 9] = NAN
    x.run()
    assert status(x.ws) == sgp.SGP_OK
    x.compare(seqs=[0])
    for t, h in ((2, 5), (3, 9)):
        assert x.o[t, h].isnan().all() and x.lse[t, h].isnan()
        assert torch.isfinite(x.o[t, [i for i in range(16) if i != h]]).all()


@pytest.mark.parametrize("room", [0, ROOM])
def test_kvq_attention_reports_bad_lengths(room):
    x = Kvq(7, 8, 1, [256, 128, 128, 64, 128, 128], [5, 7, 9, 11, 1, 1], 64, "int8", cap=320 + room)
    x.h[0], x.h[1], x.h[2] = 384 + room, -64, 100
    x.n[3], x.n[4] = -1, x.k.shape[2] + 1
    x.run()
    assert status(x.ws) == sgp.SGP_ERR_DEVICE_BOUNDS
    assert not x.o[:5].any() and (x.lse[:5] == -math.inf).all()
    x.compare(seqs=[5])
    x.h.copy_(ints(x.held))
    x.n.copy_(ints(x.tail))
    x.run()
    x.check()


def test_kvq_attention_output_may_be_the_query():
    for held in ([2048, 512], [256, 512, 64], [128 * (t % 3) for t in range(300)]):
        x = Kvq(8, 16, 2, held, [3] * len(held), 64, "e4m3")
        x.run()
        x.check()
        q = x.q.clone()
        sgp.sgp_kvq_attention(x.dims, x.kvq, x.h, x.cache, x.n, q, q, None, x.T, x.ws)
        assert torch.equal(q, x.o)


def test_kvq_attention_large_maxima_late():
    """Scores that rise along the cache: the running maximum is raised in every tile."""
    for fmt in ("e4m3", "int8"):
        x = Kvq(10, 8, 1, [4096], [40], 64, fmt)
        x.ks.copy_(torch.linspace(0.01, 1.0, x.ks.shape[2], device="cuda")[None, None] * (1 / 64 if fmt == "int8" else 1))
        x.q *= 3
        x.run()
        x.check()


@pytest.mark.parametrize("nq,nkv", [(1024, 1024), (2048, 128)])
def test_kvq_attention_many_heads(nq, nkv):
    x = Kvq(nq, nq, nkv, [128, 0, 64], [5, 1, 0], 64, "e4m3")
    x.run()
    x.check()


def test_kvq_attention_in_the_workspace_of_a_larger_call():
    x = Kvq(11, 16, 2, [128 * (t % 5) for t in range(9)], [t for t in range(9)], 64, "int8")
    big = torch.full((sgp.sgp_kvq_attention_workspace_bytes(x.dims, 512),), 255, dtype=torch.uint8, device="cuda")
    big[:64] = 0
    x.ws = big
    x.run()
    x.check()


@pytest.mark.parametrize("fmt,block,room", [("e4m3", 64, 0), ("int8", 16, ROOM)])
def test_rows_behind_the_last_sequence_are_left_as_they_were(fmt, block, room):
    T = 5
    x = Kvq(12, 16, 2, [128, 256, 0, 512, 128, 128, 128, 128], [3, 0, 0, 40, 64, 1, 1, 1], block, fmt, cap=640 + room)
    x.q[T:], x.k[T:], x.v[T:] = NAN, NAN, NAN
    x.n[T:], x.h[T:] = 1 << 30, 1 << 30
    x.o.fill_(5.0)
    x.lse.fill_(5.0)
    sgp.sgp_kvq_attention(x.dims, x.kvq, x.h, x.cache, x.n, x.q, x.o, x.lse, T, x.ws)
    x.check(seqs=range(T))
    assert (x.o[T:] == 5.0).all() and (x.lse[T:] == 5.0).all()
    y = Fold(12, 2, [130, 0, 64, 31, 200, 9, 9, 9], [0] * 8, block, fmt)
    y.T = T
    y.n[T:], y.h[T:] = 1 << 30, 1 << 30
    y.run(True)
    assert status(y.ws) == sgp.SGP_OK
    y.check()
    assert (y.n_out[T:] == -5).all() and (y.h_out[T:] == -5).all()
    assert torch.equal(y.k[T:].view(torch.int16), y.k0[T:].view(torch.int16))


def test_far_into_long_caches():
    """Rows past 2^32 bytes, of codes, of scales and of a bf16 cache."""
    T, nkv, cap, block = 2, 8, 1 << 22, 16                     # 4 GB of keys' codes
    x = Kvq(13, 64, nkv, [0, 0], [1, 1], block, "int8")
    kq, vq = (torch.zeros(T, nkv, cap, D, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((T, nkv, cap // block), 1 / 64, device="cuda") for _ in range(2))
    rng = np.random.default_rng(1)
    n = 320
    for t, j in ((0, 0), (1, 7)):
        for c in (kq, vq):
            c[t, j, cap - n:] = torch.from_numpy(rng.integers(-127, 128, (n, D)).astype(np.int8)).cuda()
    x.h = ints([cap, cap])
    x.kvq = sgp.make_kvq(kq, vq, ks, vs)
    x.cache = sgp.make_cache(x.k, x.v, n)
    x.run()
    assert status(x.ws) == sgp.SGP_OK
    for t, j in ((0, 0), (1, 7), (1, 3)):
        at = slice(8 * j, 8 * j + 8)
        keys, vals = (np.concatenate([f64(c[t, j, cap - n + 1:]) / 64, f64(y[t, j, :1])])
                      for c, y in ((kq, x.k), (vq, x.v)))
        o, lse, eo, el = Q.attention(f64(x.q[t, at]), keys, vals, np.full(n - 1, 1 / 64), 0, n - 1)
        within("o", x.o[t, at], o, eo)
        within("lse", x.lse[t, at], lse, el)
    # a fold at its end, and a key rotated into the last slot of a cache as long
    f = Fold(14, nkv, [40, 33], [0, 0], block, "int8")
    f.kq, f.vq, f.ks, f.vs = kq, vq, ks, vs
    f.h = ints([cap - 32, cap - 32])
    f.run(True)
    assert status(f.ws) == sgp.SGP_OK and f.h_out.tolist() == [cap, cap] and f.n_out.tolist() == [8, 1]
    for t in range(T):
        for j in range(nkv):
            c, s = Q.quantise(f64(f.k0[t, j, :32]), block, "int8")
            assert np.array_equal(bits(kq[t, j, cap - 32:]), c)
            assert np.array_equal(ks[t, j, -2:].cpu().numpy(), s.astype(np.float32))
    del kq, vq, f
    long = torch.zeros(2, nkv, 1 << 22, D, dtype=torch.bfloat16, device="cuda")
    r = Rope(2, 8, nkv, 64, "half", "none", False, 4000000)
    sgp.sgp_qk_rope_append(r.dims, r.rope, None, None, 0.0, r.pos, None, None, r.k, None,
                           sgp.make_cache(long, long), 2, ints([1, 0]), ints([(1 << 22) - 1, (1 << 22) - 2]), 2, r.ws)
    assert status(r.ws) == sgp.SGP_OK
    y, err = r.want(r.k, None)
    within("k", torch.stack([long[1, :, -1], long[0, :, -2]]), y, err)


# ---------------------------------------------------------------------------------------
# streams, graphs, the binding
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("room", [0, ROOM])
def test_captured_and_beside_another_stream(room):
    """Rotation, attention and fold captured into one graph, replayed while another stream runs the
    same operators in workspaces of its own."""
    def make(seed):
        x = Kvq(seed, 16, 2, [512, 0, 256], [70, 64, 3], 64, "e4m3", cap=1024 + room, tail_cap=200)
        x.slot = ints([69, 63, 2])
        return x, Rope(3, 16, 2, 64, "half", "none", False, 9)
    a, r = make(20)
    b, rb = make(21)

    def step(x, y, stream=None):
        sgp.sgp_qk_rope_append(x.dims, y.rope, None, None, 0.0, y.pos, y.q, x.q.view(3, -1), y.k, y.v, x.cache, 3,
                               None, x.slot, 3, y.ws, stream)
        sgp.sgp_kvq_attention(x.dims, x.kvq, x.h, x.cache, x.n, x.q, x.o, x.lse, 3, x.ws, stream)
        sgp.sgp_kvq_fold(x.dims, x.cache, x.kvq, x.cache, x.n, x.h, x.n, x.h, 3, y.ws, stream)

    def held(x):
        return (x.k, x.v, x.kq.view(torch.uint8), x.vq.view(torch.uint8), x.ks, x.vs, x.n, x.h)
    state = {id(x): [t.clone() for t in held(x)] for x in (a, b)}

    def reset(x):
        for t, s in zip(held(x), state[id(x)]):
            t.copy_(s)

    def result(x):
        return [t.clone() for t in (x.o, x.lse, *held(x))]
    want = {}
    for x, y in ((a, r), (b, rb)):
        step(x, y)
        want[id(x)] = result(x)
        assert status(x.ws) == sgp.SGP_OK and status(y.ws) == sgp.SGP_OK
        assert x.n.tolist() == [6, 0, 3] and x.h.tolist() == [576, 64, 256]
        reset(x)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        step(a, r)
    for _ in range(3):
        torch.cuda.synchronize()
        graph.replay()
        step(b, rb, side)
        torch.cuda.synchronize()
        for x in (a, b):
            for got, w in zip(result(x), want[id(x)]):
                assert torch.equal(got.view(torch.uint8), w.view(torch.uint8))
            reset(x)
    torch.cuda.synchronize()
    for w in (a.ws, b.ws, r.ws, rb.ws):
        assert status(w) == sgp.SGP_OK


def test_binding_checks_on_the_gpu():
    x = Kvq(30, 8, 1, [64], [3], 64, "e4m3")
    with pytest.raises(ValueError):
        sgp.make_kvq(x.kq.view(torch.uint8), x.vq.view(torch.uint8), x.ks, x.vs)
    with pytest.raises(ValueError):
        sgp.make_kvq(x.kq, x.vq[:, :, :64], x.ks, x.vs)
    with pytest.raises(ValueError):
        sgp.make_kvq(x.kq, x.vq, x.ks[..., :0], x.vs[..., :0])
    with pytest.raises(ValueError):
        sgp.make_kvq(x.kq, x.vq, x.ks.double(), x.vs)
    with pytest.raises(ValueError):
        sgp.make_kvq(x.kq.cpu(), x.vq, x.ks, x.vs)
    with pytest.raises(ValueError):
        sgp.sgp_kvq_attention(x.dims, x.kvq, x.h.long(), x.cache, x.n, x.q, x.o, x.lse, 1, x.ws)
    with pytest.raises(ValueError):
        sgp.sgp_kvq_attention(x.dims, x.kvq, x.h, x.cache, x.n, x.q, x.o, x.lse, 2, x.ws)
    with pytest.raises(ValueError):
        sgp.sgp_kvq_attention(sgp.make_heads(8, 2), x.kvq, x.h, x.cache, x.n, x.q, x.o, x.lse, 1, x.ws)
    with pytest.raises(sgp.SgpError):
        sgp.sgp_kvq_attention(x.dims, x.kvq, x.h, x.cache, x.n, x.q, x.o, x.lse, 1, x.ws[:256])
    with pytest.raises(ValueError):
        sgp.sgp_kvq_fold(x.dims, x.cache, x.kvq, x.cache, x.n, x.h, x.n, x.h, 2, x.ws)


# ---------------------------------------------------------------------------------------
# decode steps of a layer
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_decode_layer_with_an_8_bit_cache(fmt):
    """A prompt's bf16 cache is folded; then decode steps of a layer, op by op: QKV without rotation
    into the short bf16 cache, norms and rotation in place, attention over codes and bf16 positions, the
    rest of the layer, a fold.  Every result is checked on the inputs it had."""
    wl = synth.WORKLOADS["gptoss_layer"].with_(n_tokens=12, kv_len=300)
    inp = H.make_inputs(wl, 41)
    s, T, B = wl.shape, wl.n_tokens, 32
    d, nq, nkv = H.dims(s), s.n_q_heads, s.n_kv_heads
    G = nq // nkv
    rng = np.random.default_rng(3)
    pk, pv = (t.clone() for t in inp.caches[0])
    lens = [290 - 23 * t for t in range(T)]
    kv_len, kvq_len, count = ints(lens), ints([0] * T), ints(lens)
    tail_k, tail_v = (torch.full((T, nkv, B, D), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    codes = [torch.zeros(T, nkv, 512, D, dtype=torch.uint8, device="cuda").view(DTYPE[fmt]) for _ in range(2)]
    scales = [torch.full((T, nkv, 512 // B), NAN, device="cuda") for _ in range(2)]
    kvq, tail = sgp.make_kvq(*codes, *scales), sgp.make_cache(tail_k, tail_v)
    fws = word()
    sgp.sgp_kvq_fold(d, sgp.make_cache(pk, pv), kvq, tail, kv_len, kvq_len, kv_len, kvq_len, T, fws)
    assert kvq_len.tolist() == [n // B * B for n in lens] and kv_len.tolist() == [n % B for n in lens]
    layer = sgp.make_layer(inp.weights[0], tail_k, tail_v, 0)
    ws = H.workspace(d, T, B)
    view = sgp.layer_views(d, T, B, ws)
    aws = torch.zeros(sgp.sgp_kvq_attention_workspace_bytes(d, T), dtype=torch.uint8, device="cuda")
    lse = torch.empty(T, nq, device="cuda")
    rope = sgp.make_rope(64, 150000.0, scaling="index", factor=32.0, context=4096.0, amplitude=1.25)
    freq = Q.frequencies(64, 150000.0, "index", 32.0, 4096.0)
    gq, gk = ((1 + bf16(rng, D, scale=0.2)).bfloat16() for _ in range(2))
    x, out = inp.x.clone(), torch.empty_like(inp.x)
    op = lambda i: sgp.sgp_layer_op(d, layer, i, kv_len, x, out, T, ws)
    for step in range(40):
        kv_len += 1
        op(0), op(1)
        slot = kv_len - 1
        at = torch.arange(T, device="cuda"), slot.long()
        q0, k0 = f64(view["q"]).reshape(T, nq, D), f64(tail_k[at[0], :, at[1]])
        sgp.sgp_qk_rope_append(d, rope, gq, gk, 1e-5, count, view["q"], view["q"], None, None, tail, T, None, slot, T, fws)
        check = step % 13 == 0 or step > 37
        if check:
            kw = dict(pos=count.tolist(), freq=freq, amplitude=1.25, eps=1e-5)
            y, err = Q.rope(q0, gain=f64(gq), **kw)
            within("q", view["q"].view(T, nq, D), y, err)
            y, err = Q.rope(k0, gain=f64(gk), **kw)
            within("k", tail_k[at[0], :, at[1]], y, err)
        sgp.sgp_kvq_attention(d, kvq, kvq_len, tail, kv_len, view["q"], view["o"], lse, T, aws)
        if check:
            q = f64(view["q"]).reshape(T, nq, D)
            for t in range(T):
                h, n = int(kvq_len[t]), int(kv_len[t])
                for j in range(nkv):
                    keys, vals = (np.concatenate([Q.values(bits(c[t, j, :h]), f64(z[t, j, :h // B]), B, fmt), f64(w[t, j, :n])])
                                  for c, z, w in ((codes[0], scales[0], tail_k), (codes[1], scales[1], tail_v)))
                    hs = slice(j * G, (j + 1) * G)
                    sv = np.repeat(f64(scales[1][t, j, :h // B]), B)
                    o, z, eo, ez = Q.attention(q[t, hs], keys, vals, sv, 0, h)
                    within("o", view["o"].view(T, nq, D)[t, hs], o, eo)
                    within("lse", lse[t, hs], z, ez)
        for i in range(3, 9):
            op(i)
        x.copy_(out)
        n0, h0, kt = kv_len.tolist(), kvq_len.tolist(), tail_k.clone()
        sgp.sgp_kvq_fold(d, tail, kvq, tail, kv_len, kvq_len, kv_len, kvq_len, T, fws)
        for t in range(T):
            full = n0[t] == B
            assert (int(kv_len[t]), int(kvq_len[t])) == ((0, h0[t] + B) if full else (n0[t], h0[t]))
            if full and check:
                for j in range(nkv):
                    c, z = Q.quantise(f64(kt[t, j]), B, fmt)
                    assert np.array_equal(bits(codes[0][t, j, h0[t]:h0[t] + B]), c)
                    assert float(scales[0][t, j, h0[t] // B]) == float(np.float32(z[0]))
        count += 1
    assert torch.isfinite(out).all()
    for w in (ws, aws, fws):
        assert status(w) == sgp.SGP_OK
    assert (kvq_len + kv_len).tolist() == [n + 40 for n in lens]
