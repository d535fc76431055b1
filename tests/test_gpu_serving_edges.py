"""GPU tests of the serving operators where a call differs from the ordinary one: another call's
workspace, scores at fp32's end, policies past a cache's capacity, layers that rotate.  Tolerances
are the bounds of oracle/serving.py unless a test derives its own."""
import dataclasses

import numpy as np
import pytest
import torch

from intra_spatial_pipelining_gb300 import sgp, synth
from oracle import layer as O
from oracle import serving as S
from tests import harness as H
from tests import test_gpu_serving as base
from tests.test_gpu_serving import D, NAN, Prefix, bf16, f64, ints, within

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------------
# prefix attention
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("nq,nkv,cap,sizes", [
    (64, 8, 1024, (375, 374, 93, 5, 1)), (16, 1, 1281, (512, 300, 2)), (5, 5, 257, (300, 299, 150, 31)),
    (12, 4, 130, (512, 200, 1))])
def test_prefix_attention_in_the_workspace_of_a_larger_call(nq, nkv, cap, sizes):
    """One workspace, sized for the first of `sizes` sequences and for a capacity of `cap`, serves the
    smaller calls, and none writes behind the size that its own arguments ask for."""
    dims = sgp.make_heads(nq, nkv)
    size = sgp.sgp_prefix_attention_workspace_bytes
    room = size(dims, sizes[0], cap, 2)
    buf = torch.empty(room + 65536, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(nq + cap)
    for T in sizes:
        for c in (cap, cap // 2):
            # a few long sequences and the others short: every chunk count, little to check
            own = [c if t < 3 else int(rng.integers(0, 9)) for t in range(T)]
            x = Prefix(T + c, T, nq, nkv, [70, 3], own, [t % 3 - 1 for t in range(T)], cap=c)
            need = size(dims, T, c, 2)
            assert need <= room
            for n in (room, need):
                buf.fill_(165)
                buf[:64] = 0
                x.ws = buf[:n]
                x.o.fill_(NAN)
                x.run()
                x.check()
                assert (buf[need:] == 165).all()


@pytest.mark.parametrize("size", [1, 2, 4])
def test_prefix_attention_raises_a_maximum_twice_in_a_step(size):
    """Scaled scores past 2^28, where fp32 steps by 32, and up to the largest that a call may have: the
    first raise of a row's maximum can miss the scores by more than a weight may exceed it, and the half
    is done a third time.

    One KV head to a pair (a, d): q = size (2^15, 2^7, 0 ...), keys (191 2^8, a) on the first 64
    positions and (191 2^8, a + d) on the next, so q.k = size (191 2^23 + 128 a), exact in fp32, and
    size 128 d more.  All weight is on the second half, in equal parts: o is the mean of its values.  The
    equal weights' rounding to bf16 and the result's are one half step each; the sums are of 64 terms."""
    pairs = [(2, 4), (2, 15), (2, 22), (2, 33), (2, 51), (2, 58), (13, 4), (13, 22), (20, 15), (24, 11),
             (24, 43), (6, 29), (17, 36), (20, 58), (0, 1), (100, 7)]
    x = Prefix(41, 3, len(pairs), len(pairs), [128], [0, 0, 0], [0, 0, 0])
    x.q.zero_()
    x.q[..., 0], x.q[..., 1] = size * 2.0 ** 15, size * 2.0 ** 7
    x.pk[0, :, :128] = 0.0
    x.pk[0, :, :128, 0] = 191.0 * 2 ** 8
    for j, (a, d) in enumerate(pairs):
        x.pk[0, j, :64, 1], x.pk[0, j, 64:128, 1] = a, a + d
    x.run()
    assert x.status() == sgp.SGP_OK
    v = f64(x.pv[0, :, 64:128])
    o, mag = v.mean(1), np.abs(v).mean(1)
    err = S.UBF * mag + S.UBF * np.abs(o) * (1 + S.UBF) + 256 * S.U32 * mag
    lse = np.array([size * (191 * 2 ** 23 + 128 * (a + d)) / 8 + np.log(64) for a, d in pairs])
    for t in range(3):
        within("o", x.o[t], o, err)
        # the scale, its product with the score, m + log2(sum) and the factor ln 2 round once each
        within("lse", x.lse[t], lse, 5 * S.U32 * np.abs(lse))


# ---------------------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("cap,budget", [(300, 300), (300, 301), (1024, 33000), (9000, 60000), (30000, 40000)])
def test_kv_evict_budget_past_the_capacity(cap, budget):
    """A budget that no source cache can exceed: every position stays, the rest of the target is new."""
    rng = np.random.default_rng(cap)
    lens = [cap, cap - 1, 0]
    k, v = bf16(rng, 3, 2, cap, D), bf16(rng, 3, 2, cap, D)
    acc = torch.from_numpy(rng.random((3, 2, cap))).float().cuda()
    for t, L in enumerate(lens):
        k[t, :, L:], v[t, :, L:], acc[t, :, L:] = NAN, NAN, NAN
    ko, vo = torch.full((2, 3, 2, budget + 1, D), 3.0, dtype=torch.bfloat16, device="cuda")
    ao = torch.full((3, 2, budget + 1), NAN, device="cuda")
    dims = sgp.make_heads(2, 2)
    ws = torch.full((sgp.sgp_kv_evict_workspace_bytes(dims, 3, budget),), 255, dtype=torch.uint8, device="cuda")
    ws[:64] = 0
    n, n_out = ints(lens), ints([-1] * 3)
    kept = torch.full((3, 2, budget), -9, dtype=torch.int32, device="cuda")
    sgp.sgp_kv_evict(dims, sgp.make_cache(k, v), sgp.make_cache(ko, vo), sgp.make_evict(budget, 2, 9), n, n_out,
                     acc, ao, kept, 3, ws)
    assert sgp.sgp_status_from_workspace(ws) == sgp.SGP_OK
    assert n_out.tolist() == lens
    for t, L in enumerate(lens):
        for out, src in ((ko, k), (vo, v)):
            assert torch.equal(out[t, :, :L], src[t, :, :L]) and (out[t, :, L:] == 3.0).all()
        assert torch.equal(ao[t, :, :L], acc[t, :, :L]) and not ao[t, :, L:].any()
        assert (kept[t, :, :L] == torch.arange(L, device="cuda")).all() and (kept[t, :, L:] == -1).all()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,cap,budget", [([300, 129, 40, 0], 310, 128), ([6000, 4500], 6001, 4096),
                                             ([9000, 64], 9100, 2000)])
def test_kv_evict_values_behind_a_length_are_nan(lens, cap, budget, in_place):
    """K, V and the weights behind a length hold NaN: none of it is moved or counted."""
    T, rng = len(lens), np.random.default_rng(budget)
    k, v = bf16(rng, T, 2, cap, D), bf16(rng, T, 2, cap, D)
    acc = torch.from_numpy(rng.exponential(1.0, (T, 2, cap))).float().cuda()
    for t, L in enumerate(lens):
        k[t, :, L:], v[t, :, L:], acc[t, :, L:] = NAN, NAN, NAN
    k0, v0, a0 = k.clone(), v.clone(), acc.cpu().numpy()
    ko, vo, ao = (k, v, acc) if in_place else (torch.empty_like(k), torch.empty_like(v), torch.empty_like(acc))
    dims = sgp.make_heads(2, 2)
    ws = torch.zeros(sgp.sgp_kv_evict_workspace_bytes(dims, T, budget), dtype=torch.uint8, device="cuda")
    n = ints(lens)
    sgp.sgp_kv_evict(dims, sgp.make_cache(k, v), sgp.make_cache(ko, vo), sgp.make_evict(budget, 3, 20), n, n, acc,
                     ao, None, T, ws)
    assert sgp.sgp_status_from_workspace(ws) == sgp.SGP_OK
    assert n.tolist() == [min(L, budget) for L in lens]
    for t, L in enumerate(lens):
        for j in range(2):
            at = torch.from_numpy(S.evict(a0[t, j], L, budget, 3, 20)).cuda()
            m = len(at)
            assert torch.equal(ko[t, j, :m], k0[t, j, at]) and torch.equal(vo[t, j, :m], v0[t, j, at])
            assert torch.isfinite(vo[t, j, :m]).all() and not ao[t, j, m:].any()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T,nkv,cap", [(2, 1, 4096), (2, 1, 4097), (40, 8, 4096), (40, 8, 4097)])
def test_kv_evict_where_the_selections_take_turns(T, nkv, cap, in_place):
    """Capacities on both sides of the border, few and many caches, lengths from none to all of it."""
    lens = [cap - (t * 611) % (cap + 1) for t in range(T)]
    base.test_kv_evict(T, nkv, lens, cap, 1000, 900, 3, 50, "ties", in_place)


# ---------------------------------------------------------------------------------------
# padded batches, and the ends of what the arguments may be
# ---------------------------------------------------------------------------------------
def test_rows_behind_the_last_sequence_are_left_as_they_were():
    """Every operator called for 5 sequences on tensors of 8; what lies behind is as it was, and what is
    only read there is NaN or out of range."""
    T, N = 5, 8
    own = [70, 0, 3, 129, 64]
    x = Prefix(61, N, 16, 2, [200], own + [1, 1, 1], [0, -1, 0, 0, -1, 0, 0, 0])
    x.q[T:], x.k[T:], x.v[T:] = NAN, NAN, NAN
    x.kv_len[T:], x.pof[T:] = 1 << 30, 1 << 30
    x.o.fill_(5.0)
    x.lse.fill_(5.0)
    sgp.sgp_prefix_attention(x.dims, x.cache, x.prefix, x.kv_len, x.q, x.o, x.lse, T, x.ws)
    assert x.status() == sgp.SGP_OK
    assert (x.o[T:] == 5.0).all() and (x.lse[T:] == 5.0).all()
    z = lambda t: np.nan_to_num(f64(t))
    o, lse, eo, el = S.prefix_attention(f64(x.q[:T]), z(x.k[:T]), z(x.v[:T]), own, z(x.pk), z(x.pv), [200],
                                        x.of[:T], 0)
    within("o", x.o[:T], o, eo)
    within("lse", x.lse[:T], lse, el)
    cap = x.cache.kv_cap
    acc = torch.full((N, 2, cap), 7.0, device="cuda")
    sgp.sgp_attention_weights(x.dims, x.cache, x.kv_len, x.q, x.lse, acc, T, x.ws)
    assert x.status() == sgp.SGP_OK and (acc[T:] == 7.0).all()
    add, err = S.attention_weights(f64(x.q[:T]), z(x.k[:T]), own, f64(x.lse[:T]))
    within("acc", acc[:T], 7.0 + add, err + S.U32 * (7.0 + add))
    ws = torch.zeros(sgp.sgp_kv_evict_workspace_bytes(x.dims, T, 32), dtype=torch.uint8, device="cuda")
    kept, a0, k0 = torch.full((N, 2, 32), -7, dtype=torch.int32, device="cuda"), f64(acc), x.k.clone()
    for to in (40, None):                                     # into another cache, then in place
        ko, vo = (x.k, x.v) if to is None else torch.full((2, N, 2, to, D), 3.0, dtype=torch.bfloat16, device="cuda")
        ao = acc if to is None else torch.full((N, 2, to), 3.0, device="cuda")
        behind = [t[T:].clone() for t in (ko, vo, ao, x.kv_len)]
        n_out = x.kv_len if to is None else torch.full_like(x.kv_len, -3)
        sgp.sgp_kv_evict(x.dims, x.cache, sgp.make_cache(ko, vo), sgp.make_evict(32, 2, 5), x.kv_len, n_out, acc,
                         ao, kept, T, ws)
        assert sgp.sgp_status_from_workspace(ws) == sgp.SGP_OK
        assert n_out[:T].tolist() == [min(n, 32) for n in own] and (kept[T:] == -7).all()
        for t, was in zip((ko, vo, ao), behind):
            assert torch.equal(t[T:].view(torch.uint8), was.view(torch.uint8))
        assert torch.equal(n_out[T:], behind[3] if to is None else torch.full_like(behind[3], -3))
        for t in range(T):
            for j in range(2):
                want = S.evict(a0[t, j], own[t], 32, 2, 5)
                assert kept[t, j, :len(want)].tolist() == want.tolist()
                assert torch.equal(ko[t, j, :len(want)], k0[t, j, torch.from_numpy(want).cuda()])
    rng = np.random.default_rng(3)
    a, b, xx, y = bf16(rng, 2, 8, 64), bf16(rng, 2, 96, 8), bf16(rng, N, 64), bf16(rng, N, 96)
    out, of = torch.full_like(y, 3.0), ints([0, 1, -1, 0, 1, 1 << 30, 0, -9])
    xx[T:], y[T:] = NAN, NAN
    sgp.sgp_lora_apply(sgp.make_lora(a, b), of, xx, y, out, T, x.ws)
    assert x.status() == sgp.SGP_OK and (out[T:] == 3.0).all()
    want, err = S.lora(f64(xx[:T]), f64(y[:T]), f64(a), f64(b), [1.0] * 2, [8] * 2, of[:T].tolist())
    within("y", out[:T], want, err)


@pytest.mark.parametrize("nq,nkv", [(1024, 1024), (2048, 512), (256, 16)])
def test_many_heads(nq, nkv):
    """As many KV heads as there may be, and as many query heads to one."""
    own = [65, 1, 0]
    x = Prefix(nq, 3, nq, nkv, [130, 3], own, [0, 1, -1])
    x.run()
    x.check()
    acc = torch.zeros(3, nkv, x.cache.kv_cap, device="cuda")
    sgp.sgp_attention_weights(x.dims, x.cache, x.kv_len, x.q, x.lse, acc, 3, x.ws)
    assert x.status() == sgp.SGP_OK
    add, err = S.attention_weights(f64(x.q), np.nan_to_num(f64(x.k)), own, f64(x.lse))
    within("acc", acc, add, err + S.U32 * add)
    assert not acc[1, :, 1:].any() and not acc[2].any()


@pytest.mark.parametrize("i,o,r", [(1 << 20, 32, 8), (32, 1 << 20, 8), (65536, 65568, 128)])
def test_lora_apply_wide(i, o, r):
    """The widest rows."""
    rng = np.random.default_rng(r + o)
    x, y = bf16(rng, 3, i), bf16(rng, 3, o)
    a, b = bf16(rng, 2, r, i, scale=i ** -0.5), bf16(rng, 2, o, r, scale=r ** -0.5)
    ws, of = torch.zeros(64, dtype=torch.uint8, device="cuda"), [1, -1, 1]
    want, err = S.lora(f64(x), f64(y), f64(a), f64(b), [1.0] * 2, [r] * 2, of)
    sgp.sgp_lora_apply(sgp.make_lora(a, b), ints(of), x, y, y, 3, ws)
    assert sgp.sgp_status_from_workspace(ws) == sgp.SGP_OK
    within("y", y, want, err)


# ---------------------------------------------------------------------------------------
# layers that rotate queries and keys, run op by op
# ---------------------------------------------------------------------------------------
THETA = 150000.0


class RopeLayer:
    """A layer with 24 sequences on a shared prompt of 333 positions (every sixth without), run op by
    op with its own rotation (base THETA) or without."""

    def __init__(self, seed, own):
        self.T, self.P, self.own = 24, 333, own
        wl = synth.WORKLOADS["gptoss_layer"].with_(n_tokens=self.T, kv_len=max(own) + 4)
        self.inp = H.make_inputs(wl, seed)
        self.s = s = wl.shape
        self.plain = H.dims(s)
        self.rotating = H.dims(dataclasses.replace(s, rope_theta=THETA))
        self.nq, self.nkv, self.G = s.n_q_heads, s.n_kv_heads, s.n_q_heads // s.n_kv_heads
        self.k, self.v = (t.clone() for t in self.inp.caches[0])
        self.cap = self.k.shape[2]
        self.layer = sgp.make_layer(self.inp.weights[0], self.k, self.v, 0)
        self.kv_len = ints(own)
        rng = np.random.default_rng(seed)
        # distances matter: keys as large as the layer's own scores allow
        self.pk_raw = rng.standard_normal((self.nkv, self.P, D))
        self.pv = bf16(rng, 1, self.nkv, self.P, D)
        self.of = [-1 if t % 6 == 5 else 0 for t in range(self.T)]
        self.pof = ints(self.of)
        self.ws = H.workspace(self.plain, self.T, self.cap)
        self.view = sgp.layer_views(self.plain, self.T, self.cap, self.ws)
        n = sgp.sgp_prefix_attention_workspace_bytes(self.plain, self.T, self.cap, 1)
        self.pws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        self.lse = torch.empty(self.T, self.nq, device="cuda")
        self.out = torch.empty_like(self.inp.x)

    def prompt(self, first):
        """The prompt with its keys rotated for first, first + 1, ..."""
        k = np.stack([O.rope(self.pk_raw[:, p], first + p, THETA) for p in range(self.P)], 1)
        self.pk = torch.from_numpy(k)[None].to(torch.bfloat16).cuda()
        self.prefix = sgp.make_prefix(self.pk, self.pv, ints([self.P]), self.pof)

    def qkv(self, dims):
        for op in (0, 1):
            sgp.sgp_layer_op(dims, self.layer, op, self.kv_len, self.inp.x, self.out, self.T, self.ws)
        return f64(self.view["q"]).reshape(self.T, self.nq, D)

    def attend(self):
        sgp.sgp_prefix_attention(self.plain, self.layer, self.prefix, self.kv_len,
                                 self.view["q"].view(self.T, self.nq, D),
                                 self.view["o"].view(self.T, self.nq, D), self.lse, self.T, self.pws)
        assert sgp.sgp_status_from_workspace(self.pws) == sgp.SGP_OK
        assert sgp.sgp_status_from_workspace(self.ws) == sgp.SGP_OK

    def check(self, q, keys):
        """q[t] [nq][d] and keys(t, j) [n][d] in 64 bits, values as they are stored."""
        for t in range(self.T):
            L = int(self.kv_len[t])
            for j in range(self.nkv):
                v = f64(self.v[t, j, :L])
                if self.of[t] >= 0:
                    v = np.concatenate([f64(self.pv[0, j]), v])
                h = slice(j * self.G, (j + 1) * self.G)
                o, lse, eo, el = S.attention(q[t, h], keys(t, j), v, 0)
                within("o", self.view["o"].view(self.T, self.nq, D)[t, h], o, eo)
                within("lse", self.lse[t, h], lse, el)


def pair_sum(x):
    """|a| + |b| of every rotated pair, in both of its places."""
    a = np.abs(x)
    s = a[..., :D // 2] + a[..., D // 2:]
    return np.concatenate([s, s], -1)


def test_shared_prompt_in_a_layer_that_rotates_by_its_slots():
    """The layer rotates for its own slots; the prompt's keys are stored for p - len.  Turned by the
    prompt's length, every vector stands at its true position: the prompt's at 0 ... len - 1, the own
    ones behind them."""
    x = RopeLayer(51, [200 - 7 * t for t in range(24)])
    x.prompt(-x.P)
    raw = x.qkv(x.plain)                                   # what the projection gives, not rotated
    for step in range(2):
        q = x.qkv(x.rotating)
        for t in range(x.T):
            # two roundings to bf16 (of a pair's elements before, of the result after); the angle
            want = O.rope(raw[t], int(x.kv_len[t]) - 1, THETA)
            bound = S.UBF * (np.abs(want) * (1 + S.UBF) + pair_sum(raw[t]) * (1 + S.UBF)) + 2.0 ** -16 * pair_sum(raw[t])
            assert (np.abs(q[t] - want) <= bound).all()
        x.attend()
        turn = [x.P if g >= 0 else 0 for g in x.of]
        pk = [np.stack([O.rope(k, x.P, THETA) for k in f64(x.pk[0, j])]) for j in range(x.nkv)]
        for j in range(x.nkv):                             # the stored prompt, turned: its true rotation
            want = np.stack([O.rope(x.pk_raw[j, p], p, THETA) for p in range(x.P)])
            assert (np.abs(pk[j] - want) <= S.UBF * pair_sum(f64(x.pk[0, j])) * (1 + S.UBF) * 2).all()

        def keys(t, j):
            own = O.rope(f64(x.k[t, j, :int(x.kv_len[t])]), turn[t], THETA)
            return np.concatenate([pk[j], own]) if x.of[t] >= 0 else own
        x.check(np.stack([O.rope(q[t], turn[t], THETA) for t in range(x.T)]), keys)
        x.kv_len += 1


def test_eviction_in_a_layer_whose_caller_rotates():
    """Own caches at positions 0 ... 199 are cut to 96; the layer projects without rotation, and q and
    the new key are rotated for the positions that the sequences really have, behind the prompt."""
    n, budget = 200, 96
    x = RopeLayer(52, [n] * 24)
    x.prompt(0)
    start = [x.P if g >= 0 else 0 for g in x.of]           # position of a sequence's first own token
    rng = np.random.default_rng(9)
    raw = rng.standard_normal((x.T, x.nkv, n, D))
    own = np.stack([np.stack([O.rope(raw[t, :, i], start[t] + i, THETA) for i in range(n)], 1) for t in range(x.T)])
    x.k[:, :, :n] = torch.from_numpy(own).to(torch.bfloat16)
    acc = torch.from_numpy(rng.exponential(1.0, (x.T, x.nkv, x.cap))).float().cuda()
    kept = torch.empty(x.T, x.nkv, budget, dtype=torch.int32, device="cuda")
    ews = torch.zeros(sgp.sgp_kv_evict_workspace_bytes(x.plain, x.T, budget), dtype=torch.uint8, device="cuda")
    sgp.sgp_kv_evict(x.plain, x.layer, x.layer, sgp.make_evict(budget, 4, 16), x.kv_len, x.kv_len, acc, acc, kept,
                     x.T, ews)
    assert sgp.sgp_status_from_workspace(ews) == sgp.SGP_OK
    stored = [[torch.from_numpy(own[t, j, kept[t, j].cpu().numpy()]).to(torch.bfloat16) for j in range(x.nkv)]
              for t in range(x.T)]
    for step in range(2):
        x.kv_len += 1
        slot = budget + step
        q = x.qkv(x.plain)
        new = f64(x.k[:, :, slot])
        # the caller's rotation, of the queries and of the row that the projection appended
        q = np.stack([O.rope(q[t], start[t] + n + step, THETA) for t in range(x.T)])
        new = np.stack([O.rope(new[t], start[t] + n + step, THETA) for t in range(x.T)])
        q, new = torch.from_numpy(q).to(torch.bfloat16), torch.from_numpy(new).to(torch.bfloat16)
        x.view["q"].copy_(q.reshape(x.T, -1))
        x.k[:, :, slot] = new.cuda()
        x.attend()
        for t in range(x.T):
            for j in range(x.nkv):
                stored[t][j] = torch.cat([stored[t][j], new[t, j][None]])

        def keys(t, j):
            k = f64(stored[t][j])
            return np.concatenate([f64(x.pk[0, j]), k]) if x.of[t] >= 0 else k
        x.check(f64(q), keys)
