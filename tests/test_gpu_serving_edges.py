"""GPU tests of the serving operators where a call differs from the ordinary one: another call's
workspace, scores at fp32's end, policies past a cache's capacity, layers that rotate.  Tolerances
are the bounds of oracle/serving.py unless a test derives its own."""
import numpy as np
import pytest
import torch

from intra_spatial_pipelining_gb300 import sgp
from oracle import serving as S
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


def test_prefix_attention_raises_a_maximum_twice_in_a_step():
    """Scaled scores past 2^28, where fp32 steps by 32: the first raise of a row's maximum can miss the
    scores by more than a weight may exceed it, and the half is done a third time.

    One KV head to a pair (a, d): q = (2^15, 2^7, 0 ...), keys (191 2^8, a) on the first 64 positions
    and (191 2^8, a + d) on the next, so q.k = 191 2^23 + 128 a, exact in fp32, and 128 d more.  All
    weight is on the second half, in equal parts: o is the mean of its values.  The equal weights'
    rounding to bf16 and the result's are one half step each; the sums are of 64 terms."""
    pairs = [(2, 4), (2, 15), (2, 22), (2, 33), (2, 51), (2, 58), (13, 4), (13, 22), (20, 15), (24, 11),
             (24, 43), (6, 29), (17, 36), (20, 58), (0, 1), (100, 7)]
    x = Prefix(41, 3, len(pairs), len(pairs), [128], [0, 0, 0], [0, 0, 0])
    x.q.zero_()
    x.q[..., 0], x.q[..., 1] = 2.0 ** 15, 2.0 ** 7
    x.pk[0, :, :128] = 0.0
    x.pk[0, :, :128, 0] = 191.0 * 2 ** 8
    for j, (a, d) in enumerate(pairs):
        x.pk[0, j, :64, 1], x.pk[0, j, 64:128, 1] = a, a + d
    x.run()
    assert x.status() == sgp.SGP_OK
    v = f64(x.pv[0, :, 64:128])
    o, mag = v.mean(1), np.abs(v).mean(1)
    err = S.UBF * mag + S.UBF * np.abs(o) * (1 + S.UBF) + 256 * S.U32 * mag
    lse = np.array([(191 * 2 ** 23 + 128 * (a + d)) / 8 + np.log(64) for a, d in pairs])
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
