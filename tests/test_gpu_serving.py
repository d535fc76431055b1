"""GPU parity of the serving operators against their 64-bit definitions.  Tolerances are the
bounds of oracle/serving.py, which count the roundings of each kernel; eviction is exact.
What lies behind a length, a rank or a row is NaN in every test, and outputs start as NaN."""
import numpy as np
import pytest
import torch

from intra_spatial_pipelining_gb300 import sgp, synth
from oracle import layer as O
from oracle import serving as S
from tests import harness as H

pytestmark = pytest.mark.gpu

NAN = float("nan")
D = 64


def bf16(rng, *shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(torch.bfloat16).cuda()


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def within(name, got, ref, bound):
    g = f64(got).reshape(ref.shape)
    fin = np.isfinite(ref)
    same = np.array_equal(np.isfinite(g), fin) and np.array_equal(g[~fin], ref[~fin])
    assert same, f"{name}: not finite elsewhere"
    over = float(np.max(np.abs(g[fin] - ref[fin]) - np.broadcast_to(bound, ref.shape)[fin], initial=-1.0))
    assert over <= 0, f"{name}: {over:.3e} over its bound"


class Prefix:
    """Inputs of one prefix attention; what lies behind a length is NaN."""

    def __init__(self, seed, T, nq, nkv, p_lens, own, of, window=0, cap=None, pcap=None, scale=1.0):
        rng = np.random.default_rng(seed)
        self.T, self.nq, self.nkv, self.window = T, nq, nkv, window
        self.own, self.p_lens, self.of = list(own), list(p_lens), list(of)
        cap = cap or max(1, max(own) + 3)
        self.q = bf16(rng, T, nq, D, scale=scale)
        self.k, self.v = bf16(rng, T, nkv, cap, D), bf16(rng, T, nkv, cap, D)
        for t, L in enumerate(own):
            self.k[t, :, L:] = NAN
            self.v[t, :, L:] = NAN
        self.pk = self.pv = None
        self.prefix = None
        if p_lens:
            pcap = pcap or max(1, max(p_lens) + 5)
            self.pk, self.pv = (bf16(rng, len(p_lens), nkv, pcap, D) for _ in range(2))
            for g, L in enumerate(p_lens):
                self.pk[g, :, L:] = NAN
                self.pv[g, :, L:] = NAN
            self.plen, self.pof = ints(p_lens), ints(of)
            self.prefix = sgp.make_prefix(self.pk, self.pv, self.plen, self.pof)
        self.kv_len = ints(own)
        self.dims = sgp.make_heads(nq, nkv)
        self.cache = sgp.make_cache(self.k, self.v, window)
        n = sgp.sgp_prefix_attention_workspace_bytes(self.dims, T, cap, len(p_lens))
        # only the status word needs to be clear
        self.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        self.ws[:64] = 0
        self.o = torch.full((T, nq, D), NAN, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((T, nq), NAN, dtype=torch.float32, device="cuda")

    def run(self, stream=None, lse=True, o=None):
        sgp.sgp_prefix_attention(self.dims, self.cache, self.prefix, self.kv_len, self.q,
                                 self.o if o is None else o, self.lse if lse else None, self.T, self.ws,
                                 stream)

    def status(self):
        return sgp.sgp_status_from_workspace(self.ws)

    def ref(self):
        z = lambda t: np.nan_to_num(f64(t))
        return S.prefix_attention(f64(self.q), z(self.k), z(self.v), self.own,
                                  None if self.pk is None else z(self.pk),
                                  None if self.pv is None else z(self.pv), self.p_lens, self.of,
                                  self.window)

    def check(self):
        assert self.status() == sgp.SGP_OK
        o, lse, eo, el = self.ref()
        within("o", self.o, o, eo)
        within("lse", self.lse, lse, el)


CASES = {
    # one prefix, lengths around a tile of positions and around none
    "one_token": (1, 1, 1, [1], [1], [0], 0),
    "no_own": (3, 8, 1, [127], [0, 0, 0], [0, 0, 0], 0),
    "no_prefix_positions": (3, 8, 1, [0], [5, 1, 0], [0, 0, 0], 0),
    "tile": (2, 8, 2, [128], [1, 2], [0, 0], 0),
    "tile_plus_one": (2, 16, 2, [129], [130, 7], [0, 0], 0),
    "no_prefix_at_all": (4, 16, 2, [], [1, 0, 1030, 64], [-1] * 4, 0),
    # group sizes that do not divide a tile of rows, more sequences than one tile takes
    "group_3": (100, 3, 1, [300], [t % 5 for t in range(100)], [0] * 100, 0),
    "group_5": (53, 10, 2, [257], [t % 7 for t in range(53)], [0] * 53, 0),
    "group_7": (38, 7, 1, [640], [1] * 38, [0] * 38, 0),
    "group_12": (45, 24, 2, [513], [t % 3 for t in range(45)], [0] * 45, 0),
    "group_16": (17, 32, 2, [385], [9] * 17, [0] * 17, 0),
    "batch_512": (512, 8, 1, [1500], [t % 11 for t in range(512)], [0] * 512, 0),
    # several prefixes, one of them empty, one that nobody has, members anywhere, some without
    "tenants": (61, 16, 2, [700, 0, 129, 64, 1], [(t * 37) % 90 for t in range(61)],
                [(0, 2, -1, 1, 4, 0, 2)[t % 7] for t in range(61)], 0),
    "each_its_own": (40, 8, 1, [t * 13 for t in range(40)], [t % 4 for t in range(40)],
                     list(range(39, -1, -1)), 0),
    "long_own": (2, 16, 2, [200], [2100, 1024], [0, -1], 0),
    # windows: inside the own cache, across both, past the whole, of one
    "window_own": (5, 8, 1, [300], [200, 128, 129, 500, 1100], [0] * 5, 128),
    "window_across": (6, 16, 2, [1000], [0, 1, 60, 127, 128, 3], [0] * 6, 128),
    "window_tenants": (9, 8, 2, [900, 40, 130], [0, 5, 70, 9, 0, 100, 3, 2, 1],
                       [0, 1, 2, 0, -1, 2, 1, 0, 2], 100),
    "window_wide": (4, 8, 1, [50], [3, 0, 70, 9], [0] * 4, 100000),
    "window_1": (4, 8, 1, [50], [3, 0, 70, 1], [0, 0, 0, -1], 1),
}


@pytest.mark.parametrize("name", CASES)
def test_prefix_attention(name):
    T, nq, nkv, p_lens, own, of, window = CASES[name]
    x = Prefix(sum(map(ord, name)), T, nq, nkv, p_lens, own, of, window)
    x.run()
    x.check()
    first = x.o.clone()
    x.run(lse=False)                              # without lse, and again: the same bits
    assert torch.equal(first, x.o)


@pytest.mark.parametrize("T,nq,nkv,p_lens,own,of,window", [
    (64, 64, 8, [4096], [(t * 53) % 600 for t in range(64)], [0] * 64, 0),
    (300, 8, 1, [9000, 2000], [(t * 7) % 90 for t in range(300)], [t % 2 for t in range(300)], 0),
    (128, 32, 4, [5000], [(t * 5) % 128 for t in range(128)], [0] * 128, 3000)])
def test_prefix_attention_same_bits_every_time(T, nq, nkv, p_lens, own, of, window):
    """Every SM busy for many steps: a buffer taken too early would show as another result."""
    x = Prefix(77, T, nq, nkv, p_lens, own, of, window)
    x.run()
    assert x.status() == sgp.SGP_OK
    o, lse = x.o.clone(), x.lse.clone()
    other = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(60):
        x.o.zero_()
        x.run()
        other += (x.o != o).any() | (x.lse != lse).any()
    assert int(other) == 0
    keep = [0, T // 2, T - 1]
    y = Prefix(77, T, nq, nkv, p_lens, own, of, window)
    z = lambda t: np.nan_to_num(f64(t))
    want = S.prefix_attention(f64(y.q[keep]), z(y.k[keep]), z(y.v[keep]), [own[t] for t in keep], z(y.pk),
                              z(y.pv), p_lens, [of[t] for t in keep], window)
    within("o", o[keep], want[0], want[2])
    within("lse", lse[keep], want[1], want[3])


def test_prefix_attention_large_scores():
    """Scores of a few hundred: the running maximum moves by more than fp32's exponent range of
    a weight, and most weights vanish."""
    x = Prefix(5, 9, 8, 1, [900], [t * 30 for t in range(9)], [0] * 9, scale=40.0)
    x.run()
    x.check()


def test_prefix_attention_rising_scores():
    """Keys along the query, longer with the position: every tile of positions raises the maximum."""
    x = Prefix(6, 33, 8, 1, [1100], [4] * 33, [0] * 33)
    x.q[:] = x.q[:1, :1]
    ramp = torch.linspace(0.0, 12.0, 1100, device="cuda")[:, None]
    x.pk[0, 0, :1100] = (x.q[0, 0].float() * ramp / 8).bfloat16()
    x.run()
    x.check()
    x.pk[0, 0, :1100] = x.pk[0, 0, :1100].flip(0)     # and falling
    x.run()
    x.check()


def test_prefix_attention_infinite_keys_in_other_rows():
    """Infinite or NaN values of one sequence's own cache reach no other sequence."""
    x = Prefix(7, 4, 8, 1, [140], [20, 20, 20, 20], [0] * 4)
    x.k[2, :, 3] = float("inf")
    x.v[1, :, 5] = NAN
    x.run()
    assert torch.isnan(x.o[1]).any()
    x.k[2, :, 3] = 0.0
    keep = [0, 3]
    o, lse, eo, el = x.ref()
    within("o", x.o[keep], o[keep], eo[keep])
    within("lse", x.lse[keep], lse[keep], el[keep])


def test_prefix_attention_output_may_be_the_query():
    a = Prefix(8, 20, 16, 2, [300], [t for t in range(20)], [0] * 20)
    a.run()
    want = a.o.clone()
    a.run(o=a.q)
    assert torch.equal(a.q, want)


def test_prefix_attention_reports_bad_lengths_and_indices():
    x = Prefix(9, 6, 8, 1, [200, 100], [10] * 6, [0, 1, 0, 1, 0, 1])
    x.kv_len.copy_(ints([10, -1, 10, 10, 1 << 30, 10]))
    x.pof.copy_(ints([0, 1, 2, -7, 0, 1 << 30]))
    x.run()
    assert x.status() == sgp.SGP_ERR_DEVICE_BOUNDS
    x.own, x.of = [10, 0, 10, 10, 0, 10], [0, 1, -1, -1, 0, -1]
    o, lse, eo, el = x.ref()
    within("o", x.o, o, eo)
    within("lse", x.lse, lse, el)
    x.plen.copy_(ints([-5, 1 << 30]))
    x.run()
    assert x.status() == sgp.SGP_ERR_DEVICE_BOUNDS
    x.of = [-1] * 6
    o, lse, eo, el = x.ref()
    within("o", x.o, o, eo)
    within("lse", x.lse, lse, el)
    assert x.status() == sgp.SGP_OK              # reading the status cleared it


def test_prefix_attention_captured_and_beside_another_stream():
    """Two captured calls with a workspace each, replayed at the same time as an eager call on a
    third stream, on inputs that change between replays."""
    xs = [Prefix(20 + i, 40, 16, 2, [600, 200], [(t * 7) % 50 for t in range(40)],
                 [(t * 3) % 2 for t in range(40)]) for i in range(3)]
    for x in xs:
        x.run()
    torch.cuda.synchronize()
    graphs = []
    for x in xs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for rep in range(3):
        for x in xs:
            x.q.copy_(bf16(np.random.default_rng(100 + rep), 40, 16, D))
            x.o.fill_(NAN)
            x.kv_len.copy_(ints([(t * 7 + rep) % 50 for t in range(40)]))
            x.own = [(t * 7 + rep) % 50 for t in range(40)]
            for t, L in enumerate(x.own):            # one more position holds numbers now
                x.k[t, :, :L] = torch.nan_to_num(x.k[t, :, :L])
                x.v[t, :, :L] = torch.nan_to_num(x.v[t, :, :L])
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        xs[2].run(stream=streams[2])
        torch.cuda.synchronize()
        for x in xs:
            x.check()


def test_operators_behind_other_nodes_of_a_graph():
    """Each operator directly behind a copy, a kernel of another stream that joins, and one another;
    what they write is read by the next node."""
    x = Prefix(31, 30, 16, 2, [400], [(t * 7) % 50 + 1 for t in range(30)], [0] * 30)
    rng = np.random.default_rng(8)
    a, b = bf16(rng, 2, 16, 1024), bf16(rng, 2, 1024, 16)
    lora, of, ws = sgp.make_lora(a, b), ints([t % 2 for t in range(30)]), torch.zeros(64, dtype=torch.uint8, device="cuda")
    cap, budget = x.cache.kv_cap, 20
    acc, acc2 = torch.zeros(30, 2, cap, device="cuda"), torch.zeros(30, 2, budget, device="cuda")
    to = [torch.zeros(30, 2, budget, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ews = torch.zeros(sgp.sgp_kv_evict_workspace_bytes(x.dims, 30, budget), dtype=torch.uint8, device="cuda")
    q_in, lens, n_out = torch.empty_like(x.q), x.kv_len.clone(), ints([0] * 30)
    side = torch.cuda.Stream()

    def step():
        s = torch.cuda.current_stream()
        side.wait_stream(s)
        with torch.cuda.stream(side):
            lens2 = lens.clone()                                 # a copy, on another branch
            acc.zero_()
        x.q.copy_(q_in)
        s.wait_stream(side)
        sgp.sgp_lora_apply(lora, of, x.q.view(30, -1), x.q.view(30, -1), xq.view(30, -1), 30, ws)
        sgp.sgp_prefix_attention(x.dims, x.cache, x.prefix, lens2, xq, x.o, x.lse, 30, x.ws)
        sgp.sgp_attention_weights(x.dims, x.cache, lens2, xq, x.lse, acc, 30, ws)
        side.wait_stream(s)
        with torch.cuda.stream(side):
            summed = acc.sum()                                   # reads beside the eviction
        sgp.sgp_kv_evict(x.dims, x.cache, sgp.make_cache(*to), sgp.make_evict(budget, 1, 4), lens2, n_out,
                         acc, acc2, None, 30, ews)
        s.wait_stream(side)
        return [t.clone() for t in (x.o, x.lse, acc, acc2, n_out, to[0], summed)]

    xq = torch.empty_like(x.q)
    q_in.copy_(bf16(rng, 30, 16, D))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for rep in range(4):
        q_in.copy_(bf16(rng, 30, 16, D))
        lens.copy_(ints([(t * 7 + rep) % 50 + 1 if (t * 7 + rep) % 50 < x.own[t] else x.own[t] for t in range(30)]))
        for t in (x.o, acc, acc2, xq, *to):
            t.fill_(0)
        want = step()
        torch.cuda.synchronize()
        for t in (x.o, acc, acc2, xq, *to):
            t.fill_(0)
        graph.replay()
        graph.replay()                                           # directly behind one another
        torch.cuda.synchronize()
        for status in (x.ws, ws, ews):
            assert sgp.sgp_status_from_workspace(status) == sgp.SGP_OK
        for got, ref in zip(outs, want):
            assert torch.equal(got, ref)
        x.q.copy_(xq)                                            # what the attention was given
        x.own = lens.tolist()
        x.check()


def test_prefix_attention_far_into_long_caches():
    """Element offsets past 2^31 in the own cache and in the prefix: a window at their ends."""
    cap, W = (1 << 25) + 300, 200
    x = Prefix(11, 2, 8, 1, [10], [70, 3], [0, 0], W)
    own = [cap - 5, 60]
    k = torch.zeros(2, 1, cap, D, dtype=torch.bfloat16, device="cuda")
    pk = torch.zeros(2, 1, cap, D, dtype=torch.bfloat16, device="cuda")
    v, pv = torch.zeros_like(k), torch.zeros_like(pk)
    rng = np.random.default_rng(12)
    for t in (k, v):
        t[0, 0, own[0] - W:own[0]] = bf16(rng, W, D)
        t[1, 0, :60] = bf16(rng, 60, D)
    for t in (pk, pv):
        t[1, 0, cap - 9 - W:cap - 9] = bf16(rng, W, D)
    dims = sgp.make_heads(8, 1)
    prefix = sgp.make_prefix(pk, pv, ints([cap, cap - 9]), ints([1, 1]))
    ws = torch.zeros(sgp.sgp_prefix_attention_workspace_bytes(dims, 2, cap, 2), dtype=torch.uint8,
                     device="cuda")
    sgp.sgp_prefix_attention(dims, sgp.make_cache(k, v, W), prefix, ints(own), x.q, x.o, x.lse, 2, ws)
    assert sgp.sgp_status_from_workspace(ws) == sgp.SGP_OK
    for t in range(2):
        if t == 0:
            ks, vs = k[0, 0, own[0] - W:own[0]], v[0, 0, own[0] - W:own[0]]
        else:
            a = cap - 9 - (W - 60)
            ks, vs = (torch.cat([p[1, 0, a:cap - 9], c[1, 0, :60]]) for p, c in ((pk, k), (pv, v)))
        o, lse, eo, el = S.attention(f64(x.q[t]), f64(ks), f64(vs), 0)
        within("o", x.o[t], o, eo)
        within("lse", x.lse[t], lse, el)


# ---------------------------------------------------------------------------------------
# accumulated attention weights
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,nq,nkv,lens,cap", [
    (1, 1, 1, [1], 1), (2, 8, 1, [64, 65], 70), (3, 16, 2, [0, 63, 200], 201),
    (5, 24, 2, [1, 127, 128, 129, 700], 701), (33, 15, 3, [(t * 29) % 150 for t in range(33)], 150),
    (512, 8, 1, [t % 90 for t in range(512)], 91), (1, 64, 8, [5000], 5000), (4, 32, 2, [70] * 4, 81)])
def test_attention_weights(T, nq, nkv, lens, cap):
    rng = np.random.default_rng(T * 1000 + nq)
    q, k = bf16(rng, T, nq, D), bf16(rng, T, nkv, cap, D)
    for t, L in enumerate(lens):
        k[t, :, L:] = NAN
    lse = np.full((T, nq), -np.inf, dtype=np.float32)
    for t, L in enumerate(lens):
        for h in range(nq):
            if L:
                s = f64(q[t, h]) @ f64(k[t, h // (nq // nkv), :L]).T / 8.0
                lse[t, h] = np.log(np.exp(s).sum()) + 0.25        # a prefix takes its share
    if T > 1:
        lse[1, 0] = -np.inf                                       # a head that attended nothing
    old = torch.from_numpy(rng.random((T, nkv, cap))).float().cuda()
    acc = old.clone()
    dims, ws = sgp.make_heads(nq, nkv), torch.zeros(64, dtype=torch.uint8, device="cuda")
    lt = torch.from_numpy(lse).cuda()
    sgp.sgp_attention_weights(dims, sgp.make_cache(k, k), ints(lens), q, lt, acc, T, ws)
    assert sgp.sgp_status_from_workspace(ws) == sgp.SGP_OK
    add, err = S.attention_weights(f64(q), np.nan_to_num(f64(k)), lens, lse.astype(np.float64))
    want = f64(old) + add
    within("acc", acc, want, err + S.U32 * np.abs(want))
    for t, L in enumerate(lens):
        assert torch.equal(acc[t, :, L:], old[t, :, L:])          # behind the length: untouched


def test_attention_weights_bad_length_and_long_cache():
    cap = (1 << 25) + 77                                          # element offsets past 2^31
    k = torch.zeros(2, 1, cap, D, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(4)
    tail = bf16(rng, 50, D)
    k[1, 0, cap - 50:] = tail
    q = bf16(rng, 2, 8, D)
    lse = torch.full((2, 8), 3.0, device="cuda")
    acc = torch.zeros(2, 1, cap, device="cuda")
    dims, ws = sgp.make_heads(8, 1), torch.zeros(64, dtype=torch.uint8, device="cuda")
    sgp.sgp_attention_weights(dims, sgp.make_cache(k, k), ints([cap + 1, cap]), q, lse, acc, 2, ws)
    assert sgp.sgp_status_from_workspace(ws) == sgp.SGP_ERR_DEVICE_BOUNDS
    assert not acc[0].any()                                       # out of range: nothing is added
    add, err = S.attention_weights(f64(q[1:]), f64(tail)[None, None], [50], f64(lse[1:]))
    within("tail", acc[1, 0, cap - 50:], add[0, 0], err[0, 0])
    zero = 8 * np.exp(-3.0)
    got = f64(acc[1, 0, :cap - 50])
    assert np.abs(got - zero).max() <= zero * 64 * S.U32


# ---------------------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------------------
def evict_inputs(seed, T, nkv, lens, cap, kind):
    rng = np.random.default_rng(seed)
    k, v = bf16(rng, T, nkv, cap, D), bf16(rng, T, nkv, cap, D)
    acc = rng.exponential(1.0, (T, nkv, cap)).astype(np.float32)
    if kind == "ties":
        acc = np.floor(acc * 2) / 2
    elif kind == "equal":
        acc[:] = 1.25
    elif kind == "odd":
        pick = rng.integers(0, 8, acc.shape)
        for i, x in enumerate((np.nan, np.inf, -np.inf, -0.0, 0.0, -1.5, 1e-42)):
            acc[pick == i] = x
    elif kind == "falling":
        acc = np.sort(acc, -1)[..., ::-1].copy()
    for t, L in enumerate(lens):
        acc[t, :, L:] = np.nan
        k[t, :, L:] = NAN
    return k, v, torch.from_numpy(acc).cuda()


EVICTIONS = [
    (1, 1, [1], 1, 1, 1, 0, 0, "plain"), (2, 2, [9, 8], 9, 12, 8, 1, 1, "plain"),
    (3, 1, [300, 0, 129], 300, 200, 128, 4, 32, "plain"), (3, 2, [300, 40, 129], 310, 77, 77, 0, 0, "ties"),
    (4, 2, [513, 64, 65, 900], 901, 70, 64, 0, 64, "plain"), (2, 1, [700, 650], 700, 640, 600, 599, 1, "odd"),
    (2, 3, [700, 650], 700, 640, 333, 5, 17, "odd"), (2, 1, [1000, 999], 1000, 500, 400, 0, 0, "equal"),
    (2, 2, [1000, 999], 1000, 500, 1, 0, 0, "falling"), (1, 1, [8192], 8192, 8000, 8000, 3, 7, "plain"),
    (1, 2, [9000], 9001, 4100, 4097, 4, 100, "ties"), (1, 1, [32768], 32768, 20000, 20000, 0, 0, "plain"),
    (1, 1, [70001], 70005, 33000, 33000, 2, 2, "ties"), (1, 1, [70001], 70005, 69999, 69999, 0, 5, "odd"),
    (512, 1, [t % 60 for t in range(512)], 60, 31, 30, 2, 8, "plain"),
    # both selections either side of where they take turns
    (3, 2, [5000, 4097, 1], 5000, 4600, 4500, 7, 90, "odd"), (2, 1, [8193, 6000], 8193, 2000, 2000, 1, 0, "equal"),
    (304, 1, [4100 - 13 * t for t in range(304)], 4100, 2100, 2049, 3, 100, "ties")]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T,nkv,lens,cap,cap_out,budget,sink,recent,kind", EVICTIONS)
def test_kv_evict(T, nkv, lens, cap, cap_out, budget, sink, recent, kind, in_place):
    k, v, acc = evict_inputs(budget, T, nkv, lens, cap, kind)
    k0, v0, a0 = k.clone(), v.clone(), acc.cpu().numpy()
    if in_place:
        cap_out, ko, vo, ao = cap, k, v, acc
        if budget > cap:
            pytest.skip("the budget is past the source's capacity")
    else:
        ko, vo = torch.full((2, T, nkv, cap_out, D), 3.0, dtype=torch.bfloat16, device="cuda")
        ao = torch.full((T, nkv, cap_out), NAN, device="cuda")
    before_k, before_v = ko.clone(), vo.clone()
    dims = sgp.make_heads(nkv, nkv)
    ws = torch.full((sgp.sgp_kv_evict_workspace_bytes(dims, T, budget),), 255, dtype=torch.uint8,
                    device="cuda")
    ws[:64] = 0
    n_in = ints(lens)
    n_out = n_in if in_place or T == 4 else torch.full_like(n_in, -1)   # the lengths in place, or not
    kept = torch.full((T, nkv, budget), -9, dtype=torch.int32, device="cuda") if T != 3 else None
    sgp.sgp_kv_evict(dims, sgp.make_cache(k, v), sgp.make_cache(ko, vo), sgp.make_evict(budget, sink, recent),
                     n_in, n_out, acc, ao, kept, T, ws)
    assert sgp.sgp_status_from_workspace(ws) == sgp.SGP_OK
    assert n_out.tolist() == [min(L, budget) for L in lens]
    bits = lambda t: t.view(torch.int16)
    for t, L in enumerate(lens):
        for j in range(nkv):
            want = S.evict(a0[t, j], L, budget, sink, recent)
            n, at = len(want), torch.from_numpy(want).cuda()
            if kept is not None:
                assert kept[t, j, :n].tolist() == want.tolist(), (t, j)
                assert (kept[t, j, n:] == -1).all()
            assert torch.equal(bits(ko[t, j, :n]), bits(k0[t, j, at])), (t, j)
            assert torch.equal(bits(vo[t, j, :n]), bits(v0[t, j, at])), (t, j)
            assert np.array_equal(f64(ao[t, j, :n]), a0[t, j, want].astype(np.float64), equal_nan=True)
            assert not ao[t, j, n:].any()                    # a new position starts at zero
            assert torch.equal(bits(ko[t, j, n:]), bits(before_k[t, j, n:]))
            assert torch.equal(bits(vo[t, j, n:]), bits(before_v[t, j, n:]))


def test_kv_evict_bad_lengths_leave_the_sequence():
    k, v, acc = evict_inputs(1, 3, 2, [50, 50, 50], 50, "plain")
    k0, a0 = k.clone(), acc.clone()
    n = ints([51, 50, -1])
    dims = sgp.make_heads(2, 2)
    ws = torch.zeros(sgp.sgp_kv_evict_workspace_bytes(dims, 3, 20), dtype=torch.uint8, device="cuda")
    c = sgp.make_cache(k, v)
    sgp.sgp_kv_evict(dims, c, c, sgp.make_evict(20, 2, 5), n, n, acc, acc, None, 3, ws)
    assert sgp.sgp_status_from_workspace(ws) == sgp.SGP_ERR_DEVICE_BOUNDS
    assert n.tolist() == [51, 20, -1]
    for t in (0, 2):
        assert torch.equal(k[t], k0[t]) and torch.equal(acc[t], a0[t])


def test_kv_evict_far_into_a_long_cache():
    """Element offsets past 2^31: the last positions of a long cache move to its front."""
    cap = (1 << 25) + 40
    k = torch.zeros(2, 1, cap, D, dtype=torch.bfloat16, device="cuda")
    tail = bf16(np.random.default_rng(2), 30, D)
    k[1, 0, cap - 30:] = tail
    v = k.clone()
    acc = torch.zeros(2, 1, cap, device="cuda")
    acc[1, 0, cap - 30:] = torch.arange(30, device="cuda") + 1.0
    n = ints([5, cap])
    dims = sgp.make_heads(1, 1)
    ws = torch.zeros(sgp.sgp_kv_evict_workspace_bytes(dims, 2, 25), dtype=torch.uint8, device="cuda")
    c = sgp.make_cache(k, v)
    sgp.sgp_kv_evict(dims, c, c, sgp.make_evict(25, 1, 4), n, n, acc, acc, None, 2, ws)
    assert sgp.sgp_status_from_workspace(ws) == sgp.SGP_OK
    assert n.tolist() == [5, 25]
    assert torch.equal(k[1, 0, 1:25], tail[6:]) and torch.equal(v[1, 0, 1:25], tail[6:])
    assert acc[1, 0, 1:25].tolist() == [float(x) for x in range(7, 31)] and not acc[1, 0, 25:].any()


# ---------------------------------------------------------------------------------------
# adapters
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,n,i,o,r,ranks,of,in_place", [
    (1, 1, 64, 32, 8, [8], [0], False), (1, 1, 2880, 4096, 16, None, [0], True),
    (5, 2, 96, 160, 16, [16, 5], [0, 1, -1, 1, 0], False), (17, 1, 256, 64, 24, [17], [0] * 17, False),
    (33, 3, 320, 320, 40, [40, 0, 1], [t % 4 - 1 for t in range(33)], True),
    (64, 24, 4096, 2880, 64, [8 * (a % 9) for a in range(24)], [(t * 7) % 25 - 1 for t in range(64)], False),
    (130, 2, 2880, 512, 128, [128, 121], [t % 2 for t in range(130)], False),
    (512, 400, 64, 96, 8, None, [(t * 11) % 400 for t in range(512)], True),
    (512, 1, 128, 2880, 32, None, [0] * 512, False), (512, 4096, 32, 32, 8, None, [4095] * 512, False),
    (40, 3, 160, 96, 16, None, [-1] * 40, False)])
def test_lora_apply(T, n, i, o, r, ranks, of, in_place):
    rng = np.random.default_rng(T + n + i)
    ld_x, ld_y, ld_z = i + 16, o + 8, o + 24
    x = torch.full((T, ld_x), NAN, dtype=torch.bfloat16, device="cuda")
    y = torch.full((T, ld_y), NAN, dtype=torch.bfloat16, device="cuda")
    z = torch.full((T, ld_z), 7.0, dtype=torch.bfloat16, device="cuda")
    x[:, :i], y[:, :o] = bf16(rng, T, i), bf16(rng, T, o)
    a, b = bf16(rng, n, r, i, scale=i ** -0.5), bf16(rng, n, o, r, scale=r ** -0.5)
    rk = ranks or [r] * n
    for k in range(min(n, 30)):
        a[k, rk[k]:] = NAN                                     # what lies behind an adapter's rank
        b[k, :, rk[k]:] = NAN
    scale = rng.uniform(0.5, 2.0, n).astype(np.float32)
    st, rt = torch.from_numpy(scale).cuda(), ints(rk)
    p = sgp.make_lora(a, b, st if n != 2 else None, rt if ranks else None)
    ws = torch.zeros(64, dtype=torch.uint8, device="cuda")
    y_in, y_out = y[:, :o], (y[:, :o] if in_place else z[:, :o])
    want, err = S.lora(f64(x[:, :i]), f64(y[:, :o]), np.nan_to_num(f64(a)), np.nan_to_num(f64(b)),
                       scale.astype(np.float64) if n != 2 else np.ones(n), rk, of)
    sgp.sgp_lora_apply(p, ints(of), x[:, :i], y_in, y_out, T, ws)
    assert sgp.sgp_status_from_workspace(ws) == sgp.SGP_OK
    within("y", y_out, want, err)
    if in_place:
        assert torch.isnan(y[:, o:]).all()                     # between the rows: untouched
    else:
        assert (z[:, o:] == 7.0).all()


def test_lora_apply_reports_bad_indices_and_ranks():
    rng = np.random.default_rng(3)
    x, y, a, b = bf16(rng, 6, 64), bf16(rng, 6, 64), bf16(rng, 3, 8, 64), bf16(rng, 3, 64, 8)
    ranks, of = ints([8, 9, -1]), ints([0, 3, 1, 2, -5, 1 << 30])
    p = sgp.make_lora(a, b, None, ranks)
    out, ws = torch.empty_like(y), torch.zeros(64, dtype=torch.uint8, device="cuda")
    sgp.sgp_lora_apply(p, of, x, y, out, 6, ws)
    assert sgp.sgp_status_from_workspace(ws) == sgp.SGP_ERR_DEVICE_BOUNDS
    assert torch.equal(out[1:], y[1:])
    want, err = S.lora(f64(x), f64(y), f64(a), f64(b), [1.0], [8], [0] + [-1] * 5)
    within("y", out, want, err)


def test_lora_apply_infinities():
    """An infinite A x stays infinite, with the sign that B gives it."""
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 5], x[1, 5] = float("inf"), 1.0
    a = torch.zeros(1, 8, 64, dtype=torch.bfloat16, device="cuda")
    a[:, :, 5] = 2.0
    a[:, :, :5] = 1.0
    b = torch.ones(1, 96, 8, dtype=torch.bfloat16, device="cuda")
    b[:, 48:] = -1.0
    y = torch.ones(2, 96, dtype=torch.bfloat16, device="cuda")
    x[0, 6:] = 0.0
    a[:, :, 6:] = 1.0
    ws = torch.zeros(64, dtype=torch.uint8, device="cuda")
    sgp.sgp_lora_apply(sgp.make_lora(a, b), ints([0, 0]), x, y, y, 2, ws)
    assert sgp.sgp_status_from_workspace(ws) == sgp.SGP_OK
    assert (y[0, :48] == float("inf")).all() and (y[0, 48:] == float("-inf")).all()
    assert (y[1, :48] == 17.0).all() and (y[1, 48:] == -15.0).all()


def test_lora_and_eviction_and_weights_captured():
    """One graph with all three, replayed on new inputs, beside a second graph on another stream."""
    def make(seed):
        rng = np.random.default_rng(seed)
        st = dict(x=bf16(rng, 20, 128), y=bf16(rng, 20, 1024), a=bf16(rng, 3, 16, 128, scale=0.1),
                  b=bf16(rng, 3, 1024, 16, scale=0.2), of=ints([t % 4 - 1 for t in range(20)]),
                  k=bf16(rng, 20, 2, 90, D), lens=ints([90 - t for t in range(20)]),
                  lse=torch.full((20, 16), 5.0, device="cuda"), acc=torch.zeros(20, 2, 90, device="cuda"),
                  q=torch.empty(20, 1024, dtype=torch.bfloat16, device="cuda"),
                  ko=torch.zeros(20, 2, 50, D, dtype=torch.bfloat16, device="cuda"),
                  ao=torch.zeros(20, 2, 50, device="cuda"), n_out=ints([0] * 20))
        st["v"], st["vo"] = st["k"].clone(), st["ko"].clone()
        st["dims"] = sgp.make_heads(16, 2)
        st["ws"] = torch.zeros(sgp.sgp_kv_evict_workspace_bytes(st["dims"], 20, 48), dtype=torch.uint8,
                               device="cuda")
        return st

    def run(st):
        sgp.sgp_lora_apply(sgp.make_lora(st["a"], st["b"]), st["of"], st["x"], st["y"], st["q"], 20, st["ws"])
        c = sgp.make_cache(st["k"], st["v"])
        sgp.sgp_attention_weights(st["dims"], c, st["lens"], st["q"], st["lse"], st["acc"], 20, st["ws"])
        sgp.sgp_kv_evict(st["dims"], c, sgp.make_cache(st["ko"], st["vo"]), sgp.make_evict(48, 2, 8),
                         st["lens"], st["n_out"], st["acc"], st["ao"], None, 20, st["ws"])
    outs = ("q", "acc", "ko", "vo", "ao", "n_out")
    a, b, eager = make(1), make(2), make(3)
    graphs = []
    for st in (a, b):
        run(st)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(st)
        graphs.append(g)
    for rep in range(2):
        fresh = [make(50 + 2 * rep + i) for i in range(2)]
        for st, f in zip((a, b), fresh):
            for key in ("x", "y", "a", "b", "k", "v", "acc", "ko", "vo", "ao"):
                st[key].copy_(f[key])
        torch.cuda.synchronize()
        for g, s in zip(graphs, (torch.cuda.Stream(), torch.cuda.Stream())):
            with torch.cuda.stream(s):
                g.replay()
        run(eager)
        torch.cuda.synchronize()
        for st, f in zip((a, b), fresh):
            run(f)
            torch.cuda.synchronize()
            assert sgp.sgp_status_from_workspace(st["ws"]) == sgp.SGP_OK
            for key in outs:
                assert torch.equal(st[key], f[key]), key


def test_binding_checks_on_the_gpu():
    x = Prefix(1, 2, 8, 1, [20], [3, 4], [0, 0])
    for kw in (dict(kv_len=x.kv_len.long()), dict(q=x.q.float()), dict(q=x.q[:1]), dict(q=x.q.cpu()),
               dict(lse=x.lse.double()), dict(o=torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda")[..., :64])):
        a = dict(kv_len=x.kv_len, q=x.q, o=x.o, lse=x.lse) | kw
        with pytest.raises(ValueError):
            sgp.sgp_prefix_attention(x.dims, x.cache, x.prefix, a["kv_len"], a["q"], a["o"], a["lse"], 2, x.ws)
    wide = sgp.make_heads(8, 2)                              # more KV heads than the caches have
    three = sgp.make_prefix(*x.prefix.tensors[:3], x.prefix.tensors[3][:1])
    one = sgp.make_cache(*(t[:1] for t in x.cache.tensors))
    for dims, cache, prefix in ((wide, x.cache, x.prefix), (x.dims, one, x.prefix), (x.dims, x.cache, three)):
        with pytest.raises(ValueError):
            sgp.sgp_prefix_attention(dims, cache, prefix, x.kv_len, x.q, x.o, x.lse, 2, x.ws)
    acc = torch.zeros(2, 1, x.cache.kv_cap, device="cuda")
    with pytest.raises(ValueError):
        sgp.sgp_attention_weights(x.dims, one, x.kv_len, x.q, x.lse, acc, 2, x.ws)
    for a, b in ((one, x.cache), (x.cache, one)):
        with pytest.raises(ValueError):
            sgp.sgp_kv_evict(x.dims, a, b, sgp.make_evict(2), x.kv_len, x.kv_len, acc, acc, None, 2, x.ws)
    with pytest.raises(sgp.SgpError) as e:
        sgp.sgp_prefix_attention(x.dims, x.cache, x.prefix, x.kv_len, x.q, x.o, x.lse, 2, x.ws[:256])
    assert e.value.code == sgp.SGP_ERR_INVALID_ARG


# ---------------------------------------------------------------------------------------
# the operators together, in a layer that runs op by op
# ---------------------------------------------------------------------------------------
def test_decode_layer_with_shared_prompt_adapters_and_eviction():
    """Two decode steps of one layer: QKV, adapters on the queries, attention over a shared prompt
    and the own caches (in the place of the layer's attention), its weights accumulated, output
    projection, adapters on the residual, router, experts; then the caches are cut to a budget.
    Every operator's result is checked on the inputs it had."""
    wl = synth.WORKLOADS["gptoss_layer"].with_(n_tokens=24, kv_len=700)
    inp = H.make_inputs(wl, 31)
    s, T = wl.shape, wl.n_tokens
    d = H.dims(s)
    rng = np.random.default_rng(8)
    k, v = (t.clone() for t in inp.caches[0])
    cap, nkv, nq = k.shape[2], s.n_kv_heads, s.n_q_heads
    own = [cap - 2 - (t % 9) for t in range(T)]
    kv_len = ints(own)
    layer = sgp.make_layer(inp.weights[0], k, v, 0)
    pk, pv = bf16(rng, 1, nkv, 333, D, scale=0.02), bf16(rng, 1, nkv, 333, D, scale=0.02)
    plen, pof = ints([333]), ints([-1 if t % 6 == 5 else 0 for t in range(T)])
    prefix = sgp.make_prefix(pk, pv, plen, pof)
    of = ints([t % 4 - 1 for t in range(T)])
    qa, qb = bf16(rng, 3, 16, s.hidden, scale=0.02), bf16(rng, 3, s.q_width, 16, scale=0.05)
    oa, ob = bf16(rng, 3, 32, s.q_width, scale=0.02), bf16(rng, 3, s.hidden, 32, scale=0.05)
    on_q, on_o = sgp.make_lora(qa, qb), sgp.make_lora(oa, ob)
    ws = H.workspace(d, T, cap)
    view = sgp.layer_views(d, T, cap, ws)
    pws = torch.zeros(sgp.sgp_prefix_attention_workspace_bytes(d, T, cap, 1), dtype=torch.uint8, device="cuda")
    ews = torch.zeros(sgp.sgp_kv_evict_workspace_bytes(d, T, 512), dtype=torch.uint8, device="cuda")
    lse = torch.empty(T, nq, device="cuda")
    acc = torch.zeros(T, nkv, cap, device="cuda")
    x, out = inp.x.clone(), torch.empty_like(inp.x)
    op = lambda i: sgp.sgp_layer_op(d, layer, i, kv_len, x, out, T, ws)
    ones = [1.0] * 3
    for step in range(2):
        lens = [n + step for n in own]
        op(0), op(1)
        q0, a0 = view["q"].clone(), view["a"].clone()
        sgp.sgp_lora_apply(on_q, of, view["a"], view["q"], view["q"], T, pws)
        want, err = S.lora(f64(a0), f64(q0), f64(qa), f64(qb), ones, [16] * 3, of.tolist())
        within("q", view["q"], want, err)
        sgp.sgp_prefix_attention(d, layer, prefix, kv_len, view["q"].view(T, nq, D),
                                 view["o"].view(T, nq, D), lse, T, pws)
        o, z, eo, ez = S.prefix_attention(f64(view["q"]).reshape(T, nq, D), f64(k), f64(v), lens, f64(pk),
                                          f64(pv), [333], pof.tolist(), 0)
        within("o", view["o"], o.reshape(T, -1), eo.reshape(T, -1))
        within("lse", lse, z, ez)
        before = f64(acc)
        sgp.sgp_attention_weights(d, layer, kv_len, view["q"].view(T, nq, D), lse, acc, T, pws)
        add, ea = S.attention_weights(f64(view["q"]).reshape(T, nq, D), f64(k), lens, f64(lse))
        within("acc", acc, before + add, ea + S.U32 * np.abs(before + add))
        op(3)
        h0, o0 = view["h"].clone(), view["o"].clone()
        sgp.sgp_lora_apply(on_o, of, view["o"], view["h"], view["h"], T, pws)
        want, err = S.lora(f64(o0), f64(h0), f64(oa), f64(ob), ones, [32] * 3, of.tolist())
        within("h", view["h"], want, err)
        for i in range(4, 9):
            op(i)
        H.assert_close("u", view["u"], O.rmsnorm(f64(view["h"]), f64(inp.weights[0]["g_mlp"]), s.rms_eps))
        assert torch.isfinite(out).all()
        x.copy_(out)
        if step == 0:
            kv_len += 1
    assert sgp.sgp_status_from_workspace(ws) == sgp.SGP_OK
    assert sgp.sgp_status_from_workspace(pws) == sgp.SGP_OK
    a0, k0, v0, lens = acc.cpu().numpy(), k.clone(), v.clone(), kv_len.tolist()
    sgp.sgp_kv_evict(d, layer, layer, sgp.make_evict(512, 4, 64), kv_len, kv_len, acc, acc, None, T, ews)
    assert sgp.sgp_status_from_workspace(ews) == sgp.SGP_OK
    assert kv_len.tolist() == [512] * T
    for t in range(T):
        for j in range(nkv):
            keep = torch.from_numpy(S.evict(a0[t, j], lens[t], 512, 4, 64)).cuda()
            assert torch.equal(k[t, j, :512], k0[t, j, keep]) and torch.equal(v[t, j, :512], v0[t, j, keep])
            assert np.array_equal(f64(acc[t, j, :512]), a0[t, j, keep.cpu().numpy()].astype(np.float64))
            assert not acc[t, j, 512:].any()
    # the next step appends behind the kept rows and attends to them
    kv_len += 1
    op(0), op(1)
    sgp.sgp_prefix_attention(d, layer, prefix, kv_len, view["q"].view(T, nq, D), view["o"].view(T, nq, D), lse,
                             T, pws)
    o, z, eo, ez = S.prefix_attention(f64(view["q"]).reshape(T, nq, D), f64(k), f64(v), [513] * T, f64(pk),
                                      f64(pv), [333], pof.tolist(), 0)
    within("o", view["o"], o.reshape(T, -1), eo.reshape(T, -1))
    assert sgp.sgp_status_from_workspace(pws) == sgp.SGP_OK
