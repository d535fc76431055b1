// Decode attention over prefixes that sequences of a batch share, and the merge with the
// attention over each sequence's own cache.
//
//   s_p = q_h . k_p / sqrt(d) over the prefix's positions, then the own ones;
//   o   = sum_p softmax(s)_p v_p,   lse = log sum_p exp(s_p).
// Softmax splits over any cut of the positions: with m = max s, l = sum exp(s - m) and
// a = sum exp(s - m) v of each part, the whole has M = max m, L = sum l exp(m - M) and
// o = sum a exp(m - M) / L.  Three kernels: the own caches (attn_decode_kernel, partials only),
// the prefixes (here), the merge (here).
//
// A prefix is read once for all query rows of its group (sequences x heads of one KV head),
// so the prefix part is a matrix product, not a stream: 4 d flops for every (row, position)
// against 256 bytes for every position.
#include <climits>

#include "kernels.h"
#include "mma.cuh"

namespace sgp {

namespace {

constexpr int kPThreads = 384;
constexpr int kPHalf = kPrefixKeys * 128;     // K (or V) bytes of a step

// The groups of the batch, built by every CTA in shared memory.
struct Plan {
    int mem[kPrefixMax];         // sequences by group, in sequence order
    int of[kPrefixMax];          // group of a sequence or -1
    int rank[kPrefixMax];        // its place in the group
    int base[kPrefixMax + 1];    // first entry of a group in mem
    int tile0[kPrefixMax + 1];   // first tile of a group
    int step0[kPrefixMax + 1];   // first step of a group
    int tiles[kPrefixMax];       // tiles per KV head
    int steps[kPrefixMax];       // steps per tile
    int first[kPrefixMax];       // first step's place in the prefix (in steps)
    int len[kPrefixMax];
    int low[kPrefixMax];         // least position that some sequence of the group sees
};

// exclusive prefix sums over n <= kPrefixMax values of three arrays by one warp; x[n] = total
__device__ __forceinline__ void scan3(int* a, int* b, int* c, int n, int lane) {
    int ra = 0, rb = 0, rc = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const int va = i < n ? a[i] : 0, vb = i < n ? b[i] : 0, vc = i < n ? c[i] : 0;
        int sa = va, sb = vb, sc = vc;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int ta = __shfl_up_sync(0xffffffffu, sa, o), tb = __shfl_up_sync(0xffffffffu, sb, o),
                      tc = __shfl_up_sync(0xffffffffu, sc, o);
            if (lane >= o) {
                sa += ta;
                sb += tb;
                sc += tc;
            }
        }
        if (i < n) {
            a[i] = ra + sa - va;
            b[i] = rb + sb - vb;
            c[i] = rc + sc - vc;
        }
        ra += __shfl_sync(0xffffffffu, sa, 31);
        rb += __shfl_sync(0xffffffffu, sb, 31);
        rc += __shfl_sync(0xffffffffu, sc, 31);
    }
    if (lane == 0) {
        a[n] = ra;
        b[n] = rb;
        c[n] = rc;
    }
}

__device__ void build_plan(Plan& pl, const PrefixProblem& P, const KCtx& ctx) {
    const int tid = threadIdx.x, lane = tid & 31, n = P.prefix.n;
    for (int g = tid; g < n; g += blockDim.x) {
        int len = P.prefix.len[g];
        if (len < 0 || len > P.prefix.cap) {
            if (blockIdx.x == 0) report(ctx, ST_BOUNDS, (uint32_t)len);
            len = 0;
        }
        pl.len[g] = len;
        pl.low[g] = INT_MAX;
        pl.base[g] = 0;  // members, until the scan
    }
    for (int t = tid; t < P.T; t += blockDim.x) {
        const int g = P.prefix.of[t];
        if (g >= n && blockIdx.x == 0) report(ctx, ST_BOUNDS, (uint32_t)g);
        pl.of[t] = g >= 0 && g < n ? g : -1;
    }
    __syncthreads();
    // place of every sequence in its group: 32 sequences a round, counts kept per group
    if (tid < 32) {
        for (int t0 = 0; t0 < P.T; t0 += 32) {
            const int t = t0 + lane;
            const int g = t < P.T ? pl.of[t] : -1;
            const unsigned same = __match_any_sync(0xffffffffu, g);
            const int before = __popc(same & ((1u << lane) - 1u));
            const int had = g >= 0 ? pl.base[g] : 0;
            __syncwarp();
            if (g >= 0) {
                pl.rank[t] = had + before;
                if (before == 0) pl.base[g] = had + __popc(same);
            }
            __syncwarp();
        }
    }
    if (P.window > 0)
        for (int t = tid; t < P.T; t += blockDim.x) {
            const int g = pl.of[t];
            if (g < 0) continue;
            const int own = P.kv_len[t];
            const int at = pl.len[g] + (own >= 0 && own <= P.kv_cap ? own : 0) - P.window;
            atomicMin(&pl.low[g], max(0, at));
        }
    __syncthreads();
    for (int g = tid; g < n; g += blockDim.x) {
        const int low = P.window > 0 ? pl.low[g] : 0;
        const int members = pl.base[g], len = pl.len[g];
        const int first = low / kPrefixKeys;
        const bool some = members > 0 && low < len;
        pl.low[g] = low;
        pl.first[g] = first;
        pl.tiles[g] = some ? (members + P.tile_seqs - 1) / P.tile_seqs : 0;
        pl.steps[g] = some ? (len + kPrefixKeys - 1) / kPrefixKeys - first : 0;
        pl.tile0[g] = pl.tiles[g] * P.nkv;
        pl.step0[g] = pl.tile0[g] * pl.steps[g];
    }
    __syncthreads();
    if (tid < 32) scan3(pl.base, pl.tile0, pl.step0, n, lane);
    __syncthreads();
    for (int t = tid; t < P.T; t += blockDim.x) {
        const int g = pl.of[t];
        if (g >= 0) pl.mem[pl.base[g] + pl.rank[t]] = t;
        if (blockIdx.x == 0) {
            PrefixSeq s = {0, 0, 0, 0, 0, pl.step0[n], {0, 0}};
            if (g >= 0) s = {pl.tile0[g], pl.tiles[g], pl.step0[g], pl.steps[g], pl.rank[t], pl.step0[n], {0, 0}};
            P.seq[t] = s;
        }
    }
    __syncthreads();
}

// Step x of the call: group, KV head, tile of that pair, step within the tile.
struct Step {
    int g, kvh, tile, k;
};
__device__ __forceinline__ Step step_at(const Plan& pl, int n, int x) {
    int lo = 0, hi = n;  // the last group that begins at or before x (empty ones begin with it)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pl.step0[mid] <= x) lo = mid;
        else hi = mid;
    }
    const int r = x - pl.step0[lo], i = r / pl.steps[lo];
    return {lo, i / pl.tiles[lo], i % pl.tiles[lo], r % pl.steps[lo]};
}

// Warp 0 loads keys and values (TMA, a ring of steps), warps 4-7 and 8-11 are two softmax groups
// of 128 rows each, and warps 1 and 2 issue one group's matrix products each.  A step's positions
// are taken in halves of 64.  Per half and group
//     S = Q K^T   (M = 128 rows, N = 64 positions, K = 64), accumulators in tensor memory;
//     P = exp2(scale S - m) by the group's threads, one row each, back to tensor memory as bf16;
//     O += P V    (M = 128, N = 64 dims, K = 64), P read from tensor memory.
// S and P have two buffers each, and a half takes one signal either way: the softmax's "P(i) is
// written" also frees S(i), and the products' "S(i + 2) is complete" also says that O holds P(i)
// (it was issued behind it).  What a wait costs, 100 to 250 cycles although it passes at once, is
// what a half has to be long against.
// The weights are taken against a maximum m that is only raised when a row's scores pass it by
// more than 2^8 (weights up to 256 lose nothing in bf16 or fp32); the half's own maximum is found
// beside the exponentials, and in the rare case that it does, O and the sum are rescaled and the
// half is done again.  m begins at 0, when the first scores are near it.
constexpr int kPStages = 5;
constexpr int kPSub = 64;           // positions of a half
constexpr float kPRaise = 8.f;
constexpr uint32_t kTmemS = 0, kTmemP = 256, kTmemO = 384;  // columns; per group 2 x 64, 2 x 32, 64

struct PrefixBars {
    uint64_t kv_full[kPStages], kv_empty[kPStages];
    uint64_t q_full[2];        // the group's query rows are in shared memory
    uint64_t s_full[2][2];     // [group][buffer]; the group's half i uses buffer i & 1
    uint64_t p_full[2][2];
    uint64_t pv_done[2];       // phase i: O holds half i (a rescale and a tile's end wait for it)
    uint32_t tmem;
    int err;
};

// The part of a tile that a share holds: steps [s.k, s.k + steps), halves of them that hold
// positions of the prefix.
__device__ __forceinline__ int halves_of(const Plan& pl, const Step& s, int steps) {
    const int p0 = (pl.first[s.g] + s.k) * kPrefixKeys;
    return (min(pl.len[s.g] - p0, steps * kPrefixKeys) + kPSub - 1) / kPSub;
}

__global__ void __launch_bounds__(kPThreads, 1)
    prefix_attn_kernel(const __grid_constant__ PrefixProblem P, const KCtx ctx) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* qs = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));  // [2][128 rows]
    uint8_t* ring = qs + 2 * 128 * 128;
    PrefixBars& bar = *reinterpret_cast<PrefixBars*>(ring + kPStages * 2 * kPHalf);
    Plan& pl = *reinterpret_cast<Plan*>(&bar + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_launch();
    if (tid == 0) {
        for (int s = 0; s < kPStages; ++s) {
            mbar_init(&bar.kv_full[s], 1);
            mbar_init(&bar.kv_empty[s], 2);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(&bar.q_full[h], 4);
            mbar_init(&bar.pv_done[h], 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(&bar.s_full[h][i], 1);
                mbar_init(&bar.p_full[h][i], 4);
            }
        }
        bar.err = 0;
        fence_barrier_init();
        prefetch_tensormap(&P.tmK);
        prefetch_tensormap(&P.tmV);
    }
    if (warp == 1) {
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    task_begin(ctx);
    build_plan(pl, P, ctx);  // ends with a barrier
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    const int n = P.prefix.n, total = pl.step0[n];
    const int shares = min(kPrefixShares, total);  // none of them empty
    const int b = blockIdx.x;
    const int x0 = b < shares ? (int)((long long)b * total / shares) : 0;
    const int x1 = b < shares ? (int)((long long)(b + 1) * total / shares) : 0;
    volatile int* err = &bar.err;
    auto gave_up = [&](uint32_t where) {
        report(ctx, ST_TIMEOUT, where);
        *err = 1;
    };

    if (warp == 0) {
        if (elect_one()) {
            const uint64_t pol = policy_evict_last();  // the other row tiles read it too
            uint32_t it = 0;
            for (int x = x0; x < x1 && !*err; ++it, ++x) {
                const uint32_t st = it % kPStages, use = it / kPStages;
                if (use > 0 && !mbar_wait_near(&bar.kv_empty[st], (use - 1) & 1u, ctx.timeout_ns)) {
                    gave_up(20);
                    break;
                }
                const Step s = step_at(pl, n, x);
                const int row = (s.g * P.nkv + s.kvh) * P.prefix.cap + (pl.first[s.g] + s.k) * kPrefixKeys;
                uint8_t* dst = ring + st * 2 * kPHalf;
                mbar_arrive_expect_tx(&bar.kv_full[st], 2 * kPHalf);
                tma_load_2d(dst, &P.tmK, &bar.kv_full[st], 0, row, pol);
                tma_load_2d(dst + kPHalf, &P.tmV, &bar.kv_full[st], 0, row, pol);
            }
            if (*err)  // loads in flight into this CTA's shared memory (bounded)
                for (uint32_t i = it > kPStages ? it - kPStages : 0; i < it; ++i)
                    (void)mbar_wait_near(&bar.kv_full[i % kPStages], (i / kPStages) & 1u, 10000000ull);
        }
        __syncwarp();
    } else if (warp <= 2) {
        if (elect_one()) {
            const int h = warp - 1;
            constexpr uint32_t id_s = idesc_bf16_f32(128, kPSub), id_o = idesc_bf16_f32(128, 64) | kIdescBmn;
            // descriptors advance by address / 16: 32 bytes to the next 16 dims, 16 rows of V
            const uint64_t dq = smem_desc_sw128(smem_u32(qs + h * 128 * 128));
            const uint64_t dk0 = smem_desc_sw128(smem_u32(ring)), dv0 = dk0 + kPHalf / 16;
            constexpr int kStageD = 2 * kPHalf / 16, kHalfD = kPSub * 128 / 16;
            const uint32_t ts = tmem + kTmemS + 128 * h, to = tmem + kTmemO + 64 * h, tp = tmem + kTmemP + 64 * h;
            uint32_t n_q = 0, n = 0;               // tiles of this group, halves whose S is issued
            uint32_t st_s = 0, ph_s = 0, st_p = 0;  // stages of the next S and the next product
            bool ok = true;
            auto scores = [&](int j) {  // S = Q K^T of the tile's half j
                if ((j & 1) == 0 && !(ok = mbar_wait_near(&bar.kv_full[st_s], ph_s, ctx.timeout_ns))) {
                    gave_up(22);
                    return;
                }
                const uint64_t dk = dk0 + st_s * kStageD + (j & 1) * kHalfD;
#pragma unroll
                for (int k = 0; k < 4; ++k) tc_mma_bf16(ts + 64 * (n & 1u), dq + 2 * k, dk + 2 * k, id_s, k > 0);
                tc_commit(&bar.s_full[h][n & 1u]);
                ++n;
                if ((j & 1) && ++st_s == kPStages) st_s = 0, ph_s ^= 1;
            };
            for (int x = x0; x < x1 && ok;) {
                const Step s = step_at(pl, P.prefix.n, x);
                const int steps = min(x1 - x, pl.steps[s.g] - s.k), halves = halves_of(pl, s, steps);
                const int rows = min(P.tile_seqs, pl.base[s.g + 1] - pl.base[s.g] - s.tile * P.tile_seqs) * P.G;
                x += steps;
                if (rows <= 128 * h) {  // no rows here: the stages are free for this group's part
                    for (int i = 0; i < steps && ok; ++i) {
                        if (!(ok = mbar_wait_near(&bar.kv_full[st_s], ph_s, ctx.timeout_ns))) gave_up(31);
                        mbar_arrive(&bar.kv_empty[st_s]);
                        if (++st_s == kPStages) st_s = 0, ph_s ^= 1;
                    }
                    st_p = st_s;
                    continue;
                }
                if (!(ok = mbar_wait_near(&bar.q_full[h], n_q++ & 1u, ctx.timeout_ns))) {
                    gave_up(23);
                    break;
                }
                tc_fence_after();
                const uint32_t n0 = n;  // number of the tile's first half
                scores(0);
                if (ok && halves > 1) scores(1);
                for (int j = 0; j < halves && ok; ++j) {
                    const uint32_t i = n0 + j, buf = i & 1u;
                    if (!(ok = mbar_wait_near(&bar.p_full[h][buf], (i >> 1) & 1u, ctx.timeout_ns))) {
                        gave_up(21);
                        break;
                    }
                    tc_fence_after();
                    const uint64_t dv = dv0 + st_p * kStageD + (j & 1) * kHalfD;
#pragma unroll
                    for (int k = 0; k < kPSub / 16; ++k)  // O += P V
                        tc_mma_bf16_ta(to, tp + 32 * buf + 8 * k, dv + k * (16 * 128 / 16), id_o, !(j == 0 && k == 0));
                    tc_commit(&bar.pv_done[h]);
                    if ((j & 1) || j + 1 == halves) {
                        tc_commit(&bar.kv_empty[st_p]);
                        if (++st_p == kPStages) st_p = 0;
                    }
                    if (j + 2 < halves) scores(j + 2);
                }
                if (halves & 1) {  // the last stage's second half holds no positions
                    if (++st_s == kPStages) st_s = 0, ph_s ^= 1;
                }
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int h = (warp - 4) >> 2, quad = warp & 3;  // a warp reads its quadrant's TMEM lanes
        const int r = h * 128 + quad * 32 + lane;        // this thread's row of the tile
        const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t ts = tl + kTmemS + 128 * h, to = tl + kTmemO + 64 * h, tp = tl + kTmemP + 64 * h;
        const int row_of = (65536 + P.G - 1) / P.G;      // r / G = r * row_of >> 16 for r < 256
        const float2 sc2 = make_float2(P.scale_log2, P.scale_log2);
        uint32_t it = 0;  // halves of this group
        bool ok = true;
        // every wait's outcome is the warp's: its tensor-memory accesses are warp-wide
        auto wait = [&](uint64_t* bar_, uint32_t parity, uint32_t where) {
            if (__all_sync(0xffffffffu, mbar_wait_near(bar_, parity, ctx.timeout_ns))) return true;
            if (lane == 0) gave_up(where);
            return false;
        };
        for (int x = x0; x < x1 && ok;) {
            const Step s = step_at(pl, n, x);
            const int steps = min(x1 - x, pl.steps[s.g] - s.k), halves = halves_of(pl, s, steps);
            const int seq0 = pl.base[s.g] + s.tile * P.tile_seqs;
            const int rows = min(P.tile_seqs, pl.base[s.g + 1] - seq0) * P.G;
            const int i0 = x - x0;  // first step's place in the share
            x += steps;
            if (rows <= 128 * h) continue;
            const int len = pl.len[s.g], seen = pl.low[s.g];
            // this warp's 32 query rows, 8 lanes to a row, into the swizzled tile (zeros past the
            // tile's rows: rows do not mix, and theirs are not stored)
            {
                uint8_t* dst = qs + h * 128 * 128;
                uint4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = h * 128 + quad * 32 + i * 4 + (lane >> 3), q = row * row_of >> 16;
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (row < rows) {
                        const bf16* src = P.q + (size_t)pl.mem[seq0 + q] * P.nq * 64 +
                                          (size_t)(s.kvh * P.G + row - q * P.G) * 64;
                        v[i] = reinterpret_cast<const uint4*>(src)[lane & 7];
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4*>(dst + sw128(quad * 32 + i * 4 + (lane >> 3), lane & 7)) = v[i];
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.q_full[h]);
            }
            int low = 0;
            if (P.window > 0 && r < rows) {
                const int own = P.kv_len[pl.mem[seq0 + (r * row_of >> 16)]];
                low = max(0, len + (own >= 0 && own <= P.kv_cap ? own : 0) - P.window);
            }
            const bool live = h * 128 + quad * 32 < rows;  // some row of this warp counts
            float m = 0.f;  // what the weights are taken against (scaled scores, base 2)
            float2 l2 = make_float2(0.f, 0.f);
            int pos0 = (pl.first[s.g] + s.k) * kPrefixKeys;
            for (int j = 0; j < halves; ++j, ++it, pos0 += kPSub) {
                const uint32_t buf = it & 1u;
                if (!(ok = wait(&bar.s_full[h][buf], (it >> 1) & 1u, 24))) break;
                tc_fence_after();
                if (pos0 + kPSub > len || pos0 < seen) {
                    // what lies behind the prefix, or before what any sequence of the group sees,
                    // is arbitrary and its weight is 0: clear V there (each group of warps for its
                    // own product; the other's writes are the same zeros)
                    const uint32_t i = i0 + (j >> 1), st = i % kPStages;
                    if (!(ok = wait(&bar.kv_full[st], (i / kPStages) & 1u, 27))) break;
                    uint4* v4 = reinterpret_cast<uint4*>(ring + st * 2 * kPHalf + kPHalf + (j & 1) * kPSub * 128);
                    for (int e = quad * 32 + lane; e < kPSub * 8; e += 128)
                        if (pos0 + (e >> 3) >= len || pos0 + (e >> 3) < seen) v4[e] = make_uint4(0, 0, 0, 0);
                    fence_proxy_async();
                }
                if (live) {
                    if (pos0 + kPSub > len || __any_sync(0xffffffffu, pos0 < low)) {
                        // hide positions in tensor memory (rare: a loop keeps the code small)
#pragma unroll 1
                        for (int c = 0; c < kPSub; c += 16) {
                            float v[16];
                            uint32_t w[16];
                            tmem_ld_wait_x16(ts + 64 * buf + c, v);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const int at = pos0 + c + e;
                                w[e] = __float_as_uint(at >= len || at < low ? -INFINITY : v[e]);
                            }
                            tmem_st_x16(ts + 64 * buf + c, w);
                        }
                        tmem_st_wait();
                    }
                    const float2 l_old = l2;
                    while (true) {
                        // a row that has seen nothing yet: every score is -inf, every weight 0
                        const float sub = m == -INFINITY ? 0.f : -m;
                        const float2 sub2 = make_float2(sub, sub);
                        float sr[64], mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        tmem_ld_wait_x64(ts + 64 * buf, sr);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float2 v = make_float2(sr[32 * c + 2 * e], sr[32 * c + 2 * e + 1]);
                                mx[e & 1] = fmaxf(mx[e & 1], v.x);
                                mx[2 + (e & 1)] = fmaxf(mx[2 + (e & 1)], v.y);
                                v = fma2(v, sc2, sub2);
                                v.x = ex2(v.x);
                                v.y = ex2(v.y);
                                l2 = add2(l2, v);
                                // the weight's rounding to bf16, the second product's operand type
                                w[e] = pack_bf16x2(v.x, v.y);
                            }
                            tmem_st_x16(tp + 32 * buf + 16 * c, w);
                        }
                        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * P.scale_log2;
                        // the first half also raises from below: its scores may be far under 0
                        const bool far = top > m + kPRaise || (j == 0 && m == 0.f && top < -kPRaise);
                        if (!__any_sync(0xffffffffu, far)) break;
                        const float nm = j == 0 ? top : fmaxf(m, top);
                        const float c = j == 0 || m == -INFINITY ? 0.f : ex2(m - nm);
                        m = nm;
                        l2 = make_float2(l_old.x * c, l_old.y * c);
                        if (j == 0) continue;
                        if (!(ok = wait(&bar.pv_done[h], (it - 1) & 1u, 25))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < 64; q += 16) {
                            float o[16];
                            uint32_t w[16];
                            tmem_ld_wait_x16(to + q, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * c);
                            tmem_st_x16(to + q, w);
                        }
                    }
                    if (!ok) break;
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[h][buf]);
            }
            if (!ok) break;
            // the last product, then this row's partial
            if (!wait(&bar.pv_done[h], (it - 1) & 1u, 26)) break;
            tc_fence_after();
            if (live) {
                const size_t slot = b + (size_t)(pl.tile0[s.g] + s.kvh * pl.tiles[s.g] + s.tile);
                const size_t at = slot * kPrefixRows + r;
                float o[64];
                tmem_ld_wait_x64(to, o);
                if (r < rows) {
                    float4* dst = reinterpret_cast<float4*>(P.part_acc + at * 64);
#pragma unroll
                    for (int j = 0; j < 16; ++j) dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    *reinterpret_cast<float2*>(P.part_ml + at * 2) = make_float2(m, l2.x + l2.y);
                }
            }
            tc_fence_before();
        }
    }
    // the merge waits for this kernel: the own caches' kernel before it must be complete too
    griddep_wait();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
    task_end(ctx);
}

// One warp per (sequence, KV head): lane l holds dims 2l, 2l + 1 of every query head.  The
// partials join in a fixed order: the prefix's shares, then the own chunks.
template <int GP>
__global__ void __launch_bounds__(128) prefix_merge_kernel(const PrefixMergeProblem P, const KCtx ctx) {
    griddep_wait();
    task_begin(ctx);
    const int lane = threadIdx.x & 31;
    const int pair = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (pair < P.T * P.nkv) {
        const int t = pair / P.nkv, kvh = pair % P.nkv;
        // the prefix's shares [s0, s1] and this sequence's rows in their slots
        int s0 = 0, s1 = -1;
        size_t row0 = 0;
        if (P.seq != nullptr) {
            const PrefixSeq q = P.seq[t];
            if (q.tiles > 0) {
                const int tile = kvh * q.tiles + q.i / P.tile_seqs;
                const int x = q.step + tile * q.steps;
                // share s holds the steps [s total / shares, (s + 1) total / shares)
                const long long shares = min(kPrefixShares, q.total);
                s0 = (int)(((x + 1) * shares - 1) / q.total);
                s1 = (int)(((x + q.steps) * shares - 1) / q.total);
                row0 = (size_t)(q.tile + tile) * kPrefixRows + (size_t)(q.i % P.tile_seqs) * P.G;
            }
        }
        int L = P.kv_len[t];
        if (L < 0 || L > P.kv_cap) L = 0;
        const int first = P.window > 0 ? max(0, L - P.window) : 0;
        const int S = (L - first + P.chunk - 1) / P.chunk;
        const float* oml = P.own_ml + (size_t)pair * P.S_max * 32;
        const float* oacc = P.own_acc + (size_t)pair * P.S_max * 64 * 16;
        // lane h: head h's maximum over all parts
        const bool has = lane < P.G;
        float M = -INFINITY;
        for (int s = s0; s <= s1; ++s)
            if (has) M = fmaxf(M, __ldcg(P.pre_ml + ((size_t)s * kPrefixRows + row0 + lane) * 2));
        for (int c = 0; c < S; ++c)
            if (has) M = fmaxf(M, __ldcg(oml + c * 32 + 2 * lane));
        const float sub = M == -INFINITY ? 0.f : M;
        float a[GP][2], Ls = 0.f;
#pragma unroll
        for (int h = 0; h < GP; ++h) a[h][0] = a[h][1] = 0.f;
        for (int s = s0; s <= s1; ++s) {
            const size_t r = (size_t)s * kPrefixRows + row0;
            float w = 0.f;
            if (has) {
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(P.pre_ml + (r + lane) * 2));
                w = exp2f(ml.x - sub);
                Ls = fmaf(w, ml.y, Ls);
            }
#pragma unroll
            for (int h = 0; h < GP; ++h) {
                const float wh = __shfl_sync(0xffffffffu, w, h);
                if (h < P.G) {
                    const float2 v = __ldcg(reinterpret_cast<const float2*>(P.pre_acc + (r + h) * 64 + 2 * lane));
                    a[h][0] = fmaf(wh, v.x, a[h][0]);
                    a[h][1] = fmaf(wh, v.y, a[h][1]);
                }
            }
        }
        for (int c = 0; c < S; ++c) {
            float w = 0.f;
            if (has) {
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(oml + c * 32 + 2 * lane));
                w = exp2f(ml.x - sub);
                Ls = fmaf(w, ml.y, Ls);
            }
#pragma unroll
            for (int h4 = 0; h4 < GP; h4 += 4) {
                const float4 v0 = __ldcg(reinterpret_cast<const float4*>(oacc + ((size_t)c * 64 + 2 * lane) * 16 + h4));
                const float4 v1 = __ldcg(reinterpret_cast<const float4*>(oacc + ((size_t)c * 64 + 2 * lane + 1) * 16 + h4));
                const float e0[4] = {v0.x, v0.y, v0.z, v0.w}, e1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float wh = __shfl_sync(0xffffffffu, w, h4 + q);
                    if (h4 + q < P.G) {
                        a[h4 + q][0] = fmaf(wh, e0[q], a[h4 + q][0]);
                        a[h4 + q][1] = fmaf(wh, e1[q], a[h4 + q][1]);
                    }
                }
            }
        }
        // a row that sees nothing: o = 0, lse = -inf
        const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
        bf16* o = P.o + (size_t)t * P.nq * 64 + (size_t)kvh * P.G * 64;
#pragma unroll
        for (int h = 0; h < GP; ++h) {
            const float ih = __shfl_sync(0xffffffffu, inv, h);
            if (h < P.G)
                *reinterpret_cast<uint32_t*>(o + h * 64 + 2 * lane) = pack_bf16x2(a[h][0] * ih, a[h][1] * ih);
        }
        if (P.lse != nullptr && has)
            P.lse[(size_t)t * P.nq + kvh * P.G + lane] =
                Ls == 0.f ? -INFINITY : (M + log2f(Ls)) * 0.6931471805599453f;
    }
    task_end(ctx);
}

}  // namespace

int enqueue_prefix(Launcher& L, const PrefixProblem& p, const KCtx& c) {
    const size_t smem = 1024 + 2 * 128 * 128 + kPStages * 2 * kPHalf + sizeof(PrefixBars) + sizeof(Plan);
    void* args[] = {(void*)&p, (void*)&c};
    return L.launch((const void*)prefix_attn_kernel, dim3(kPrefixShares), dim3(kPThreads), smem, args,
                    true);
}

int enqueue_prefix_merge(Launcher& L, const PrefixMergeProblem& p, const KCtx& c) {
    void* args[] = {(void*)&p, (void*)&c};
    const void* f = p.G <= 8 ? (const void*)prefix_merge_kernel<8> : (const void*)prefix_merge_kernel<16>;
    return L.launch(f, dim3((p.T * p.nkv + 3) / 4), dim3(128), 0, args, true);
}

}  // namespace sgp
