// Decode attention over prefixes that sequences of a batch share, and the merge with the
// attention over each sequence's own cache.
//
//   s_p = q_h . k_p / sqrt(d) over the prefix's positions, then the own ones;
//   o   = sum_p softmax(s)_p v_p,   lse = log sum_p exp(s_p).
// Softmax splits over any cut of the positions: with m = max s, l = sum exp(s - m) and
// a = sum exp(s - m) v of each part, the whole has M = max m, L = sum l exp(m - M) and
// o = sum a exp(m - M) / L.
//
// Two kernels.  In the first, some CTAs take the prefixes and the others the own caches, and every
// part leaves its (m, l, a); the second merges them.  A prefix is read once for all query rows of
// its group (sequences x heads of one KV head), so the prefix part is a matrix product on tcgen05,
// 4 d flops for every (row, position) against 256 bytes for every position; the own part is a
// stream of the caches through warp-level products, bound by HBM.  Side by side, each has what
// the other leaves idle.
//
// Measured (replayed): 64 sequences x 64 / 8 heads on a prefix of 8192 beside own caches of up to
// 1024, 76 MB and 9.1 GFLOP, 27.6 us (2.8 TB/s); 512 sequences x 8 / 1 heads on 32,768, 34.6 GFLOP,
// 53 us (650 TFLOP/s); two sequences on 500 positions 11 us.  Of these about 5.5 us pass before the
// first product (the plan of the groups 3.2, the query tile 2.4) and 5 us in the merge.
//
// Instructions that run once are met cold, about 300 cycles for eight of them, so what surrounds the
// loops is kept short: no unrolling, few divisions, one copy of what several warps need.
#include <climits>

#include "serving.cuh"

namespace sgp {

namespace {

constexpr int kPThreads = 384;
constexpr int kOwnWarps = kPThreads / 32;
constexpr int kOwnPos = 64;                  // positions of an own warp's stage
constexpr int kOwnHalf = kOwnPos * 128;      // K (or V) bytes of it
constexpr int kPHalf = kPrefixKeys * 128;     // K (or V) bytes of a step
// The prefixes' work is cut into equal shares by units, a step each and these for the beginning of a
// tile: what lies between two tiles (output, queries, first product: 2.7 us) is worth two steps.
constexpr int kTileUnits = 2;

// The groups of the batch, built by every CTA in shared memory.
struct Plan {
    int mem[kPrefixMax];         // sequences by group, in sequence order
    int of[kPrefixMax];          // group of a sequence or -1
    int rank[kPrefixMax];        // its place in the group
    int base[kPrefixMax + 1];    // first entry of a group in mem
    int tile0[kPrefixMax + 1];   // first tile of a group
    int step0[kPrefixMax + 1];   // first unit of a group
    int tiles[kPrefixMax];       // tiles per KV head
    int steps[kPrefixMax];       // steps per tile
    int first[kPrefixMax];       // first step's place in the prefix (in steps)
    int len[kPrefixMax];
    int low[kPrefixMax];         // least position that some sequence of the group sees
    int chunk0[kPrefixMax + 1];  // own chunks (all KV heads) before a sequence
    int own_first[kPrefixMax];   // first own position seen
    int own_len[kPrefixMax];
    int block_chunks[kPrefixMax / 32], block_pos[kPrefixMax / 32];  // of 32 sequences: own chunks, positions
    int n_own;                   // CTAs that take the own caches; the others take the prefixes:
    int shares, q, n_long;       // shares of q units, the first n_long of one more
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

// Chunks of n own positions.
__device__ __forceinline__ int chunks_of(int n, const PrefixProblem& P) {
    return (n + (1 << P.chunk_log2) - 1) >> P.chunk_log2;
}

// CTAs that take the own caches: what makes the slower part fastest, of the multiples of 5.  Measured
// from the launch on: own CTAs begin after 5.5 us, each of their warps takes 1.8 us for 64 positions
// of a chunk or fewer (416 x 8 caches of up to 4 positions: 130 us on 5 CTAs, 23 on 75), all
// together at most 5 TB/s; prefix CTAs take 1.37 us for a unit and 7.5 for all else.
__device__ __forceinline__ int own_ctas(long long own_pos, int chunks, int nkv, int units, int lane) {
    const int x = lane < 31 ? 5 * lane : kPrefixCtas, y = kPrefixCtas - x;
    const float pos = (float)own_pos * (float)nkv;
    const float rounds = ceilf(__fdividef((float)chunks, (float)(kOwnWarps * x)));
    const float warp = rounds * fmaxf(__fdividef(pos, (float)chunks), 64.f) * (1800.f / 64.f);
    const float own = x > 0 ? 5500.f + fmaxf(pos * (256.f / 5000.f), warp) : 0.f;
    const float pre = y > 0 ? 7500.f + 1370.f * (__fdividef((float)units, (float)y) + 0.5f) : 0.f;
    float cost = fmaxf(own, pre);
    if ((x == 0 && own_pos > 0) || (y == 0 && units > 0)) cost = INFINITY;
    int best = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float c = __shfl_xor_sync(0xffffffffu, cost, o);
        const int z = __shfl_xor_sync(0xffffffffu, best, o);
        if (c < cost || (c == cost && z < best)) {
            cost = c;
            best = z;
        }
    }
    return best;
}

// `scratch`: kPrefixMax / 32 * kPrefixMax ints (the stages, not in use yet).  Sequences are taken in
// blocks of 32, a warp to a block, and the blocks' counts added up by whoever needs them: a warp
// that went through 16 blocks alone took 5 us.
__device__ void build_plan(Plan& pl, int* scratch, const PrefixProblem& P, const KCtx& ctx) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = P.prefix.n;
    const int blocks = (P.T + 31) / 32;
    int* count = scratch;  // [block][group]: sequences of the group in the block
    for (int i = tid; i < blocks * n; i += kPThreads) count[i] = 0;
    for (int g = tid; g < n; g += kPThreads) {
        int len = P.prefix.len[g];
        if (len < 0 || len > P.prefix.cap) {
            if (blockIdx.x == 0) report(ctx, ST_BOUNDS, (uint32_t)len);
            len = 0;
        }
        pl.len[g] = len;
        pl.low[g] = INT_MAX;
    }
    __syncthreads();
#pragma unroll 1
    for (int blk = warp; blk < blocks; blk += kOwnWarps) {
        const int t = blk * 32 + lane;
        int g = t < P.T && n > 0 ? P.prefix.of[t] : -1;
        int own = t < P.T ? P.kv_len[t] : 0;
        if (g >= n) {
            if (n > 0 && blockIdx.x == 0) report(ctx, ST_BOUNDS, (uint32_t)g);
            g = -1;
        }
        if (own < 0 || own > P.kv_cap) {
            if (blockIdx.x == 0) report(ctx, ST_BOUNDS, (uint32_t)own);
            own = 0;
        }
        g = max(g, -1);
        // a window reaches as far back in the own cache whatever lies before it
        const int first = P.window > 0 ? max(0, own - P.window) : 0;
        const unsigned same = __match_any_sync(0xffffffffu, g), before = same & ((1u << lane) - 1u);
        if (g >= 0 && before == 0) count[blk * n + g] = __popc(same);
        const int cnt = chunks_of(own - first, P) * P.nkv;
        int incl = cnt;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const int pos = __reduce_add_sync(0xffffffffu, own - first);  // (a cache has < 2^31 rows)
        if (lane == 31) {
            pl.block_chunks[blk] = incl;
            pl.block_pos[blk] = pos;
        }
        if (t < P.T) {
            pl.of[t] = g;
            pl.own_len[t] = own;
            pl.own_first[t] = first;
            pl.rank[t] = __popc(before);
            pl.chunk0[t] = incl - cnt;
        }
    }
    __syncthreads();
    for (int t = tid; t < P.T; t += kPThreads) {
        const int g = pl.of[t], blk = t >> 5;
        int chunks = 0, rank = 0;
        for (int i = 0; i < blk; ++i) {
            chunks += pl.block_chunks[i];
            if (g >= 0) rank += count[i * n + g];
        }
        pl.chunk0[t] += chunks;
        pl.rank[t] += rank;
        if (P.window > 0 && g >= 0) atomicMin(&pl.low[g], max(0, pl.len[g] + pl.own_len[t] - P.window));
    }
    for (int g = tid; g < n; g += kPThreads) {
        int members = 0;
        for (int i = 0; i < blocks; ++i) members += count[i * n + g];
        pl.base[g] = members;
    }
    fence_proxy_async();  // the scratch becomes the target of TMA loads
    __syncthreads();
    for (int g = tid; g < n; g += kPThreads) {
        const int low = P.window > 0 ? pl.low[g] : 0;
        const int members = pl.base[g], len = pl.len[g];
        const int first = low / kPrefixKeys;
        const bool some = members > 0 && low < len;
        pl.low[g] = low;
        pl.first[g] = first;
        // members / tile_seqs rounded up, exact below 2^22 / tile_seqs
        pl.tiles[g] = some ? (int)((unsigned)(members + P.tile_seqs - 1) * P.tile_inv >> 22) : 0;
        pl.steps[g] = some ? (len + kPrefixKeys - 1) / kPrefixKeys - first : 0;
        pl.tile0[g] = pl.tiles[g] * P.nkv;
        pl.step0[g] = pl.tile0[g] * (pl.steps[g] + kTileUnits);
    }
    __syncthreads();
    if (warp == 0) {
        scan3(pl.base, pl.tile0, pl.step0, n, lane);
        const int chunks = __reduce_add_sync(0xffffffffu, lane < blocks ? pl.block_chunks[lane] : 0);
        long long pos = lane < blocks ? pl.block_pos[lane] : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) pos += __shfl_xor_sync(0xffffffffu, pos, o);
        __syncwarp();
        const int x = own_ctas(pos, chunks, P.nkv, pl.step0[n], lane);
        if (lane == 0) {
            const int total = pl.step0[n], shares = min(kPrefixCtas - x, total);  // none empty
            pl.chunk0[P.T] = chunks;
            pl.n_own = x;
            pl.q = shares > 0 ? total / shares : 1;
            pl.n_long = total - pl.q * shares;
            pl.shares = shares;
        }
    }
    __syncthreads();
    for (int t = tid; t < P.T; t += kPThreads) {
        const int g = pl.of[t];
        if (g >= 0) pl.mem[pl.base[g] + pl.rank[t]] = t;
    }
    __syncthreads();
}

// Unit x of the call: group, KV head, tile of that pair, unit (then step) within the tile.
struct Step {
    int g, kvh, tile, k;
};
__device__ __noinline__ Step step_at(const Plan& pl, int n, int x) {
    int lo = 0, hi = n;  // the last group that begins at or before x (empty ones begin with it)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pl.step0[mid] <= x) lo = mid;
        else hi = mid;
    }
    const int units = pl.steps[lo] + kTileUnits, r = x - pl.step0[lo], i = r / units, kvh = i / pl.tiles[lo];
    return {lo, kvh, i - kvh * pl.tiles[lo], r - i * units};
}
// What the units [x, x1) hold of s's tile: its steps from s.k on, how many; x goes to the next tile.
__device__ __forceinline__ int take_tile(const Plan& pl, int& x, int x1, Step& s) {
    const int m = min(x1 - x, pl.steps[s.g] + kTileUnits - s.k), end = s.k + m - kTileUnits;
    x += m;
    s.k = max(0, s.k - kTileUnits);
    return end - s.k;
}

// The own caches: independent warps, each with a private stage of 64 positions, K and V halves
// refilled by themselves (K as soon as the scores are computed, V after its product), as the decode
// layer's attention streams its caches.  S^T = K q^T and O^T += V^T P^T on warp-level products, the
// heads of a group their N; a chunk's (m, l, a) go to its partial.
struct OwnChunk {
    int t, kvh, c, p0, p1;
};
__device__ __forceinline__ OwnChunk own_chunk(const Plan& pl, const PrefixProblem& P, int i) {
    int lo = 0, hi = P.T;  // the last sequence whose chunks begin at or before i
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pl.chunk0[mid] <= i) lo = mid;
        else hi = mid;
    }
    const int per = (pl.chunk0[lo + 1] - pl.chunk0[lo]) / P.nkv, r = i - pl.chunk0[lo];
    const int kvh = r / per, c = r - kvh * per, p0 = pl.own_first[lo] + (c << P.chunk_log2);
    return {lo, kvh, c, p0, min(pl.own_len[lo], p0 + (1 << P.chunk_log2))};
}
// The chunk behind k, if there is one (the search and its divisions took 600 cycles a chunk).
__device__ __forceinline__ void own_next(const Plan& pl, const PrefixProblem& P, OwnChunk& k) {
    ++k.c;
    k.p0 = k.p1;
    if (k.p0 >= pl.own_len[k.t]) {
        k.c = 0;
        if (++k.kvh == P.nkv) {
            k.kvh = 0;
            do ++k.t;
            while (pl.own_first[k.t] >= pl.own_len[k.t]);
        }
        k.p0 = pl.own_first[k.t];
    }
    k.p1 = min(pl.own_len[k.t], k.p0 + (1 << P.chunk_log2));
}

template <int NT>
__device__ void own_part(const PrefixProblem& P, const Plan& pl, uint8_t* ring_all, uint64_t* bars,
                         const KCtx& ctx) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, cq = lane & 3;
    const long long total = pl.chunk0[P.T], W = (long long)pl.n_own * kOwnWarps;
    const long long gw = (long long)warp * pl.n_own + blockIdx.x;
    const int i1 = (int)((gw + 1) * total / W);
    int i = (int)(gw * total / W);
    if (i >= i1) return;
    uint8_t* ring = ring_all + (size_t)warp * 2 * kOwnHalf;
    uint64_t *bar_k = bars + 2 * warp, *bar_v = bar_k + 1;
    const uint32_t ka = smem_u32(ring), va = ka + kOwnHalf;
    const uint64_t pol = policy_evict_first();
    OwnChunk cs = own_chunk(pl, P, i), ld = cs;
    int ld_i = i, ld_p = ld.p0, v_row = 0;
    // The query fragments of a new (sequence, KV head) are asked for with its first keys, which is
    // after the last use of the ones before
    uint32_t qf[NT][4][2];
    int pair = -1;
    uint32_t n_k = 0, n_v = 0, c_k = 0, c_v = 0;  // halves issued and consumed
    auto issue_k = [&] {
        const int ld_pair = ld.t * P.nkv + ld.kvh;
        v_row = ld_pair * P.kv_cap + ld_p;
        if (lane == 0) {
            mbar_arrive_expect_tx(bar_k, kOwnHalf);
            tma_load_2d(ring, &P.tmK, bar_k, 0, v_row, pol);
        }
        ++n_k;
        if (ld_pair != pair) {
            pair = ld_pair;
            const bf16* q = P.q + (size_t)pair * P.G * 64;  // [T][nkv][G][64]
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const int h = nt * 8 + g;
                    const uint32_t* src = reinterpret_cast<const uint32_t*>(q + h * 64 + kk * 16 + 2 * cq);
                    qf[nt][kk][0] = h < P.G ? src[0] : 0u;
                    qf[nt][kk][1] = h < P.G ? src[4] : 0u;
                }
        }
        ld_p += kOwnPos;
        if (ld_p >= ld.p1) {
            if (++ld_i < i1) own_next(pl, P, ld);
            ld_p = ld.p0;
        }
    };
    auto issue_v = [&] {
        if (lane == 0) {
            mbar_arrive_expect_tx(bar_v, kOwnHalf);
            tma_load_2d(ring + kOwnHalf, &P.tmV, bar_v, 0, v_row, pol);
        }
        ++n_v;
    };
    issue_k();
    issue_v();
    float m[NT][2], l[NT][2], o[4][NT][4];
    bool ok = true;
    for (; i < i1 && ok; ++i) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int md = 0; md < 4; ++md) o[md][nt][0] = o[md][nt][1] = o[md][nt][2] = o[md][nt][3] = 0.f;
        }
        for (int p = cs.p0; p < cs.p1; p += kOwnPos) {
            if (__any_sync(0xffffffffu, !mbar_wait(bar_k, c_k & 1u, ctx.timeout_ns))) {
                if (lane == 0) report(ctx, ST_TIMEOUT, 40);
                ok = false;
                break;
            }
            ++c_k;
            const int valid = min(kOwnPos, cs.p1 - p);
            float s[4][NT][4];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
                const int r = mt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    uint32_t a[4];
                    ldsm_x4(ka + sw128(r, kk * 2 + (lane >> 4)), a);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(s[mt][nt], a, qf[nt][kk][0], qf[nt][kk][1]);
                }
            }
            // K is consumed: the next keys load beside the softmax and the V product
            fence_proxy_async();
            __syncwarp();
            if (ld_i < i1) issue_k();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = s[mt][nt][e] * P.scale_log2;
                        if (mt * 16 + (e >> 1) * 8 + g >= valid) v = -INFINITY;
                        s[mt][nt][e] = v;
                        mx[e & 1] = fmaxf(mx[e & 1], v);
                    }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], d));
                    const float nm = fmaxf(m[nt][e], mx[e]);
                    const float c = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - nm);
                    const float sub = nm == -INFINITY ? 0.f : nm;
                    m[nt][e] = nm;
                    float sum = 0.f;
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const float w = ex2(s[mt][nt][2 * f + e] - sub);
                            s[mt][nt][2 * f + e] = w;
                            sum += w;
                        }
                    l[nt][e] = l[nt][e] * c + sum;
#pragma unroll
                    for (int md = 0; md < 4; ++md) {
                        o[md][nt][e] *= c;
                        o[md][nt][2 + e] *= c;
                    }
                }
            }
            if (__any_sync(0xffffffffu, !mbar_wait(bar_v, c_v & 1u, ctx.timeout_ns))) {
                if (lane == 0) report(ctx, ST_TIMEOUT, 41);
                ok = false;
                break;
            }
            ++c_v;
            if (valid < kOwnPos) {  // what lies behind the chunk is arbitrary: its weight is 0
                uint4* v4 = reinterpret_cast<uint4*>(ring + kOwnHalf);
                for (int e = valid * 8 + lane; e < kOwnPos * 8; e += 32) v4[e] = make_uint4(0, 0, 0, 0);
                __syncwarp();
            }
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                uint32_t b0[NT], b1[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {  // rounded to bf16, V's type, as for the prefixes
                    b0[nt] = movmatrix_t(pack_bf16x2(s[ks][nt][0], s[ks][nt][1]));
                    b1[nt] = movmatrix_t(pack_bf16x2(s[ks][nt][2], s[ks][nt][3]));
                }
                const int r = ks * 16 + ((lane >> 4) << 3) + (lane & 7);
#pragma unroll
                for (int md = 0; md < 4; ++md) {
                    uint32_t a[4];
                    ldsm_x4_t(va + sw128(r, md * 2 + ((lane >> 3) & 1)), a);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(o[md][nt], a, b0[nt], b1[nt]);
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (n_v < n_k) issue_v();
        }
        if (!ok) break;
        const size_t at = ((size_t)(cs.t * P.nkv + cs.kvh) * P.S_max + cs.c) * P.G;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
                const int h = nt * 8 + 2 * cq + e;
                if (h >= P.G) continue;
                if (g == 0) *reinterpret_cast<float2*>(P.own_ml + (at + h) * 2) = make_float2(m[nt][e], l[nt][e]);
                float* acc = P.own_acc + (at + h) * 64 + g;
#pragma unroll
                for (int md = 0; md < 4; ++md) {
                    acc[md * 16] = o[md][nt][e];
                    acc[md * 16 + 8] = o[md][nt][2 + e];
                }
            }
        if (i + 1 < i1) own_next(pl, P, cs);
    }
    // loads in flight into this warp's stage, if it gave up (bounded)
    for (; c_k < n_k; ++c_k) (void)mbar_wait(bar_k, c_k & 1u, 10000000ull);
    for (; c_v < n_v; ++c_v) (void)mbar_wait(bar_v, c_v & 1u, 10000000ull);
}

// The prefixes.  Warp 0 loads keys and values (TMA, a ring of steps), warps 4-7 and 8-11 are two
// softmax groups of 128 rows each, and warps 1 and 2 issue one group's matrix products each.  A
// step's positions are taken in halves of 64.  Per half and group
//     S = Q K^T   (M = 128 rows, N = 64 positions, K = 64), accumulators in tensor memory;
//     P = exp2(scale S - m) by the group's threads, one row each, as bf16 over S's first columns;
//     O += P V    (M = 128, N = 64 dims, K = 64), P read from tensor memory.
// Three buffers hold S, then P: "P(i) is written" frees nothing but lets the product begin, and
// S(i + 3) is issued when that product is complete (the two are not ordered otherwise).  With two
// buffers for S and two for P the softmax found S late; with three it is complete 98 % of the time.
// The weights are taken against a maximum m that is only raised when a row's scores pass it by
// more than 2^8 (weights up to 256 lose nothing in bf16 or fp32); the half's own maximum is found
// beside the exponentials, and in the rare case that it does, O and the sum are rescaled and the
// half is done again, before P takes S's place.  m begins at 0, when the first scores are near it.
//
// A half takes 0.6 to 0.7 us where 0.26 us of exponentials (8 a cycle and scheduler) are its floor:
// two softmax warps to a scheduler do not cover each other's waits (a barrier that passes at once
// costs 150 cycles, 32 columns of scores 130, P's way back 85).  Without any arithmetic in the
// softmax the kernel would take 0.42 us for a half, the way from P through both products to S.
constexpr int kPStages = 5;
constexpr int kPSub = 64;           // positions of a half
constexpr float kPRaise = 8.f;
constexpr uint32_t kPBufs = 3;      // S (then P) of so many halves
constexpr uint32_t kTmemS = 0, kTmemO = 384;  // columns; per group 3 x 64 and 64

struct PrefixBars {
    uint64_t kv_full[kPStages], kv_empty[kPStages];
    uint64_t q_full[2];        // the group's query rows are in shared memory
    uint64_t s_full[2][kPBufs];  // [group][buffer]; the group's half i uses buffer i % 3, phase i / 3
    uint64_t p_full[2][kPBufs];
    uint64_t pv_done[2][kPBufs];  // O holds the half
    uint64_t own[kOwnWarps][2];  // an own warp's K and V halves
    uint32_t tmem;
    int err;
};

// The part of a tile that a share holds: steps [s.k, s.k + steps), halves of them that hold
// positions of the prefix.
__device__ __forceinline__ int halves_of(const Plan& pl, const Step& s, int steps) {
    const int p0 = (pl.first[s.g] + s.k) * kPrefixKeys;
    return (min(pl.len[s.g] - p0, steps * kPrefixKeys) + kPSub - 1) / kPSub;
}

// The share that holds unit x: the first n_long have q + 1 units, the others q.
__device__ __forceinline__ int share_of(const Plan& pl, int x) {
    const int r = x - pl.n_long * (pl.q + 1);
    return r < 0 ? x / (pl.q + 1) : pl.n_long + r / pl.q;
}

// The parts of every (sequence, KV head), for the merge: pairs i, i + stride, ...
__device__ void list_parts(const Plan& pl, const PrefixProblem& P, int i, int stride) {
    for (; i < P.T * P.nkv; i += stride) {
        const int t = i / P.nkv, kvh = i - t * P.nkv, g = pl.of[t];
        PrefixParts p = {0, 0, 0, chunks_of(pl.own_len[t] - pl.own_first[t], P)};
        if (g >= 0 && pl.tiles[g] > 0) {
            const int rank = pl.rank[t], seq = (int)((unsigned)rank * P.tile_inv >> 22);
            const int tile = kvh * pl.tiles[g] + seq;
            const int x = pl.step0[g] + tile * (pl.steps[g] + kTileUnits) + kTileUnits;  // its first step
            const int s0 = share_of(pl, x);
            p.slot = s0 + pl.tile0[g] + tile;
            p.row = (rank - seq * P.tile_seqs) * P.G;
            p.n_pre = share_of(pl, x + pl.steps[g] - 1) - s0 + 1;
        }
        P.parts[i] = p;
    }
}

template <int NT>
__global__ void __launch_bounds__(kPThreads, 1)
    prefix_attn_kernel(const __grid_constant__ PrefixProblem P, const KCtx ctx) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* qs = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));  // [2][128 rows]
    uint8_t* ring = qs + 2 * 128 * 128;  // (the own warps' stages take the place of both)
    static_assert(2 * 128 * 128 + kPStages * 2 * kPHalf >= kOwnWarps * 2 * kOwnHalf, "own stages fit");
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
            for (int i = 0; i < (int)kPBufs; ++i) {
                mbar_init(&bar.s_full[h][i], 1);
                mbar_init(&bar.p_full[h][i], 4);
                mbar_init(&bar.pv_done[h][i], 1);
            }
        }
        for (int i = 0; i < kOwnWarps; ++i) {
            mbar_init(&bar.own[i][0], 1);
            mbar_init(&bar.own[i][1], 1);
        }
        bar.err = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    griddep_wait();  // what is above may run beside the kernel before
    task_begin(ctx);
    static_assert(kPrefixMax / 32 * kPrefixMax * 4 <= 2 * 128 * 128 + kPStages * 2 * kPHalf, "scratch fits");
    build_plan(pl, reinterpret_cast<int*>(qs), P, ctx);  // ends with a barrier
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    const int n = P.prefix.n;
    const int b = (int)blockIdx.x - pl.n_own;  // this CTA's share
    const int x0 = b * pl.q + min(b, pl.n_long);
    const int x1 = b < pl.shares ? x0 + pl.q + (b < pl.n_long ? 1 : 0) : x0;
    volatile int* err = &bar.err;
    auto gave_up = [&](uint32_t where) {
        report(ctx, ST_TIMEOUT, where);
        *err = 1;
    };

    if (b < 0) {
        if (pl.n_own == kPrefixCtas) list_parts(pl, P, blockIdx.x * kPThreads + tid, kPrefixCtas * kPThreads);
        own_part<NT>(P, pl, qs, &bar.own[0][0], ctx);
    } else if (warp == 0) {
        if (elect_one()) {
            const uint64_t pol = policy_evict_last();  // the other row tiles read it too
            uint32_t it = 0;
            for (int x = x0; x < x1 && !*err;) {
                Step s = step_at(pl, n, x);
                const int steps = take_tile(pl, x, x1, s);
                int row = (s.g * P.nkv + s.kvh) * P.prefix.cap + (pl.first[s.g] + s.k) * kPrefixKeys;
#pragma unroll 1
                for (int i = 0; i < steps; ++i, ++it, row += kPrefixKeys) {
                    const uint32_t st = it % kPStages, use = it / kPStages;
                    if (use > 0 && !mbar_wait_near(&bar.kv_empty[st], (use - 1) & 1u, ctx.timeout_ns)) {
                        gave_up(20);
                        break;
                    }
                    uint8_t* dst = ring + st * 2 * kPHalf;
                    mbar_arrive_expect_tx(&bar.kv_full[st], 2 * kPHalf);
                    tma_load_2d(dst, &P.tmPK, &bar.kv_full[st], 0, row, pol);
                    tma_load_2d(dst + kPHalf, &P.tmPV, &bar.kv_full[st], 0, row, pol);
                }
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
            const uint32_t ts = tmem + kTmemS + 64 * kPBufs * h, to = tmem + kTmemO + 64 * h;
            uint32_t n_q = 0;                      // tiles of this group
            uint32_t buf_s = 0;                    // buffer of the next S
            uint32_t buf_p = 0, ph_p = 0;          // buffer and phase of the next P
            uint32_t st_s = 0, ph_s = 0, st_p = 0;  // stages of the next S and the next product
            bool ok = true;
            auto scores = [&](int j) {  // S = Q K^T of the tile's half j
                if ((j & 1) == 0 && !(ok = mbar_wait_near(&bar.kv_full[st_s], ph_s, ctx.timeout_ns))) {
                    gave_up(22);
                    return;
                }
                const uint64_t dk = dk0 + st_s * kStageD + (j & 1) * kHalfD;
#pragma unroll
                for (int k = 0; k < 4; ++k) tc_mma_bf16(ts + 64 * buf_s, dq + 2 * k, dk + 2 * k, id_s, k > 0);
                tc_commit(&bar.s_full[h][buf_s]);
                if (++buf_s == kPBufs) buf_s = 0;
                if ((j & 1) && ++st_s == kPStages) st_s = 0, ph_s ^= 1;
            };
            for (int x = x0; x < x1 && ok;) {
                Step s = step_at(pl, P.prefix.n, x);
                const int steps = take_tile(pl, x, x1, s);
                if (steps <= 0) continue;
                const int halves = halves_of(pl, s, steps);
                const int rows = min(P.tile_seqs, pl.base[s.g + 1] - pl.base[s.g] - s.tile * P.tile_seqs) * P.G;
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
                for (int j = 0; j < min(halves, (int)kPBufs) && ok; ++j) scores(j);
                for (int j = 0; j < halves && ok; ++j) {
                    if (!(ok = mbar_wait_near(&bar.p_full[h][buf_p], ph_p, ctx.timeout_ns))) {
                        gave_up(21);
                        break;
                    }
                    tc_fence_after();
                    const uint64_t dv = dv0 + st_p * kStageD + (j & 1) * kHalfD;
#pragma unroll
                    for (int k = 0; k < kPSub / 16; ++k)  // O += P V
                        tc_mma_bf16_ta(to, ts + 64 * buf_p + 8 * k, dv + k * (16 * 128 / 16), id_o, !(j == 0 && k == 0));
                    tc_commit(&bar.pv_done[h][buf_p]);
                    // the next S of this buffer: it may pass the product unless that is complete
                    if (!(ok = mbar_wait_near(&bar.pv_done[h][buf_p], ph_p, ctx.timeout_ns))) {
                        gave_up(33);
                        break;
                    }
                    tc_fence_after();
                    if ((j & 1) || j + 1 == halves) {
                        mbar_arrive(&bar.kv_empty[st_p]);
                        if (++st_p == kPStages) st_p = 0;
                    }
                    if (++buf_p == kPBufs) buf_p = 0, ph_p ^= 1;
                    if (j + (int)kPBufs < halves) scores(j + kPBufs);
                }
                if (halves & 1) {  // the last stage's second half holds no positions
                    if (++st_s == kPStages) st_s = 0, ph_s ^= 1;
                }
            }
        }
        __syncwarp();
    } else if (warp == 3) {
        list_parts(pl, P, b * 32 + lane, (kPrefixCtas - pl.n_own) * 32);
    } else {
        const int h = (warp - 4) >> 2, quad = warp & 3;  // a warp reads its quadrant's TMEM lanes
        const int r = h * 128 + quad * 32 + lane;        // this thread's row of the tile
        const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t ts = tl + kTmemS + 64 * kPBufs * h, to = tl + kTmemO + 64 * h;
        const int row_of = (65536 + P.G - 1) / P.G;      // r / G = r * row_of >> 16 for r < 256
        const float2 sc2 = make_float2(P.scale_log2, P.scale_log2);
        uint32_t buf = 0, ph = 0;  // buffer and phase of the half
        int done = 0;              // steps of earlier tiles
        bool ok = true;
        // every wait's outcome is the warp's: its tensor-memory accesses are warp-wide
        auto wait = [&](uint64_t* bar_, uint32_t parity, uint32_t where) {
            if (__all_sync(0xffffffffu, mbar_wait_near(bar_, parity, ctx.timeout_ns))) return true;
            if (lane == 0) gave_up(where);
            return false;
        };
        auto multiplied = [&](uint32_t where) {  // the half before
            return buf > 0 ? wait(&bar.pv_done[h][buf - 1], ph, where) : wait(&bar.pv_done[h][kPBufs - 1], ph ^ 1u, where);
        };
        for (int x = x0; x < x1 && ok;) {
            Step s = step_at(pl, n, x);
            const int steps = take_tile(pl, x, x1, s);
            if (steps <= 0) continue;
            const int halves = halves_of(pl, s, steps);
            const int seq0 = pl.base[s.g] + s.tile * P.tile_seqs;
            const int rows = min(P.tile_seqs, pl.base[s.g + 1] - seq0) * P.G;
            const int i0 = done;  // first step's place in the share
            done += steps;
            if (rows <= 128 * h) continue;
            const int len = pl.len[s.g], seen = pl.low[s.g];
            // this warp's 32 query rows, 8 lanes to a row, into the swizzled tile (zeros past the
            // tile's rows: rows do not mix, and theirs are not stored)
            {
                const int q = r * row_of >> 16;
                const int at = r < rows ? pl.mem[seq0 + q] * P.nq + s.kvh * P.G + r - q * P.G : -1;
                uint8_t* dst = qs + (h * 128 + quad * 32) * 128;
                uint4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int src = __shfl_sync(0xffffffffu, at, i * 4 + (lane >> 3));
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (src >= 0) v[i] = reinterpret_cast<const uint4*>(P.q + (size_t)src * 64)[lane & 7];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(dst + sw128(i * 4 + (lane >> 3), lane & 7)) = v[i];
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.q_full[h]);
            }
            int low = 0;
            if (P.window > 0 && r < rows) {
                low = max(0, len + pl.own_len[pl.mem[seq0 + (r * row_of >> 16)]] - P.window);
            }
            const bool live = h * 128 + quad * 32 < rows;  // some row of this warp counts
            float m = 0.f;  // what the weights are taken against (scaled scores, base 2)
            float2 l2 = make_float2(0.f, 0.f);
            int pos0 = (pl.first[s.g] + s.k) * kPrefixKeys;
            for (int j = 0; j < halves; ++j, pos0 += kPSub) {
                if (!(ok = wait(&bar.s_full[h][buf], ph, 24))) break;
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
                    float2 l_old = l2;  // of the halves before, against m
                    for (int tries = 0;; ++tries) {
                        // a row that has seen nothing yet: every score is -inf, every weight 0
                        const float sub = m == -INFINITY ? 0.f : -m;
                        const float2 sub2 = make_float2(sub, sub);
                        float sa[32], sb[32], mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        uint32_t wa[16], wb[16];
                        auto weights = [&](const float (&sr)[32], uint32_t (&w)[16]) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float2 v = fma2_ordered(make_float2(sr[2 * e], sr[2 * e + 1]), sc2, sub2);
                                mx[e & 1] = fmaxf(mx[e & 1], v.x);
                                mx[2 + (e & 1)] = fmaxf(mx[2 + (e & 1)], v.y);
                                v.x = ex2(v.x);
                                v.y = ex2(v.y);
                                l2 = add2(l2, v);
                                // The weight's rounding to bf16: a product's operands have one
                                // type, V's.  It makes o's error 1.2 to 1.5 times that of one
                                // rounding; a second product with the rest would double the
                                // tensor work and lengthen the softmax, which bounds the kernel.
                                w[e] = pack_bf16x2(v.x, v.y);
                            }
                        };
                        // the second scores are on their way beside the first ones' exponentials
                        tmem_ld_wait_x32(ts + 64 * buf, sa);
                        tmem_ld_x32(ts + 64 * buf + 32, sb);
                        weights(sa, wa);
                        tmem_ld_wait();
                        weights(sb, wb);
                        const float over = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));  // past m
                        // the first half also raises from below: its scores may be far under 0
                        const bool far = over > (m == -INFINITY ? -INFINITY : kPRaise) ||
                                         (j == 0 && m == 0.f && over < -kPRaise);
                        // (scaled scores past 2^28 round by more than that: m is near enough the second
                        // time, and weights up to 2^64 below 2^31)
                        if (!__any_sync(0xffffffffu, far) || tries == 2) {
                            tmem_st_x16(ts + 64 * buf, wa);  // P takes S's place
                            tmem_st_x16(ts + 64 * buf + 16, wb);
                            break;
                        }
                        const float top = over - sub, nm = j == 0 ? top : fmaxf(m, top);
                        const float c = j == 0 || m == -INFINITY ? 0.f : ex2(m - nm);
                        m = nm;
                        l_old.x *= c;
                        l_old.y *= c;
                        l2 = l_old;
                        if (j == 0) continue;
                        if (!(ok = multiplied(25))) break;
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
                if (++buf == kPBufs) buf = 0, ph ^= 1;
            }
            if (!ok) break;
            // the last product, then this row's partial
            if (!multiplied(26)) break;
            tc_fence_after();
            if (live) {
                const size_t slot = b + (size_t)(pl.tile0[s.g] + s.kvh * pl.tiles[s.g] + s.tile);
                const size_t at = slot * kPrefixRows + r;
                if (r < rows) *reinterpret_cast<float2*>(P.pre_ml + at * 2) = make_float2(m, l2.x + l2.y);
                // The rows leave through this warp's part of the query tile, 16 dims at a time: a
                // thread's own row straight to memory is 32 lines to a store
                float4* buf = reinterpret_cast<float4*>(qs + (h * 128 + quad * 32) * 128);  // [32][4]
                const int row0 = h * 128 + quad * 32 + (lane >> 2);
                float4* dst = reinterpret_cast<float4*>(P.pre_acc + (slot * kPrefixRows + row0) * 64) + (lane & 3);
#pragma unroll 1
                for (int c = 0; c < 64; c += 16, dst += 4) {
                    float o[16];
                    tmem_ld_wait_x16(to + c, o);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        buf[lane * 4 + (i ^ (lane >> 1 & 3))] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int q = 8 * i + (lane >> 2);
                        if (row0 + 8 * i < rows) dst[8 * i * 16] = buf[q * 4 + ((lane & 3) ^ (q >> 1 & 3))];
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
    task_end(ctx);
}

// The merge: one warp per (sequence, query head), lane l holds dims 2l and 2l + 1.  The parts join
// in a fixed order, the prefix's shares, then the own chunks, 32 at a time.  Little work behind a
// chain of dependent loads: a part list written by the first kernel, the first accumulators loaded
// beside the maxima.
__global__ void __launch_bounds__(512) prefix_merge_kernel(const __grid_constant__ PrefixProblem P, const KCtx ctx) {
    griddep_wait();
    task_begin(ctx);
    const int lane = threadIdx.x & 31, h = threadIdx.x >> 5;
    const int pair = blockIdx.x, t = pair / P.nkv, kvh = pair - t * P.nkv;
    const PrefixParts q = P.parts[pair];
    const size_t row = (size_t)q.slot * kPrefixRows + q.row + h;
    const size_t own = ((size_t)pair * P.S_max - q.n_pre) * P.G + h;  // part k >= n_pre at own + G k
    const unsigned own_step = P.G * 64;
    const float *pre_acc = P.pre_acc + row * 64 + 2 * lane, *own_acc = P.own_acc + own * 64 + 2 * lane;
    const int parts = q.n_pre + q.n_own;
    float M = -INFINITY, L = 0.f;
    float2 a = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 < parts; k0 += 32) {
        const int nk = min(32, parts - k0);
        auto acc_of = [&](int k) {
            const float* p = k < q.n_pre ? pre_acc + (size_t)k * (kPrefixRows * 64)
                                         : own_acc + (size_t)(unsigned)k * own_step;
            return __ldcg(reinterpret_cast<const float2*>(p));
        };
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < nk) {
            const int k = k0 + lane;
            const bool pre = k < q.n_pre;
            ml = __ldcg(reinterpret_cast<const float2*>(pre ? P.pre_ml + row * 2 : P.own_ml + own * 2) +
                        (size_t)(unsigned)k * (pre ? (unsigned)kPrefixRows : (unsigned)P.G));
        }
        float2 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < nk) v[i] = acc_of(k0 + i);
        const float top = fmaxf(M, warp_max(ml.x)), sub = top == -INFINITY ? 0.f : top;
        const float old = ex2(M - sub), w = ex2(ml.x - sub);
        M = top;
        L = fmaf(L, old, warp_sum(w * ml.y));
        a.x *= old;
        a.y *= old;
#pragma unroll 1
        for (int i0 = 0; i0 < nk; i0 += 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float wk = __shfl_sync(0xffffffffu, w, i0 + i);
                if (i0 + i < nk) {
                    a.x = fmaf(wk, v[i].x, a.x);
                    a.y = fmaf(wk, v[i].y, a.y);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i0 + 8 + i < nk) v[i] = acc_of(k0 + i0 + 8 + i);
        }
    }
    // a row that sees nothing: o = 0, lse = -inf
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const size_t at = (size_t)t * P.nq + kvh * P.G + h;
    *reinterpret_cast<uint32_t*>(P.o + at * 64 + 2 * lane) = pack_bf16x2(a.x * inv, a.y * inv);
    if (P.lse != nullptr && lane == 0)
        P.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    task_end(ctx);
}

}  // namespace

int enqueue_prefix(Launcher& L, const PrefixProblem& p, const KCtx& c) {
    const size_t smem = 1024 + 2 * 128 * 128 + kPStages * 2 * kPHalf + sizeof(PrefixBars) + sizeof(Plan);
    void* args[] = {(void*)&p, (void*)&c};
    const void* f = p.G <= 8 ? (const void*)prefix_attn_kernel<1> : (const void*)prefix_attn_kernel<2>;
    const int e = L.launch(f, dim3(kPrefixCtas), dim3(kPThreads), smem, args, true);
    if (e) return e;
    return L.launch((const void*)prefix_merge_kernel, dim3(p.T * p.nkv), dim3(32 * p.G), 0, args, true);
}

}  // namespace sgp
