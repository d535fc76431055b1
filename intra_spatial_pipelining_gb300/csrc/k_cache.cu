// What a bounded KV cache needs beside the attention: the attention weight that each cached
// position gathers, and the eviction that keeps the heaviest positions.
//
//   weights   acc[t][j][p] += sum over the heads h of group j of exp(q_h . k_p / sqrt(d) - lse_h),
//             lse_h the log-sum-exp that the attention returned for head h;
//   eviction  keep the first n_sink and the last n_recent positions and, of the others, the
//             budget - n_sink - n_recent with the largest acc (ties to the lower position, NaN
//             below every number), in their order.
#include <algorithm>

#include "evict_words.h"
#include "serving.cuh"

namespace sgp {

namespace {

// 32 bytes that are read or written once: they leave L2 first.  (Attention weights, 295 MB, call
// after call: 45.6 us so, since a part of K is still in L2 then, 51 without; the eviction of 815 MB
// 137.5 and 140.)
__device__ __forceinline__ void load_once(const void* p, uint4& a, uint4& b) {
    asm volatile("ld.global.nc.L1::no_allocate.L2::evict_first.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p));
}

__device__ __forceinline__ void store_once(void* p, const uint4& a, const uint4& b) {
    asm volatile("st.global.L2::evict_first.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y),
                 "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

// ---------------------------------------------------------------------------------------
// Accumulated attention weights.  One pass over K; the scores are S = K q^T on warp-level
// matrix products (M = 16 positions, N = 8 heads, K = 64 dims) with K fragments loaded straight
// from global memory: lane (g, c) loads 32 bytes of rows g and g + 8, and both operands read
// the same permutation of the dims, so each product still sums matching pairs.  An item is 64
// positions of one (sequence, KV head); the warps of the grid share the items in equal runs.
// Bound by HBM: 64 sequences x 64 / 8 heads, up to 8192 positions, 295 MB, 45.6 us call after call
// and 52.5 with nothing in L2 (5.6 TB/s, 0.83 of a copy's rate; the next item's loads issued beside
// this one's products made no difference to either); 3 sequences of up to 577 positions 4.0 us, of
// which a launch is 2.
// ---------------------------------------------------------------------------------------
constexpr int kWThreads = 256;
constexpr int kWPos = 64;
constexpr int kWMax = 512;

template <int NT>
__global__ void __launch_bounds__(kWThreads, 2) weights_kernel(const WeightsProblem P, const KCtx ctx) {
    __shared__ int pre[kWMax + 1];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cq = lane & 3;
    griddep_wait();
    task_begin(ctx);
    if (warp == 0) {  // items before each sequence
        int run = 0;
        for (int t0 = 0; t0 < P.T; t0 += 32) {
            const int t = t0 + lane;
            int L = t < P.T ? P.kv_len[t] : 0;
            if (L < 0 || L > P.cap) {
                if (blockIdx.x == 0) report(ctx, ST_BOUNDS, (uint32_t)L);
                L = 0;
            }
            const int cnt = (L + kWPos - 1) / kWPos * P.nkv;
            int incl = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (t < P.T) pre[t] = run + incl - cnt;
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) pre[P.T] = run;
    }
    __syncthreads();
    const long long total = pre[P.T], W = (long long)gridDim.x * (kWThreads / 32);
    const long long gw = (long long)warp * gridDim.x + blockIdx.x;
    const int i0 = (int)(gw * total / W), i1 = (int)((gw + 1) * total / W);
    if (i0 < i1) {
        int t = 0, hi = P.T;  // largest t with pre[t] <= i0
        while (hi - t > 1) {
            const int mid = (t + hi) >> 1;
            if (pre[mid] <= i0) t = mid;
            else hi = mid;
        }
        int last = -1;  // pair whose queries are loaded
        uint32_t qf[NT][2][4];
        float off[NT][2];  // lse of heads 2 cq, 2 cq + 1 of each tile, in base 2
        for (int i = i0; i < i1; ++i) {
            while (i >= pre[t + 1]) ++t;
            const int per = (pre[t + 1] - pre[t]) / P.nkv, r = i - pre[t];
            const int kvh = r / per, p0 = (r - kvh * per) * kWPos;
            const int pair = t * P.nkv + kvh, L = P.kv_len[t], n = min(kWPos, L - p0);
            const bf16* k = P.k + ((size_t)pair * P.cap + p0) * 64;
            uint4 kf[4][2][2];  // [16-position tile][row half][dim half]
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int p = m * 16 + h * 8 + g;
                    const uint4* src = reinterpret_cast<const uint4*>(k + (size_t)min(p, n - 1) * 64);
                    load_once(src + 2 * cq, kf[m][h][0], kf[m][h][1]);
                }
            // lane (g, c) owns positions 16 c + g and 16 c + g + 8
            float* acc = P.acc + (size_t)pair * P.cap + p0 + cq * 16 + g;
            const bool own0 = cq * 16 + g < n, own1 = cq * 16 + g + 8 < n;
            const float a0 = own0 ? acc[0] : 0.f, a1 = own1 ? acc[8] : 0.f;
            if (pair != last) {
                last = pair;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int h = nt * 8 + g;
                    const uint4* src = reinterpret_cast<const uint4*>(
                        P.q + (size_t)t * P.nq * 64 + (size_t)(kvh * P.G + min(h, P.G - 1)) * 64);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint4 v = src[2 * cq + e];
                        qf[nt][e][0] = v.x;
                        qf[nt][e][1] = v.y;
                        qf[nt][e][2] = v.z;
                        qf[nt][e][3] = v.w;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int hc = nt * 8 + 2 * cq + e;
                        off[nt][e] = hc < P.G ? P.lse[(size_t)t * P.nq + kvh * P.G + hc] * 1.4426950408889634f
                                              : INFINITY;
                    }
                }
            }
            float w0 = 0.f, w1 = 0.f;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                float r0 = 0.f, r1 = 0.f;  // rows g and g + 8 over this lane's heads
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t x0[4] = {kf[m][0][e].x, kf[m][1][e].x, kf[m][0][e].y, kf[m][1][e].y};
                        const uint32_t x1[4] = {kf[m][0][e].z, kf[m][1][e].z, kf[m][0][e].w, kf[m][1][e].w};
                        mma16816(s, x0, qf[nt][e][0], qf[nt][e][1]);
                        mma16816(s, x1, qf[nt][e][2], qf[nt][e][3]);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // no weight from heads past the group, nor where nothing was attended
                        // (lse = -inf, which only an empty row has)
                        const bool live = fabsf(off[nt][e]) != INFINITY;
                        r0 += live ? exp2f(fmaf(s[e], P.scale_log2, -off[nt][e])) : 0.f;
                        r1 += live ? exp2f(fmaf(s[2 + e], P.scale_log2, -off[nt][e])) : 0.f;
                    }
                }
                r0 += __shfl_xor_sync(0xffffffffu, r0, 1);
                r1 += __shfl_xor_sync(0xffffffffu, r1, 1);
                r0 += __shfl_xor_sync(0xffffffffu, r0, 2);
                r1 += __shfl_xor_sync(0xffffffffu, r1, 2);
                if (cq == m) {
                    w0 = r0;
                    w1 = r1;
                }
            }
            if (own0) acc[0] = a0 + w0;
            if (own1) acc[8] = a1 + w1;
        }
    }
    task_end(ctx);
}

// ---------------------------------------------------------------------------------------
// Eviction: which positions stay, then the move of their rows.
//
// The keys of the positions between the sinks and the recent ones are acc mapped to unsigned
// integers of the same order, kept in shared memory (those that do not fit are read again).  The
// threshold, the need-th largest key, is found two bits a round from counts, until exactly `need`
// keys reach it; the positions above it stay, and of those equal to it the first ones.
//
// Into another cache one kernel does both: a few CTAs to a (sequence, KV head), each of which makes
// the whole selection and moves its part of the rows, so that nothing is waited for and one CTA's
// selection runs beside another's copies.  In place the selection is a kernel of its own, because
// the move overwrites what it reads.
//
// Bound by the move: 64 sequences x 8 KV heads, 8192 -> 4096 positions, take 135.5 us for 815 MB
// (6.0 TB/s), within three of the rows 0, 2, 4 ... without a selection: every second 128-byte row of
// the source does not read at a plain copy's rate.  Four CTAs of 256 threads to an SM took
// 221 us, one of 1024 146 us.  Two caches of 640 -> 512 take 9.3 us, latency: up to sixteen rounds
// of counts with a barrier each, then loads of the rows.
// ---------------------------------------------------------------------------------------
constexpr int kEThreads = 512;
constexpr int kEWarps = kEThreads / 32;
constexpr int kEUnroll = 4;  // 32-byte pieces in flight to a thread

__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 0u;             // NaN: below -inf
    if (v == 0.f) return 0x80000000u;  // -0 = +0
    const uint32_t u = __float_as_uint(v);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

constexpr int kESeg = 32;  // blocks of positions whose counts are summed at a time

struct SelectSmem {
    int cnt[2][3][kEWarps];
    int base[2][kESeg * kEWarps];  // larger and equal keys before a warp's positions of a block
    int total[2];
};

// Calls put(i, p) for the positions p that stay of `n` candidates from position `a` on, i = a ... in
// their order.  key: shared memory for n_key of the candidates' keys.  LONG: for thousands of
// positions, with all loads at once, fewer keys in the later rounds and four positions of a block to
// a thread (4 x 2 caches of up to 30,041 -> 16,809 positions: 41 us, 56 without; two of 640 -> 512
// 10.7 us so, 9.6 without, since it is more code that is met cold).
template <bool LONG, typename Put>
__device__ void select_kept(SelectSmem& sm, uint32_t* key, int n_key, const float* acc, int a, int n, int need,
                            Put put) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kPer = LONG ? 4 : 1, kEBlock = kPer * kEThreads;
    const int ns = min(n, n_key), n4 = (ns + 3) >> 2;
    if constexpr (LONG) {
#pragma unroll 4
        for (int p = tid; p < ns; p += kEThreads)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(key + p)), "l"(acc + a + p) : "memory");
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    // the last four are filled up with keys that no threshold of a count is below
#pragma unroll 4
    for (int p = tid; p < 4 * n4; p += kEThreads)
        key[p] = p < ns ? order_key(LONG ? __uint_as_float(key[p]) : acc[a + p]) : 0u;
    __syncthreads();
    uint32_t thr = 0;  // the largest value that at least `need` keys reach
    int reach = n;     // keys that reach it
    int over = 0;      // keys past the values that are still in question, [thr, thr + 2^(bit + 2))
    int m = 0, m_over = 0;                             // LONG: the keys in question once
    uint32_t* few = reinterpret_cast<uint32_t*>(sm.base);  // they are 1024 at most, and `over` then
#pragma unroll 1
    for (int bit = 30, ph = 0; bit >= 0 && reach != need; bit -= 2, ph ^= 1) {
        const uint32_t t1 = thr | 1u << bit, t2 = thr | 2u << bit, t3 = thr | 3u << bit;
        int c1 = 0, c2 = 0, c3 = 0;
        auto add = [&](uint32_t k) {
            c1 += k >= t1;
            c2 += k >= t2;
            c3 += k >= t3;
        };
        if (LONG && m > 0) {
#pragma unroll 1
            for (int p = tid; p < m; p += kEThreads) add(few[p]);
        } else {
#pragma unroll 4
            for (int p = tid; p < n4; p += kEThreads) {
                const uint4 k = reinterpret_cast<const uint4*>(key)[p];
                add(k.x);
                add(k.y);
                add(k.z);
                add(k.w);
            }
#pragma unroll 4
            for (int p = ns + tid; p < n; p += kEThreads) add(order_key(acc[a + p]));
        }
        c1 = __reduce_add_sync(0xffffffffu, c1);
        c2 = __reduce_add_sync(0xffffffffu, c2);
        c3 = __reduce_add_sync(0xffffffffu, c3);
        if (lane == 0) {
            sm.cnt[ph][0][warp] = c1;
            sm.cnt[ph][1][warp] = c2;
            sm.cnt[ph][2][warp] = c3;
        }
        __syncthreads();
        c1 = m_over + __reduce_add_sync(0xffffffffu, lane < kEWarps ? sm.cnt[ph][0][lane] : 0);
        c2 = m_over + __reduce_add_sync(0xffffffffu, lane < kEWarps ? sm.cnt[ph][1][lane] : 0);
        c3 = m_over + __reduce_add_sync(0xffffffffu, lane < kEWarps ? sm.cnt[ph][2][lane] : 0);
        if (c3 >= need) thr = t3, reach = c3;
        else if (c2 >= need) thr = t2, reach = c2, over = c3;
        else if (c1 >= need) thr = t1, reach = c1, over = c2;
        else over = c1;
        if (LONG && m == 0 && n > 4096 && reach - over <= kESeg * kEWarps * 2 && reach != need && bit > 0) {
            const uint32_t width = 1u << bit;  // the keys in question are thr and the width - 1 above it
            if (tid == 0) sm.total[0] = 0;
            __syncthreads();
            auto keep = [&](uint32_t k) {
                if (k - thr < width) few[atomicAdd(&sm.total[0], 1)] = k;  // (k < thr wraps)
            };
#pragma unroll 1
            for (int p = tid; p < ns; p += kEThreads) keep(key[p]);
#pragma unroll 1
            for (int p = ns + tid; p < n; p += kEThreads) keep(order_key(acc[a + p]));
            __syncthreads();
            m = reach - over;
            m_over = over;
        }
    }
    // keys above `top` all stay, and of those equal to it the first need - (their number)
    const bool ties = reach != need;
    const uint32_t top = ties ? thr : thr - 1;  // (thr > 0 when reach == need < n)
    const int take_eq = ties ? need - over : 0;  // (with every bit settled, `over` are above thr)
    // a thread's keys from candidate p on; what is past the end is 0 and not equal
    auto keys = [&](int p, uint32_t (&k)[kPer]) {
        if (LONG && p + 3 < ns) {
            const uint4 v = *reinterpret_cast<const uint4*>(key + p);
            k[0] = v.x, k[1 % kPer] = v.y, k[2 % kPer] = v.z, k[3 % kPer] = v.w;
        } else {
#pragma unroll
            for (int e = 0; e < kPer; ++e) k[e] = p + e < ns ? key[p + e] : p + e < n ? order_key(acc[a + p + e]) : 0u;
        }
    };
    auto count = [&](int p, const uint32_t (&k)[kPer]) {  // larger ones, and 65536 x equal ones
        uint32_t c = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) c += (k[e] > top ? 1u : 0u) + (ties && k[e] == top && p + e < n ? 65536u : 0u);
        return c;
    };
    int out0 = 0, eq0 = 0;  // taken / equal ones in earlier segments
#pragma unroll 1
    for (int p0 = 0; p0 < n; p0 += kESeg * kEBlock) {
        const int blocks = min(kESeg, (n - p0 + kEBlock - 1) / kEBlock);
        __syncthreads();
#pragma unroll 1
        for (int i = 0; i < blocks; ++i) {
            const int p = p0 + i * kEBlock + kPer * tid;
            uint32_t k[kPer];
            keys(p, k);
            const uint32_t c = __reduce_add_sync(0xffffffffu, count(p, k));
            if (lane == 0) {
                sm.base[0][i * kEWarps + warp] = (int)(c & 0xffffu);
                sm.base[1][i * kEWarps + warp] = (int)(c >> 16);
            }
        }
        __syncthreads();
        if (warp < 2) {  // exclusive sums, in the order of the positions: one warp to each
            int run = 0;
#pragma unroll 1
            for (int j0 = 0; j0 < blocks * kEWarps; j0 += 32) {
                const int j = j0 + lane, v = j < blocks * kEWarps ? sm.base[warp][j] : 0;
                int incl = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += x;
                }
                if (j < blocks * kEWarps) sm.base[warp][j] = run + incl - v;
                run += __shfl_sync(0xffffffffu, incl, 31);
            }
            if (lane == 0) sm.total[warp] = run;
        }
        __syncthreads();
#pragma unroll 1
        for (int i = 0; i < blocks; ++i) {
            const int p = p0 + i * kEBlock + kPer * tid;
            uint32_t k[kPer];
            keys(p, k);
            const uint32_t mine = count(p, k);
            uint32_t before = mine;  // of the warp's lanes below this one
            if constexpr (LONG) {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t x = __shfl_up_sync(0xffffffffu, before, o);
                    if (lane >= o) before += x;
                }
                before -= mine;
            } else {
                const uint32_t below = (1u << lane) - 1u;
                before = __popc(__ballot_sync(0xffffffffu, (mine & 1u) != 0) & below) +
                         (__popc(__ballot_sync(0xffffffffu, mine > 1u) & below) << 16);
            }
            int eq = eq0 + sm.base[1][i * kEWarps + warp] + (int)(before >> 16);
            // taken before: every larger key, and the first equal ones
            int out = out0 + sm.base[0][i * kEWarps + warp] + (int)(before & 0xffffu) + min(eq, take_eq) - min(eq0, take_eq);
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const bool same = ties && k[e] == top && p + e < n;
                if (k[e] > top || (same && eq < take_eq)) put(a + out++, a + p + e);
                eq += same;
            }
        }
        out0 += sm.total[0] + min(eq0 + sm.total[1], take_eq) - min(eq0, take_eq);
        eq0 += sm.total[1];
    }
}

// n_key, n_list: keys and kept positions that shared memory holds; with n_list = 0 the list is in P.kept.
template <bool MOVE, bool LONG>
__global__ void __launch_bounds__(kEThreads, 2)
    evict_kernel(const EvictProblem P, const int n_key, const int n_list, const KCtx ctx) {
    extern __shared__ uint32_t dyn[];  // [n_key] keys, [n_list] kept positions, SelectSmem
    SelectSmem& sm = *reinterpret_cast<SelectSmem*>(dyn + n_key + (MOVE ? n_list : 0));
    if (!MOVE || P.kv_len == P.kv_len_out) griddep_launch();  // this call's second kernel
    griddep_wait();
    task_begin(ctx);
    const int tid = threadIdx.x;
    const int part = blockIdx.x, kvh = blockIdx.y, t = blockIdx.z, pair = t * P.nkv + kvh;
    const int L = P.kv_len[t];
    const bool bad = L < 0 || L > P.cap;
    const int count = bad ? -1 : min(L, P.budget);
    // (the pair's CTAs write the same)
    int* kept = MOVE && n_list ? reinterpret_cast<int*>(dyn) + n_key : P.kept + (size_t)pair * P.budget;
    int* user = P.user_kept && part == 0 ? P.user_kept + (size_t)pair * P.budget : nullptr;
    if (kvh == 0 && part == 0 && tid == 0) {
        if (bad) report(ctx, ST_BOUNDS, (uint32_t)L);
        // the other CTAs still read kv_len: where it is written too, a later kernel does that
        if (!MOVE || P.kv_len_out == P.kv_len) P.count[t] = count;
        else if (!bad) P.kv_len_out[t] = count;
    }
    if (user)
        for (int i = max(0, count) + tid; i < P.budget; i += kEThreads) user[i] = -1;
    auto put = [&](int i, int p) {
        kept[i] = p;
        if (user) user[i] = p;
    };
    if (!bad) {
        const bool some = L > P.budget;
        const int a = some ? P.n_sink : L, need = some ? P.budget - P.n_recent - a : 0;
        for (int i = tid; i < a; i += kEThreads) put(i, i);
        if (some)
            for (int i = tid; i < P.n_recent; i += kEThreads) put(a + need + i, L - P.n_recent + i);
        // need < candidates: L is past the budget
        if (need > 0)
            select_kept<LONG>(sm, dyn, n_key, P.acc + (size_t)pair * P.cap, a, L - P.n_recent - a, need, put);
    }
    __syncthreads();
    if (MOVE && !bad) {
        const int parts = gridDim.x;
        const int r0 = (int)((long long)part * count / parts), r1 = (int)((long long)(part + 1) * count / parts);
        const size_t so = (size_t)pair * P.cap, to = (size_t)pair * P.cap_out;
        // acc first: its few loads are under way while the rows' begin
        for (int r = r0 + tid; r < r1; r += kEThreads) P.acc_out[to + r] = P.acc[so + kept[r]];
        const int c = tid & 3;  // 32-byte column of a row
        constexpr int kRows = kEThreads / 4;
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
            const uint4* src = reinterpret_cast<const uint4*>(w ? P.v : P.k) + so * 8 + 2 * c;
            uint4* dst = reinterpret_cast<uint4*>(w ? P.v_out : P.k_out) + to * 8 + 2 * c;
#pragma unroll 1
            for (int r = r0 + (tid >> 2); r < r1; r += kRows * kEUnroll) {
                uint4 v[kEUnroll][2];
#pragma unroll
                for (int u = 0; u < kEUnroll; ++u)
                    if (r + u * kRows < r1) load_once(src + (size_t)kept[r + u * kRows] * 8, v[u][0], v[u][1]);
#pragma unroll
                for (int u = 0; u < kEUnroll; ++u)
                    if (r + u * kRows < r1) store_once(dst + (size_t)(r + u * kRows) * 8, v[u][0], v[u][1]);
            }
        }
        // a new position starts at 0
        for (int r = count + part * kEThreads + tid; r < P.cap_out; r += parts * kEThreads) P.acc_out[to + r] = 0.f;
    }
    task_end(ctx);
}

__global__ void __launch_bounds__(kEThreads) evict_len_kernel(const EvictProblem P, const KCtx ctx) {
    griddep_wait();
    task_begin(ctx);
    for (int t = threadIdx.x; t < P.T; t += kEThreads)
        if (P.count[t] >= 0) P.kv_len_out[t] = P.count[t];
    task_end(ctx);
}

// The move in place: a row only ever moves down (kept[i] >= i).  The CTAs of a pair share it by
// columns, 64 bytes of every row of K or V each, so that no CTA's stores can reach what another has
// still to load; a CTA loads a run of rows, waits, and stores it, and run r's stores end below run
// r + 1's sources.  One more CTA moves acc and clears it behind the kept rows.
// Selection and move together: 64 sequences x 8 KV heads of up to 8192 positions, those past 4096 cut
// to them, 492 MB, 110 us (4.5 TB/s); 4 x 8 of 9000 -> 4500 34 us, 2 x 8 of 640 -> 512 9 us, both
// latency (one CTA selects for a pair, five move it with a barrier to a run).
constexpr int kMThreads = 256;
constexpr int kMUnroll = 8;

__global__ void __launch_bounds__(kMThreads) evict_move_kernel(const EvictProblem P, const KCtx ctx) {
    griddep_wait();
    task_begin(ctx);
    const int tid = threadIdx.x;
    const int kvh = blockIdx.y, t = blockIdx.z, pair = t * P.nkv + kvh;
    const int n = P.count[t];
    const int* kept = P.kept + (size_t)pair * P.budget;
    if (n >= 0 && blockIdx.x == 0) {  // acc, and the new length
        if (kvh == 0 && tid == 0) P.kv_len_out[t] = n;
        float* acc = P.acc_out + (size_t)pair * P.cap_out;
        for (int r0 = 0; r0 < n; r0 += kMThreads * kMUnroll) {
            float v[kMUnroll];
#pragma unroll
            for (int u = 0; u < kMUnroll; ++u) {
                const int r = r0 + u * kMThreads + tid;
                v[u] = r < n ? acc[kept[r]] : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kMUnroll; ++u) {
                const int r = r0 + u * kMThreads + tid;
                if (r < n) acc[r] = v[u];
            }
            __syncthreads();
        }
        for (int r = n + tid; r < P.cap_out; r += kMThreads) acc[r] = 0.f;
    } else if (n > 0) {
        const int s = blockIdx.x - 1, c = (s & 1) * 4 + (tid & 3);
        uint4* x = reinterpret_cast<uint4*>((s >= 2 ? P.v_out : P.k_out)) + (size_t)pair * P.cap_out * 8 + c;
        // rows that stay where they are: kept[r] == r up to the first that moves
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (kept[mid] == mid) lo = mid + 1;
            else hi = mid;
        }
        constexpr int kRun = kMThreads / 4 * kMUnroll;
        for (int r0 = lo; r0 < n; r0 += kRun) {
            uint4 v[kMUnroll];
#pragma unroll
            for (int u = 0; u < kMUnroll; ++u) {
                const int r = r0 + u * (kMThreads / 4) + (tid >> 2);
                if (r < n) v[u] = x[(size_t)kept[r] * 8];
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kMUnroll; ++u) {
                const int r = r0 + u * (kMThreads / 4) + (tid >> 2);
                if (r < n) x[(size_t)r * 8] = v[u];
            }
            __syncthreads();
        }
    }
    task_end(ctx);
}

}  // namespace

int enqueue_weights(Launcher& L, const WeightsProblem& p, const KCtx& c, int sms) {
    void* args[] = {(void*)&p, (void*)&c};
    const void* f = p.G <= 8 ? (const void*)weights_kernel<1> : (const void*)weights_kernel<2>;
    return L.launch(f, dim3(2 * sms), dim3(kWThreads), 0, args, true);
}

int enqueue_evict(Launcher& L, const EvictProblem& p, const KCtx& c) {
    const EvictWords words = evict_words(p.cap, p.budget, (int)sizeof(SelectSmem));
    const int n_key = words.key, n_list = words.list;
    // The selection for long caches, by capacity (lengths are on the device).  Without and with it,
    // half of the positions kept: 32 pairs of (sequence, KV head) of up to 3000 positions 15.7 and
    // 16.1 us, 4000 18.0 and 18.5, 6000 22.3 and 21.3, 9000 30.2 and 26.4, 30,000 112 and 90.  512 pairs
    // of 5000 83 and 82.7, 8192 131 and 130, 9000 140 and 142.7, 12,288 193 and 196, 16,384 342 and 340,
    // 16,384 -> 1000 79 and 70; in place 8192 116 and 110, 16,384 222 and 212.  What it loses most on
    // are short caches with much room: 512 of 600 positions in 16,384 20.4 and 22.5.
    const bool long_ = p.cap > 4096;
    void* args[] = {(void*)&p, (void*)&n_key, (void*)&n_list, (void*)&c};
    void* args2[] = {(void*)&p, (void*)&c};
    if (!p.in_place) {
        // as many CTAs to a pair as give every SM two, at most 16, none with fewer than 64 rows
        const int pairs = p.T * p.nkv, rows = std::min(p.budget, p.cap);
        const int parts = std::max(1, std::min({16, 304 / pairs, rows / 64}));
        const int e = L.launch(long_ ? (const void*)evict_kernel<true, true> : (const void*)evict_kernel<true, false>, dim3(parts, p.nkv, p.T), dim3(kEThreads),
                               (size_t)(n_key + n_list) * 4 + sizeof(SelectSmem), args, true);
        if (e || p.kv_len != p.kv_len_out) return e;
        return L.launch((const void*)evict_len_kernel, dim3(1), dim3(kEThreads), 0, args2, true);
    }
    const int e = L.launch(long_ ? (const void*)evict_kernel<false, true> : (const void*)evict_kernel<false, false>, dim3(1, p.nkv, p.T), dim3(kEThreads),
                           (size_t)n_key * 4 + sizeof(SelectSmem), args, true);
    if (e) return e;
    return L.launch((const void*)evict_move_kernel, dim3(5, p.nkv, p.T), dim3(kMThreads), 0, args2, true);
}

}  // namespace sgp
