// What a bounded KV cache needs beside the attention: the attention weight that each cached
// position gathers, and the eviction that keeps the heaviest positions.
//
//   weights   acc[t][j][p] += sum over the heads h of group j of exp(q_h . k_p / sqrt(d) - lse_h),
//             lse_h the log-sum-exp that the attention returned for head h;
//   eviction  keep the first n_sink and the last n_recent positions and, of the others, the
//             budget - n_sink - n_recent with the largest acc (ties to the lower position, NaN
//             below every number), in their order.
#include <algorithm>

#include "kernels.h"
#include "mma.cuh"

namespace sgp {

namespace {

// ---------------------------------------------------------------------------------------
// Accumulated attention weights.  One pass over K; the scores are S = K q^T on warp-level
// matrix products (M = 16 positions, N = 8 heads, K = 64 dims) with K fragments loaded straight
// from global memory: lane (g, c) loads 16 bytes of rows g and g + 8, and both operands read
// the same permutation of the dims, so each product still sums matching pairs.  An item is 64
// positions of one (sequence, KV head); the warps of the grid share the items in equal runs.
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
                    kf[m][h][0] = src[cq];
                    kf[m][h][1] = src[cq + 4];
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
                        const uint4 v = src[cq + 4 * e];
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
// Eviction, first kernel: which positions stay.  One CTA per (sequence, KV head).  The keys of
// the positions between the sinks and the recent ones (acc mapped to unsigned integers of the
// same order) stay in registers: warp w holds a run of 32 KPT of them, lane by lane.  The
// threshold, the need-th largest key, is found two bits a round from counts; the positions
// above it stay, and of those equal to it the first ones.
// ---------------------------------------------------------------------------------------
constexpr int kEThreads = 1024;
constexpr int kEWarps = kEThreads / 32;

__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 0u;             // NaN: below -inf
    if (v == 0.f) return 0x80000000u;  // -0 = +0
    const uint32_t u = __float_as_uint(v);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

template <int KPT>
__global__ void __launch_bounds__(kEThreads, KPT <= 8 ? 2 : 1)
    evict_select_kernel(const EvictProblem P, const KCtx ctx) {
    __shared__ int cnt[2][3][kEWarps];
    __shared__ int base[2][kEWarps];
    griddep_launch();
    griddep_wait();
    task_begin(ctx);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int kvh = blockIdx.x, t = blockIdx.y, pair = t * P.nkv + kvh;
    const int L = P.kv_len[t];
    const bool bad = L < 0 || L > P.cap || min(L, P.budget) > P.cap_out;
    if (bad && kvh == 0 && tid == 0) report(ctx, ST_BOUNDS, (uint32_t)L);
    const int count = bad ? -1 : min(L, P.budget);
    if (kvh == 0 && tid == 0) P.count[t] = count;
    int* kept = P.kept + (size_t)pair * P.budget;
    int* user = P.user_kept ? P.user_kept + (size_t)pair * P.budget : nullptr;
    auto put = [&](int i, int p) {
        kept[i] = p;
        if (user) user[i] = p;
    };
    if (user)
        for (int i = max(0, count) + tid; i < P.budget; i += kEThreads) user[i] = -1;
    if (!bad && L <= P.budget) {
        for (int i = tid; i < L; i += kEThreads) put(i, i);
    } else if (!bad) {
        const float* acc = P.acc + (size_t)pair * P.cap;
        const int a = P.n_sink, n = L - P.n_recent - a;       // candidates [a, a + n)
        const int need = P.budget - P.n_recent - a;
        for (int i = tid; i < a; i += kEThreads) put(i, i);
        for (int i = tid; i < P.n_recent; i += kEThreads) put(a + need + i, L - P.n_recent + i);
        // runs of 32 KPT kEWarps candidates; more than one only beyond the registers
        constexpr int kRun = 32 * KPT * kEWarps;
        const int runs = (n + kRun - 1) / kRun;
        uint32_t key[KPT];
        auto load = [&](int run) {
#pragma unroll
            for (int i = 0; i < KPT; ++i) {
                const int p = run * kRun + (warp * KPT + i) * 32 + lane;
                // past the end: never counted (a key of 0 is only ever >= the threshold 0)
                key[i] = p < n ? order_key(acc[a + p]) : 0u;
            }
        };
        auto in = [&](int run, int i) { return run * kRun + (warp * KPT + i) * 32 + lane < n; };
        uint32_t thr = 0;  // largest value with at least `need` keys >= it
        if (need > 0) {  // need < n: L is past the budget
            if (runs == 1) load(0);
            for (int bit = 30, ph = 0; bit >= 0; bit -= 2, ph ^= 1) {
                int c[3] = {0, 0, 0};
                for (int run = 0; run < runs; ++run) {
                    if (runs > 1) load(run);
#pragma unroll
                    for (int i = 0; i < KPT; ++i)
#pragma unroll
                        for (int b = 0; b < 3; ++b) c[b] += key[i] >= (thr | ((uint32_t)(b + 1) << bit));
                }
#pragma unroll
                for (int b = 0; b < 3; ++b) {
                    const int s = __reduce_add_sync(0xffffffffu, c[b]);
                    if (lane == 0) cnt[ph][b][warp] = s;
                }
                __syncthreads();
#pragma unroll
                for (int b = 2; b >= 0; --b) {
                    const int s = __reduce_add_sync(0xffffffffu, cnt[ph][b][lane]);
                    if (s >= need) {
                        thr |= (uint32_t)(b + 1) << bit;
                        break;
                    }
                }
            }
        }
        if (need > 0) {
            // keys above the threshold, then how many equal ones are taken
            int c = 0;
            for (int run = 0; run < runs; ++run) {
                if (runs > 1) load(run);
#pragma unroll
                for (int i = 0; i < KPT; ++i) c += key[i] > thr;
            }
            c = __reduce_add_sync(0xffffffffu, c);
            __syncthreads();
            if (lane == 0) cnt[0][0][warp] = c;
            __syncthreads();
            const int above = __reduce_add_sync(0xffffffffu, cnt[0][0][lane]);
            const int ties = need - above;
            int out0 = 0, eq0 = 0;  // taken / equal ones in earlier runs
            for (int run = 0; run < runs; ++run) {
                if (runs > 1) load(run);
                int c_gt = 0, c_eq = 0;
#pragma unroll
                for (int i = 0; i < KPT; ++i) {
                    const bool x = in(run, i);
                    c_gt += __popc(__ballot_sync(0xffffffffu, x && key[i] > thr));
                    c_eq += __popc(__ballot_sync(0xffffffffu, x && key[i] == thr));
                }
                __syncthreads();
                if (lane == 0) {
                    base[0][warp] = c_gt;
                    base[1][warp] = c_eq;
                }
                __syncthreads();
                int gt = base[0][lane], eq = base[1][lane];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int vg = __shfl_up_sync(0xffffffffu, gt, o), ve = __shfl_up_sync(0xffffffffu, eq, o);
                    if (lane >= o) {
                        gt += vg;
                        eq += ve;
                    }
                }
                const int run_gt = __shfl_sync(0xffffffffu, gt, 31), run_eq = __shfl_sync(0xffffffffu, eq, 31);
                int my_gt = __shfl_sync(0xffffffffu, gt, warp) - c_gt;
                int my_eq = eq0 + __shfl_sync(0xffffffffu, eq, warp) - c_eq;
                // taken before this warp's run: every larger key, and the first `ties` equal ones
                int out = out0 + my_gt + min(my_eq, ties) - min(eq0, ties);
#pragma unroll
                for (int i = 0; i < KPT; ++i) {
                    const bool x = in(run, i);
                    const bool is_eq = x && key[i] == thr;
                    const uint32_t meq = __ballot_sync(0xffffffffu, is_eq);
                    const uint32_t below = (1u << lane) - 1u;
                    const bool take = x && (key[i] > thr || (is_eq && my_eq + __popc(meq & below) < ties));
                    const uint32_t mt = __ballot_sync(0xffffffffu, take);
                    if (take) put(a + out + __popc(mt & below), a + run * kRun + (warp * KPT + i) * 32 + lane);
                    out += __popc(mt);
                    my_eq += __popc(meq);
                }
                out0 += run_gt + min(eq0 + run_eq, ties) - min(eq0, ties);
                eq0 += run_eq;
            }
        }
    }
    task_end(ctx);
}

// ---------------------------------------------------------------------------------------
// Eviction, second kernel: the rows move.  Out of place a CTA copies a run of kept rows.  In
// place (a row only ever moves down: kept[i] >= i) the CTAs of a pair share it by columns, 64
// bytes of every row of K or V each, so that no CTA's stores can reach what another has still
// to load; a CTA loads a run of rows, waits, and stores it, and run r's stores end below run
// r + 1's sources.  One more CTA moves acc and clears it behind the kept rows.
// ---------------------------------------------------------------------------------------
constexpr int kMThreads = 256;
constexpr int kMUnroll = 8;
constexpr int kMRows = 256;  // out of place: kept rows per CTA

__global__ void __launch_bounds__(kMThreads) evict_move_kernel(const EvictProblem P, const KCtx ctx) {
    griddep_wait();
    task_begin(ctx);
    const int tid = threadIdx.x;
    const int kvh = blockIdx.y, t = blockIdx.z, pair = t * P.nkv + kvh;
    const int n = P.count[t];
    const int* kept = P.kept + (size_t)pair * P.budget;
    if (n >= 0 && blockIdx.x == 0) {  // acc, and the new length
        if (kvh == 0 && tid == 0) P.kv_len_out[t] = n;
        const float* src = P.acc + (size_t)pair * P.cap;
        float* dst = P.acc_out + (size_t)pair * P.cap_out;
        for (int r0 = 0; r0 < n; r0 += kMThreads * kMUnroll) {
            float v[kMUnroll];
#pragma unroll
            for (int u = 0; u < kMUnroll; ++u) {
                const int r = r0 + u * kMThreads + tid;
                v[u] = r < n ? src[kept[r]] : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kMUnroll; ++u) {
                const int r = r0 + u * kMThreads + tid;
                if (r < n) dst[r] = v[u];
            }
            __syncthreads();
        }
        for (int r = n + tid; r < P.cap_out; r += kMThreads) dst[r] = 0.f;
    } else if (n > 0) {
        const size_t so = (size_t)pair * P.cap * 64, to = (size_t)pair * P.cap_out * 64;
        if (!P.in_place) {
            const int r0 = (blockIdx.x - 1) * kMRows, m = min(n - r0, kMRows);
            const int c = tid & 7;  // 16-byte column of a row
            for (int w = 0; w < 2; ++w) {
                const uint4* src = reinterpret_cast<const uint4*>((w ? P.v : P.k) + so) + c;
                uint4* dst = reinterpret_cast<uint4*>((w ? P.v_out : P.k_out) + to) + c;
                uint4 v[kMUnroll];
                static_assert(kMRows == kMThreads / 8 * kMUnroll, "one pass");
#pragma unroll
                for (int u = 0; u < kMUnroll; ++u) {
                    const int r = u * (kMThreads / 8) + (tid >> 3);
                    if (r < m) v[u] = src[(size_t)kept[r0 + r] * 8];
                }
#pragma unroll
                for (int u = 0; u < kMUnroll; ++u) {
                    const int r = u * (kMThreads / 8) + (tid >> 3);
                    if (r < m) dst[(size_t)(r0 + r) * 8] = v[u];
                }
            }
        } else {
            const int s = blockIdx.x - 1, c = (s & 1) * 4 + (tid & 3);
            uint4* x = reinterpret_cast<uint4*>((s >= 2 ? P.v_out : P.k_out) + to) + c;
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
    }
    task_end(ctx);
}

}  // namespace

int enqueue_weights(Launcher& L, const WeightsProblem& p, const KCtx& c, int sms) {
    void* args[] = {(void*)&p, (void*)&c};
    const void* f = p.G <= 8 ? (const void*)weights_kernel<1> : (const void*)weights_kernel<2>;
    return L.launch(f, dim3(2 * sms), dim3(kWThreads), 0, args);
}

int enqueue_evict(Launcher& L, const EvictProblem& p, const KCtx& c) {
    void* args[] = {(void*)&p, (void*)&c};
    const void* f = p.cap <= 8 * kEThreads ? (const void*)evict_select_kernel<8>
                                           : (const void*)evict_select_kernel<32>;
    const int e = L.launch(f, dim3(p.nkv, p.T), dim3(kEThreads), 0, args);
    if (e) return e;
    const int rows = std::min(p.budget, p.cap);
    const int parts = p.in_place ? 4 : (rows + kMRows - 1) / kMRows;
    return L.launch((const void*)evict_move_kernel, dim3(1 + parts, p.nkv, p.T), dim3(kMThreads), 0, args,
                    true);
}

}  // namespace sgp
