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

constexpr int kPThreads = 512;
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
    int low[kPrefixMax];         // least visible position
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

// The simplest form: 16 warps of 16 rows, warp-level matrix products, two stages of keys.
__global__ void __launch_bounds__(kPThreads, 1)
    prefix_attn_kernel(const __grid_constant__ PrefixProblem P, const KCtx ctx) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + 4 * kPHalf);
    Plan& pl = *reinterpret_cast<Plan*>(full + 2);
    __shared__ int sh_err;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cq = lane & 3;
    griddep_launch();
    if (tid == 0) {
        mbar_init(&full[0], 1);
        mbar_init(&full[1], 1);
        fence_barrier_init();
        sh_err = 0;
    }
    task_begin(ctx);
    build_plan(pl, P, ctx);
    const int n = P.prefix.n, total = pl.step0[n];
    const int shares = min(kPrefixShares, total);  // none of them empty
    const int b = blockIdx.x;
    const int x0 = b < shares ? (int)((long long)b * total / shares) : 0;
    const int x1 = b < shares ? (int)((long long)(b + 1) * total / shares) : 0;
    const uint64_t pol = policy_evict_last();
    auto issue = [&](int x, int stage) {
        const Step s = step_at(pl, n, x);
        const int row = (s.g * P.nkv + s.kvh) * P.prefix.cap + (pl.first[s.g] + s.k) * kPrefixKeys;
        uint8_t* dst = smem + stage * 2 * kPHalf;
        mbar_arrive_expect_tx(&full[stage], 2 * kPHalf);
        tma_load_2d(dst, &P.tmK, &full[stage], 0, row, pol);
        tma_load_2d(dst + kPHalf, &P.tmV, &full[stage], 0, row, pol);
    };
    if (tid == 0 && x0 < x1) issue(x0, 0);
    uint32_t it = 0;
    bool ok = true;
    for (int x = x0; x < x1 && ok;) {
        const Step s = step_at(pl, n, x);
        const int end = min(x1, x + pl.steps[s.g] - s.k);
        const int seq0 = pl.base[s.g] + s.tile * P.tile_seqs;
        const int rows = min(P.tile_seqs, pl.base[s.g + 1] - seq0) * P.G;
        const int len = pl.len[s.g];
        const bool active = warp * 16 < rows;
        // query rows of this lane (g and g + 8 of the warp's 16) and their least positions
        uint32_t qf[4][4];
        int low[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = warp * 16 + g + 8 * h;
            const bool has = r < rows;
            const int t = has ? pl.mem[seq0 + r / P.G] : 0;
            const bf16* q = P.q + (size_t)t * P.nq * 64 + (size_t)(s.kvh * P.G + (has ? r % P.G : 0)) * 64;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                qf[kk][h] = has ? *reinterpret_cast<const uint32_t*>(q + kk * 16 + 2 * cq) : 0u;
                qf[kk][2 + h] = has ? *reinterpret_cast<const uint32_t*>(q + kk * 16 + 2 * cq + 8) : 0u;
            }
            if (has && P.window > 0) {
                const int own = P.kv_len[t];
                low[h] = max(0, len + (own >= 0 && own <= P.kv_cap ? own : 0) - P.window);
            }
        }
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[8][4];
#pragma unroll
        for (int d = 0; d < 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
        int k = s.k;
        for (; x < end; ++x, ++k, ++it) {
            const int stage = it & 1;
            if (tid == 0 && x + 1 < x1) issue(x + 1, stage ^ 1);
            if (!mbar_wait(&full[stage], (it >> 1) & 1u, ctx.timeout_ns)) {
                if (lane == 0) report(ctx, ST_TIMEOUT, 20);
                sh_err = 1;
            }
            uint8_t* ks = smem + stage * 2 * kPHalf;
            const int pos0 = (pl.first[s.g] + k) * kPrefixKeys;
            const int valid = min(kPrefixKeys, len - pos0);
            if (valid < kPrefixKeys) {  // what lies behind the prefix is arbitrary: P is 0 there
                uint4* v4 = reinterpret_cast<uint4*>(ks + kPHalf);
                for (int e = valid * 8 + tid; e < kPrefixKeys * 8; e += kPThreads)
                    v4[e] = make_uint4(0, 0, 0, 0);
                fence_proxy_async();
            }
            __syncthreads();
            if (sh_err) {
                ok = false;
                ++it;
                break;
            }
            const uint32_t ka = smem_u32(ks), va = ka + kPHalf;
            if (active) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float sc[8][4];
#pragma unroll
                    for (int j = 0; j < 8; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t bf[4];
                            const int mi = lane >> 3;
                            ldsm_x4(ka + sw128(half * 64 + j * 16 + (mi >> 1) * 8 + (lane & 7),
                                               kk * 2 + (mi & 1)), bf);
                            mma16816(sc[2 * j], qf[kk], bf[0], bf[1]);
                            mma16816(sc[2 * j + 1], qf[kk], bf[2], bf[3]);
                        }
                    }
                    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int at = half * 64 + j * 8 + 2 * cq + (e & 1);
                            float v = sc[j][e] * P.scale_log2;
                            if (at >= valid || pos0 + at < low[e >> 1]) v = -INFINITY;
                            sc[j][e] = v;
                            mx[e >> 1] = fmaxf(mx[e >> 1], v);
                        }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                        const float nm = fmaxf(m[h], mx[h]);
                        const float c = m[h] == -INFINITY ? 0.f : exp2f(m[h] - nm);
                        m[h] = nm;
                        l[h] *= c;
#pragma unroll
                        for (int d = 0; d < 8; ++d) {
                            o[d][2 * h] *= c;
                            o[d][2 * h + 1] *= c;
                        }
                        // a row that has seen nothing yet: every score is -inf, every weight 0
                        const float sub = nm == -INFINITY ? 0.f : nm;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float w = exp2f(sc[j][2 * h + e] - sub);
                                sc[j][2 * h + e] = w;
                                l[h] += w;
                            }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t a[4] = {pack_bf16x2(sc[2 * j][0], sc[2 * j][1]),
                                               pack_bf16x2(sc[2 * j][2], sc[2 * j][3]),
                                               pack_bf16x2(sc[2 * j + 1][0], sc[2 * j + 1][1]),
                                               pack_bf16x2(sc[2 * j + 1][2], sc[2 * j + 1][3])};
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            uint32_t bf[4];
                            const int mi = lane >> 3;
                            ldsm_x4_t(va + sw128(half * 64 + j * 16 + (mi & 1) * 8 + (lane & 7),
                                                 2 * d + (mi >> 1)), bf);
                            mma16816(o[2 * d], a, bf[0], bf[1]);
                            mma16816(o[2 * d + 1], a, bf[2], bf[3]);
                        }
                    }
                }
            }
            __syncthreads();
        }
        if (!ok) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            const int r = warp * 16 + g + 8 * h;
            if (r >= rows) continue;
            const size_t slot = b + (size_t)(pl.tile0[s.g] + s.kvh * pl.tiles[s.g] + s.tile);
            const size_t at = slot * kPrefixRows + r;
            if (cq == 0) *reinterpret_cast<float2*>(P.part_ml + at * 2) = make_float2(m[h], l[h]);
#pragma unroll
            for (int d = 0; d < 8; ++d)
                *reinterpret_cast<float2*>(P.part_acc + at * 64 + d * 8 + 2 * cq) =
                    make_float2(o[d][2 * h], o[d][2 * h + 1]);
        }
    }
    // the load after the last one waited for, if the loop gave up
    if (!ok && tid == 0 && it > 0) (void)mbar_wait(&full[it & 1], (it >> 1) & 1u, 10000000ull);
    // the merge waits for this kernel: the own caches' kernel before it must be complete too
    griddep_wait();
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
    const size_t smem = 1024 + 4 * kPHalf + 2 * 8 + sizeof(Plan);
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
