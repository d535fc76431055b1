// Low-rank adapters of many requests beside a shared projection:
//   y_out[t] = y_in[t] + scale_a B_a (A_a x[t]),   a = adapter_of[t]  (-1: y_out = y_in).
//
// One launch.  Sequences with the same adapter form a group, cut into tiles of 16; a cluster of
// eight CTAs takes a tile.  First product: the 64 warps of the cluster split the input features,
// M = 16 sequences, N = 8 ranks, fragments straight from global memory (both operands read the
// same permutation of the features, so that every lane loads 16 bytes); the warps' sums join in
// shared memory, the CTAs' in distributed shared memory, both in a fixed order.  Second product:
// the warps split the output features.  The intermediate A x is kept as the sum of two bf16 (16
// bits of mantissa), so that it loses nothing against y's own rounding.
// Each adapter's A and B are read once per tile; with few sequences per adapter they are what
// bounds the kernel, with one adapter it is x and y.
#include <algorithm>

#include "kernels.h"
#include "mma.cuh"

namespace sgp {

namespace {

constexpr int kLThreads = 256;
constexpr int kLWarps = kLThreads / 32;
constexpr int kLCluster = 8;
constexpr int kLTile = 16;
constexpr int kLMaxT = 512;
constexpr int kLClusters = 64;  // at most, per launch

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float dsmem_ld(const float* p, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

__host__ __device__ inline int lora_rank_pad(int r) { return (r + 15) & ~15; }
inline size_t lora_smem_bytes(int n, int r) {
    const size_t rp = lora_rank_pad(r);
    return (size_t)(kLWarps + 1) * kLTile * rp * 4   // warps' sums, the CTA's sum
           + 2 * kLTile * (rp + 8) * 2               // A x as two bf16
           + (3 * kLMaxT + kLTile + n + 1) * 4;
}

// RP: rank, rounded up to 16, at most
template <int RP>
__global__ void __cluster_dims__(kLCluster, 1, 1) __launch_bounds__(kLThreads)
    lora_kernel(const LoraProblem P, const KCtx ctx) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    constexpr int kNT = RP / 8, kKS = RP / 16;
    const int rp = lora_rank_pad(P.max_rank);
    float* red = reinterpret_cast<float*>(smem_raw);         // [warps][16][rp]
    float* part = red + kLWarps * kLTile * rp;               // [16][rp]
    bf16* hi = reinterpret_cast<bf16*>(part + kLTile * rp);  // [16][rp + 8]
    bf16* lo = hi + kLTile * (rp + 8);
    int* adp = reinterpret_cast<int*>(lo + kLTile * (rp + 8));  // [T] adapter, n: none
    int* rnk = adp + kLMaxT;                                 // [T] place in the group
    int* lead = rnk + kLMaxT;                                // [units] first sequence of a tile
    int* tok = lead + kLMaxT;                                // [16]
    int* cnt = tok + kLTile;                                 // [n + 1]
    __shared__ int n_units;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cq = lane & 3;
    const uint32_t cr = cluster_rank();
    const int cluster = blockIdx.x / kLCluster, clusters = gridDim.x / kLCluster;
    griddep_wait();
    task_begin(ctx);

    for (int i = tid; i <= P.n; i += kLThreads) cnt[i] = 0;
    for (int t = tid; t < P.T; t += kLThreads) {
        int a = P.adapter_of[t];
        if (a >= P.n && blockIdx.x == 0) report(ctx, ST_BOUNDS, (uint32_t)a);
        adp[t] = a >= 0 && a < P.n ? a : P.n;
    }
    __syncthreads();
    if (warp == 0) {
        int units = 0;
        for (int t0 = 0; t0 < P.T; t0 += 32) {
            const int t = t0 + lane;
            const int a = t < P.T ? adp[t] : -1;
            const uint32_t same = __match_any_sync(0xffffffffu, a), below = (1u << lane) - 1u;
            const int had = a >= 0 ? cnt[a] : 0, r = had + __popc(same & below);
            __syncwarp();
            if (a >= 0) {
                rnk[t] = r;
                if ((same & below) == 0) cnt[a] = had + __popc(same);
            }
            const bool first = a >= 0 && r % kLTile == 0;
            const uint32_t m = __ballot_sync(0xffffffffu, first);
            if (first) lead[units + __popc(m & below)] = t;
            units += __popc(m);
            __syncwarp();
        }
        if (lane == 0) n_units = units;
    }
    __syncthreads();

    const int gw = (int)cr * kLWarps + warp;  // warp of the cluster
    const int k_blocks = P.in >> 5, o_blocks = P.out >> 5;
    const int kb0 = gw * k_blocks / (kLCluster * kLWarps), kb1 = (gw + 1) * k_blocks / (kLCluster * kLWarps);
    const int ob0 = gw * o_blocks / (kLCluster * kLWarps), ob1 = (gw + 1) * o_blocks / (kLCluster * kLWarps);
    for (int u = cluster; u < n_units; u += clusters) {
        const int a = adp[lead[u]], tile = rnk[lead[u]] / kLTile;
        const int m = min(kLTile, cnt[a] - tile * kLTile);
        for (int t = tid; t < P.T; t += kLThreads)
            if (adp[t] == a && rnk[t] / kLTile == tile) tok[rnk[t] % kLTile] = t;
        __syncthreads();
        const int t_lo = tok[g < m ? g : 0], t_hi = tok[g + 8 < m ? g + 8 : 0];
        int rank = 0;
        if (a < P.n) {
            rank = P.rank ? P.rank[a] : P.max_rank;
            if (rank < 0 || rank > P.max_rank) {
                if (cr == 0 && tid == 0) report(ctx, ST_BOUNDS, (uint32_t)rank);
                rank = 0;
            }
        }
        if (rank == 0) {  // no adapter: the rows pass through
            if (P.y_out != P.y_in)
                for (int i = 0; i < m; ++i) {
                    const uint4* src = reinterpret_cast<const uint4*>(P.y_in + (size_t)tok[i] * P.ld_y_in);
                    uint4* dst = reinterpret_cast<uint4*>(P.y_out + (size_t)tok[i] * P.ld_y_out);
                    for (int v = (int)cr * kLThreads + tid; v < P.out / 8; v += kLCluster * kLThreads)
                        dst[v] = src[v];
                }
            __syncthreads();  // tok is free
            continue;
        }

        // ---- A x: this warp's input features ----
        float acc[kNT][4];
#pragma unroll
        for (int j = 0; j < kNT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
        const bf16* A = P.a + (size_t)a * P.max_rank * P.in;
        const uint4 z = make_uint4(0, 0, 0, 0);
        for (int kb = kb0; kb < kb1; ++kb) {
            const int k = kb * 32 + cq * 8;
            const uint4 x0 = g < m ? *reinterpret_cast<const uint4*>(P.x + (size_t)t_lo * P.ld_x + k) : z;
            const uint4 x1 = g + 8 < m ? *reinterpret_cast<const uint4*>(P.x + (size_t)t_hi * P.ld_x + k) : z;
            uint4 w[kNT];
#pragma unroll
            for (int j = 0; j < kNT; ++j)
                w[j] = j * 8 + g < rank ? *reinterpret_cast<const uint4*>(A + (size_t)(j * 8 + g) * P.in + k) : z;
            const uint32_t f0[4] = {x0.x, x1.x, x0.y, x1.y}, f1[4] = {x0.z, x1.z, x0.w, x1.w};
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
                mma16816(acc[j], f0, w[j].x, w[j].y);
                mma16816(acc[j], f1, w[j].z, w[j].w);
            }
        }
#pragma unroll
        for (int j = 0; j < kNT; ++j)
            if (j * 8 < rp) {
                float* r = red + (size_t)warp * kLTile * rp + j * 8 + 2 * cq;
                *reinterpret_cast<float2*>(r + g * rp) = make_float2(acc[j][0], acc[j][1]);
                *reinterpret_cast<float2*>(r + (g + 8) * rp) = make_float2(acc[j][2], acc[j][3]);
            }
        __syncthreads();
        for (int i = tid; i < kLTile * rp; i += kLThreads) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kLWarps; ++w) s += red[(size_t)w * kLTile * rp + i];
            part[i] = s;
        }
        cluster_sync();
        const float scale = P.scale ? P.scale[a] : 1.f;
        for (int i = tid; i < kLTile * rp; i += kLThreads) {
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < kLCluster; ++c) s += dsmem_ld(part + i, c);
            s *= scale;
            const bf16 h = __float2bfloat16_rn(s);
            const int at = (i / rp) * (rp + 8) + i % rp;
            hi[at] = h;
            lo[at] = __float2bfloat16_rn(s - __bfloat162float(h));
        }
        cluster_sync();  // every CTA has read the others' sums (and hi, lo are complete)

        // ---- y += B (A x): this warp's output features, 32 at a time ----
        const bf16* B = P.b + (size_t)a * P.out * P.max_rank;
        for (int ob = ob0; ob < ob1; ++ob) {
            float d[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.f;
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
                const int k = ks * 16 + cq * 4;
                if (ks * 16 >= rank) break;
                uint2 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // column 2c of tile j is feature 8c + 2j: a lane's outputs are neighbours
                    const int f = ob * 32 + (g >> 1) * 8 + j * 2 + (g & 1);
                    w[j] = k < rank ? *reinterpret_cast<const uint2*>(B + (size_t)f * P.max_rank + k)
                                    : make_uint2(0, 0);
                    // what lies behind the rank is not the adapter's
                    if (k + 1 >= rank) w[j].x &= 0xffffu;
                    if (k + 2 >= rank) w[j].y = 0u;
                    else if (k + 3 >= rank) w[j].y &= 0xffffu;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const bf16* v = e ? lo : hi;
                    const uint2 v0 = *reinterpret_cast<const uint2*>(v + g * (rp + 8) + k);
                    const uint2 v1 = *reinterpret_cast<const uint2*>(v + (g + 8) * (rp + 8) + k);
                    const uint32_t f[4] = {v0.x, v1.x, v0.y, v1.y};
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma16816(d[j], f, w[j].x, w[j].y);
                }
            }
            const int f0 = ob * 32 + cq * 8;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (g + 8 * h >= m) continue;
                const size_t t = h ? t_hi : t_lo;
                float y[8];
                unpack8(*reinterpret_cast<const uint4*>(P.y_in + t * P.ld_y_in + f0), y);
                uint4 o;
                o.x = pack_bf16x2(y[0] + d[0][2 * h], y[1] + d[0][2 * h + 1]);
                o.y = pack_bf16x2(y[2] + d[1][2 * h], y[3] + d[1][2 * h + 1]);
                o.z = pack_bf16x2(y[4] + d[2][2 * h], y[5] + d[2][2 * h + 1]);
                o.w = pack_bf16x2(y[6] + d[3][2 * h], y[7] + d[3][2 * h + 1]);
                *reinterpret_cast<uint4*>(P.y_out + t * P.ld_y_out + f0) = o;
            }
        }
        __syncthreads();  // hi, lo and tok are free
    }
    task_end(ctx);
}

}  // namespace

int enqueue_lora(Launcher& L, const LoraProblem& p, const KCtx& c) {
    void* args[] = {(void*)&p, (void*)&c};
    const int rp = lora_rank_pad(p.max_rank);
    const void* f = rp <= 16   ? (const void*)lora_kernel<16>
                    : rp <= 32 ? (const void*)lora_kernel<32>
                    : rp <= 64 ? (const void*)lora_kernel<64>
                               : (const void*)lora_kernel<128>;
    // tiles at most: one of every sequence, or a started one per adapter and "none" beside full ones
    const int tiles = std::min(p.T, p.n + 1 + p.T / kLTile);
    return L.launch(f, dim3(kLCluster * std::min(tiles, kLClusters)), dim3(kLThreads),
                    lora_smem_bytes(p.n, p.max_rank), args);
}

}  // namespace sgp
