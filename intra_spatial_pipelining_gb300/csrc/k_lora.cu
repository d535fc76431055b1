// Low-rank adapters of many requests beside a shared projection:
//   y_out[t] = y_in[t] + scale_a B_a (A_a x[t]),   a = adapter_of[t]  (-1: y_out = y_in).
//
// One launch.  Sequences with the same adapter form a group, cut into tiles of 16; a cluster of
// eight CTAs takes a tile.  First product: the 64 warps of the cluster split the input features,
// M = 16 sequences, N = 8 ranks, fragments straight from global memory (both operands read the
// same permutation of the features, so that every lane loads 16 bytes); the warps' sums join in
// shared memory, the CTAs' in distributed shared memory, both in a fixed order (stored into every
// other CTA instead of loaded from there, the sums came 1 us later).  Second product:
// the warps split the output features.  The intermediate A x is kept as the sum of two bf16 (16
// bits of mantissa), so that it loses nothing against y's own rounding.
// Each adapter's A and B are read once per tile; with few sequences per adapter they are most of the
// bytes, with one adapter x and y are.
//
// Bound by the chain of dependent steps, not by bytes: 64 sequences of 24 adapters of rank 64, 4096
// -> 2880, 16.4 MB, 10.4 us (1.6 TB/s), of which a launch is 2, the list of tiles 2.5, A x 2.5, its
// join through distributed shared memory 1.5 and the second product 2; one sequence, rank 16, 4.6
// us.  A cluster to a tile, not a kernel to a product: a second launch costs more than the join.
#include <algorithm>

#include "serving.cuh"

namespace sgp {

namespace {

constexpr int kLThreads = 256;
constexpr int kLWarps = kLThreads / 32;
constexpr int kLCluster = 8;
constexpr int kLTile = 16;
constexpr int kLMaxT = 512;
constexpr int kLBlocks = kLMaxT / 32;
constexpr int kLClusters = 64;  // at most, per launch

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 dsmem_ld(uint32_t p, uint32_t rank) {
    uint32_t a;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(p), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ void add4(float4& a, const float4& b) {
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
}

__host__ __device__ inline int lora_rank_pad(int r) { return (r + 15) & ~15; }
inline size_t lora_smem_bytes(int n, int r) {
    const size_t rp = lora_rank_pad(r);
    return (size_t)(kLWarps / (rp <= 32 ? 1 : rp <= 64 ? 2 : 4) + 1) * kLTile * rp * 4  // warps' sums, the CTA's sum
           + 2 * kLTile * (rp + 8) * 2               // A x as two bf16
           + (4 * kLMaxT + kLTile + kLBlocks + n + 1) * 4 + kLBlocks * kLMaxT;
}

// RP: rank, rounded up to 16, at most
template <int RP>
__global__ void __cluster_dims__(kLCluster, 1, 1) __launch_bounds__(kLThreads, RP <= 64 ? 2 : 1)
    lora_kernel(const LoraProblem P, const KCtx ctx) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    // a warp takes 32 ranks at most: more of them share its input features between warps, so that
    // the next block's loads can be in flight during the products (64 ranks to a warp spilled)
    constexpr int kRG = RP <= 32 ? 1 : RP / 32, kKW = kLWarps / kRG;
    constexpr int kNT = (RP <= 32 ? RP : 32) / 8, kKS = RP / 16;
    const int rp = lora_rank_pad(P.max_rank);
    float* red = reinterpret_cast<float*>(smem_raw);         // [kKW warps][16][rp]
    float* part = red + kKW * kLTile * rp;                   // [16][rp]
    bf16* hi = reinterpret_cast<bf16*>(part + kLTile * rp);  // [16][rp + 8]
    bf16* lo = hi + kLTile * (rp + 8);
    int* adp = reinterpret_cast<int*>(lo + kLTile * (rp + 8));  // [T] adapter, n: none
    int* key = adp + kLMaxT;                                 // [T] first sequence with the adapter
    int* rnk = key + kLMaxT;                                 // [T] place in the group
    int* lead = rnk + kLMaxT;                                // [units] first sequence of a tile
    int* tok = lead + kLMaxT;                                // [16]
    int* leads = tok + kLTile;                               // [blocks] tiles that begin in a block
    int* first = leads + kLBlocks;                           // [n + 1] first sequence with an adapter
    uint8_t* count = reinterpret_cast<uint8_t*>(first + P.n + 1);  // [blocks][T] sequences by key
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cq = lane & 3;
    const uint32_t cr = cluster_rank();
    const int cluster = blockIdx.x / kLCluster, clusters = gridDim.x / kLCluster;
    const int blocks = (P.T + 31) >> 5;

    // The tiles.  Every CTA makes the same list, sequences in blocks of 32, a warp to a block: the
    // blocks' counts by group are added up by whoever needs them.
#pragma unroll 1
    for (int i = tid; i <= P.n; i += kLThreads) first[i] = kLMaxT;
#pragma unroll 1
    for (int i = tid; i < blocks * kLMaxT / 4; i += kLThreads) reinterpret_cast<uint32_t*>(count)[i] = 0;
    griddep_wait();  // what is above may run beside the kernel before
    task_begin(ctx);
    __syncthreads();
#pragma unroll 1
    for (int t = tid; t < P.T; t += kLThreads) {
        int a = P.adapter_of[t];
        if (a >= P.n && blockIdx.x == 0) report(ctx, ST_BOUNDS, (uint32_t)a);
        a = a >= 0 && a < P.n ? a : P.n;
        adp[t] = a;
        atomicMin(&first[a], t);
    }
    __syncthreads();
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll 1
    for (int t = tid; t < blocks * 32; t += kLThreads) {
        const int k = t < P.T ? first[adp[t]] : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, k);
        if (k >= 0) {
            key[t] = k;
            rnk[t] = __popc(same & below);
            if ((same & below) == 0) count[(t >> 5) * kLMaxT + k] = (uint8_t)__popc(same);
        }
    }
    __syncthreads();
    uint32_t starts[kLMaxT / kLThreads];  // tiles that begin in this warp's blocks
#pragma unroll
    for (int i = 0; i < kLMaxT / kLThreads; ++i) {
        const int t = i * kLThreads + tid;
        int r = 1;
        if (t < P.T) {
            r = rnk[t];
#pragma unroll 1
            for (int b = 0; b < (t >> 5); ++b) r += count[b * kLMaxT + key[t]];
            rnk[t] = r;
        }
        starts[i] = __ballot_sync(0xffffffffu, t < P.T && r % kLTile == 0);
        if (lane == 0) leads[t >> 5] = __popc(starts[i]);
    }
    __syncthreads();
    const int n_units = __reduce_add_sync(0xffffffffu, lane < kLBlocks ? leads[lane] : 0);
#pragma unroll
    for (int i = 0; i < kLMaxT / kLThreads; ++i) {
        const int t = i * kLThreads + tid;
        const int before = __reduce_add_sync(0xffffffffu, lane < (t >> 5) ? leads[lane] : 0);
        if (starts[i] >> lane & 1) lead[before + __popc(starts[i] & below)] = t;
    }
    __syncthreads();

    const int gw = (int)cr * kLWarps + warp;  // warp of the cluster
    const int kw = warp % kKW, r0 = warp / kKW * 32, gk = (int)cr * kKW + kw;
    const int k_blocks = P.in >> 5, o_blocks = P.out >> 5;
    const int kb0 = gk * k_blocks / (kLCluster * kKW), kb1 = (gk + 1) * k_blocks / (kLCluster * kKW);
    const int ob0 = gw * o_blocks / (kLCluster * kLWarps), ob1 = (gw + 1) * o_blocks / (kLCluster * kLWarps);
    for (int u = cluster; u < n_units; u += clusters) {
        const int t0 = lead[u], a = adp[t0], k0 = key[t0], tile = rnk[t0] / kLTile;
        const int all = __reduce_add_sync(0xffffffffu, lane < blocks ? (int)count[lane * kLMaxT + k0] : 0);
        const int m = min(kLTile, all - tile * kLTile);
#pragma unroll 1
        for (int t = tid; t < P.T; t += kLThreads)
            if (key[t] == k0 && rnk[t] / kLTile == tile) tok[rnk[t] % kLTile] = t;
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
        const float scale = rank > 0 && P.scale ? P.scale[a] : 1.f;
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

        const bf16* B = P.b + (size_t)a * P.out * P.max_rank;
        uint2 wb[kKS][4];
        uint4 yb[2];
        auto load_out = [&](int ob) {
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
                const int k = ks * 16 + cq * 4;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // column 2c of tile j is feature 8c + 2j: a lane's outputs are neighbours
                    const int f = ob * 32 + (g >> 1) * 8 + j * 2 + (g & 1);
                    wb[ks][j] = k < rank ? *reinterpret_cast<const uint2*>(B + (size_t)f * P.max_rank + k)
                                         : make_uint2(0, 0);
                }
            }
            if (g < m) yb[0] = *reinterpret_cast<const uint4*>(P.y_in + (size_t)t_lo * P.ld_y_in + ob * 32 + cq * 8);
            if (g + 8 < m) yb[1] = *reinterpret_cast<const uint4*>(P.y_in + (size_t)t_hi * P.ld_y_in + ob * 32 + cq * 8);
        };
        // ---- A x: this warp's input features ----
        float acc[kNT][4];
#pragma unroll
        for (int j = 0; j < kNT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
        const bf16* A = P.a + (size_t)a * P.max_rank * P.in;
        const uint4 z = make_uint4(0, 0, 0, 0);
        uint4 xa[2], w[kNT];
        auto load_in = [&](int kb) {
            const int k = kb * 32 + cq * 8;
            xa[0] = g < m ? *reinterpret_cast<const uint4*>(P.x + (size_t)t_lo * P.ld_x + k) : z;
            xa[1] = g + 8 < m ? *reinterpret_cast<const uint4*>(P.x + (size_t)t_hi * P.ld_x + k) : z;
#pragma unroll
            for (int j = 0; j < kNT; ++j)
                w[j] = r0 + j * 8 + g < rank ? *reinterpret_cast<const uint4*>(A + (size_t)(r0 + j * 8 + g) * P.in + k) : z;
        };
        if (kb0 < kb1) load_in(kb0);
#pragma unroll 1
        for (int kb = kb0; kb < kb1; ++kb) {
            const uint32_t f0[4] = {xa[0].x, xa[1].x, xa[0].y, xa[1].y}, f1[4] = {xa[0].z, xa[1].z, xa[0].w, xa[1].w};
            uint4 c[kNT];
#pragma unroll
            for (int j = 0; j < kNT; ++j) c[j] = w[j];
            if (kb + 1 < kb1) load_in(kb + 1);
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
                mma16816(acc[j], f0, c[j].x, c[j].y);
                mma16816(acc[j], f1, c[j].z, c[j].w);
            }
        }
#pragma unroll
        for (int j = 0; j < kNT; ++j)
            if (r0 + j * 8 < rp) {
                float* r = red + (size_t)kw * kLTile * rp + r0 + j * 8 + 2 * cq;
                *reinterpret_cast<float2*>(r + g * rp) = make_float2(acc[j][0], acc[j][1]);
                *reinterpret_cast<float2*>(r + (g + 8) * rp) = make_float2(acc[j][2], acc[j][3]);
            }
        if (ob0 < ob1) load_out(ob0);  // on its way while the sums are joined
        __syncthreads();
        const int n4 = kLTile * rp / 4;
        for (int i = tid; i < n4; i += kLThreads) {
            float4 s = reinterpret_cast<const float4*>(red)[i];
#pragma unroll
            for (int w = 1; w < kKW; ++w) add4(s, reinterpret_cast<const float4*>(red)[w * n4 + i]);
            reinterpret_cast<float4*>(part)[i] = s;
        }
        cluster_arrive();
        cluster_wait();
        for (int i = tid; i < n4; i += kLThreads) {
            float4 v[kLCluster];
#pragma unroll
            for (int c = 0; c < kLCluster; ++c) v[c] = dsmem_ld(smem_u32(part + 4 * i), c);
#pragma unroll
            for (int c = 1; c < kLCluster; ++c) add4(v[0], v[c]);
            const int row = 4 * i / rp, col = 4 * i - row * rp, at = row * (rp + 8) + col;
            float s[4] = {v[0].x * scale, v[0].y * scale, v[0].z * scale, v[0].w * scale};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e >= rank) s[e] = 0.f;  // not the adapter's; an infinite x times 0 there is NaN
            float r[4];
            uint2 h, l;
            h.x = pack_bf16x2(s[0], s[1]);
            h.y = pack_bf16x2(s[2], s[3]);
            const float b[4] = {__uint_as_float(h.x << 16), __uint_as_float(h.x & 0xffff0000u),
                                __uint_as_float(h.y << 16), __uint_as_float(h.y & 0xffff0000u)};
#pragma unroll
            for (int e = 0; e < 4; ++e) r[e] = fabsf(b[e]) == INFINITY ? 0.f : s[e] - b[e];  // inf stays inf
            l.x = pack_bf16x2(r[0], r[1]);
            l.y = pack_bf16x2(r[2], r[3]);
            *reinterpret_cast<uint2*>(hi + at) = h;
            *reinterpret_cast<uint2*>(lo + at) = l;
        }
        cluster_arrive();  // this CTA has read the others' sums
        __syncthreads();   // hi and lo are complete

        // ---- y += B (A x): this warp's output features, 32 at a time ----
        for (int ob = ob0; ob < ob1; ++ob) {
            float d[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.f;
#pragma unroll
            for (int ks = 0; ks < kKS; ++ks) {
                const int k = ks * 16 + cq * 4;
                if (ks * 16 >= rank) break;
                if (k + 3 >= rank) {  // what lies behind the rank is not the adapter's
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (k + 1 >= rank) wb[ks][j].x &= 0xffffu;
                        if (k + 2 >= rank) wb[ks][j].y = 0u;
                        else wb[ks][j].y &= 0xffffu;
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const bf16* v = e ? lo : hi;
                    const uint2 v0 = *reinterpret_cast<const uint2*>(v + g * (rp + 8) + k);
                    const uint2 v1 = *reinterpret_cast<const uint2*>(v + (g + 8) * (rp + 8) + k);
                    const uint32_t f[4] = {v0.x, v1.x, v0.y, v1.y};
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma16816(d[j], f, wb[ks][j].x, wb[ks][j].y);
                }
            }
            const uint4 y0[2] = {yb[0], yb[1]};
            if (ob + 1 < ob1) load_out(ob + 1);
            const int f0 = ob * 32 + cq * 8;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (g + 8 * h >= m) continue;
                const size_t t = h ? t_hi : t_lo;
                float y[8];
                unpack8(y0[h], y);
                uint4 o;
                o.x = pack_bf16x2(y[0] + d[0][2 * h], y[1] + d[0][2 * h + 1]);
                o.y = pack_bf16x2(y[2] + d[1][2 * h], y[3] + d[1][2 * h + 1]);
                o.z = pack_bf16x2(y[4] + d[2][2 * h], y[5] + d[2][2 * h + 1]);
                o.w = pack_bf16x2(y[6] + d[3][2 * h], y[7] + d[3][2 * h + 1]);
                *reinterpret_cast<uint4*>(P.y_out + t * P.ld_y_out + f0) = o;
            }
        }
        cluster_wait();   // every CTA has read this one's sum
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
                    lora_smem_bytes(p.n, p.max_rank), args, true);
}

}  // namespace sgp
