// Norms and rotation of queries and keys, on their way into a cache or not.
//
//   x' = x rsqrt(mean(x^2) + eps) * gain                       (each head's row by itself)
//   (a, b) -> amplitude (a cos(f p) - b sin(f p), b cos(f p) + a sin(f p))
//
// for the pairs (a, b) of the rotated part: elements (i, i + rot / 2) or (2 i, 2 i + 1), frequency f_i,
// position p.  Sums and products are fp32; the result is rounded once.
#include "serving.cuh"

namespace sgp {

namespace {

// Four lanes to a row, a warp to eight rows of one token at a time; a lane holds 16 elements as two
// 16-byte chunks such that both elements of each of its pairs are its own: frequencies 8 c to 8 c + 7
// for lane c of the four, in either layout.  Lane i of the warp computes cosine and sine of pair i
// once for all heads.  The angle is a fraction of a turn in 64-bit fixed point, position times
// (frequency / 2 pi) modulo 1, exact however far the position.
constexpr int kRThreads = 256;
constexpr int kRWarps = kRThreads / 32;

__global__ void __launch_bounds__(kRThreads) qk_rope_kernel(const __grid_constant__ RopeProblem P, const int parts, const KCtx ctx) {
    __shared__ unsigned long long turns[32];
    __shared__ __align__(16) float2 trig[kRWarps][32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    if (tid < 32) turns[tid] = P.turns[tid];
    __syncthreads();
    griddep_wait();
    task_begin(ctx);
    const long long item = (long long)blockIdx.x * kRWarps + warp;
    if (item < (long long)P.T * parts) {
        const int t = (int)(item / parts), part = (int)(item - (long long)t * parts);
        const int half = P.rot / 2;
        {
            const unsigned long long turn = turns[lane] * (unsigned long long)(long long)P.pos[t];
            float sn, cs;
            sincospif((float)(int)(turn >> 32) * 0x1p-31f, &sn, &cs);
            trig[warp][lane] = lane < half ? make_float2(cs * P.amplitude, sn * P.amplitude) : make_float2(1.f, 0.f);
        }
        __syncwarp();
        float2 r[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(&trig[warp][8 * c + 2 * i]);
            r[2 * i] = make_float2(v.x, v.y);
            r[2 * i + 1] = make_float2(v.z, v.w);
        }
        // this lane's chunks of 8 elements
        int c0 = 2 * c, c1 = 2 * c + 1;
        if (!P.interleaved) {
            const int n = P.rot / 16;           // lanes with rotated chunks
            c0 = c < n ? c : 2 * n + 2 * (c - n);
            c1 = c < n ? c + n : c0 + 1;
        }
        // the token's row of the caches
        bool cached = P.k_cache != nullptr;
        size_t base = 0, step = 0;
        if (cached) {
            const int s = P.seq != nullptr ? P.seq[t] : t, at = P.slot[t];
            const bool out = s >= P.n_seqs || (s >= 0 && (at < 0 || at >= P.cap));
            if (out && part == 0 && lane == 0) report(ctx, ST_BOUNDS, (uint32_t)t);
            cached = s >= 0 && !out;
            if (cached) {
                base = ((size_t)s * P.nkv * P.cap + at) * 64;
                step = (size_t)P.cap * 64;
            }
        }
        const int rows = P.nq + 2 * P.nkv, groups = (rows + 7) / 8;
        const int g0 = groups * part / parts, g1 = groups * (part + 1) / parts;
#pragma unroll 2
        for (int grp = g0; grp < g1; ++grp) {
            const int row = grp * 8 + g;
            const bf16 *src = nullptr, *gain = nullptr;
            bf16* dst = nullptr;
            bool turned = true;
            if (row < P.nq) {
                if (P.q != nullptr) {
                    src = P.q + t * P.ld_q + row * 64;
                    dst = P.q_out + t * P.ld_q_out + row * 64;
                    gain = P.g_q;
                }
            } else if (row < P.nq + P.nkv) {
                const int j = row - P.nq;
                gain = P.g_k;
                if (P.k_cache == nullptr) {
                    if (P.k != nullptr) {
                        src = P.k + t * P.ld_k + j * 64;
                        dst = P.k_out + t * P.ld_k_out + j * 64;
                    }
                } else if (cached) {
                    dst = P.k_cache + base + j * step;
                    src = P.k != nullptr ? P.k + t * P.ld_k + j * 64 : dst;
                }
            } else if (row < rows && cached && P.v != nullptr) {
                const int j = row - P.nq - P.nkv;
                src = P.v + t * P.ld_v + j * 64;
                dst = P.v_cache + base + j * step;
                turned = false;
            }
            uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
            if (src != nullptr) {
                x0 = *reinterpret_cast<const uint4*>(src + 8 * c0);
                x1 = *reinterpret_cast<const uint4*>(src + 8 * c1);
            }
            float a[8], b[8];
            unpack8(x0, a);
            unpack8(x1, b);
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
            ss += __shfl_xor_sync(0xffffffffu, ss, 1);
            ss += __shfl_xor_sync(0xffffffffu, ss, 2);
            if (src == nullptr) continue;
            if (turned) {
                if (gain != nullptr) {
                    const float inv = rsqrtf(fmaf(ss, 1.f / 64.f, P.eps));
                    float ga[8], gb[8];
                    unpack8(*reinterpret_cast<const uint4*>(gain + 8 * c0), ga);
                    unpack8(*reinterpret_cast<const uint4*>(gain + 8 * c1), gb);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        a[i] *= inv * ga[i];
                        b[i] *= inv * gb[i];
                    }
                }
                if (P.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float u = a[2 * i], v = a[2 * i + 1], y = b[2 * i], z = b[2 * i + 1];
                        a[2 * i] = u * r[i].x - v * r[i].y;
                        a[2 * i + 1] = v * r[i].x + u * r[i].y;
                        b[2 * i] = y * r[4 + i].x - z * r[4 + i].y;
                        b[2 * i + 1] = z * r[4 + i].x + y * r[4 + i].y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float u = a[i], v = b[i];
                        a[i] = u * r[i].x - v * r[i].y;
                        b[i] = v * r[i].x + u * r[i].y;
                    }
                }
                x0 = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                                pack_bf16x2(a[6], a[7]));
                x1 = make_uint4(pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]), pack_bf16x2(b[4], b[5]),
                                pack_bf16x2(b[6], b[7]));
            }
            *reinterpret_cast<uint4*>(dst + 8 * c0) = x0;
            *reinterpret_cast<uint4*>(dst + 8 * c1) = x1;
        }
    }
    task_end(ctx);
}

}  // namespace

int enqueue_qk_rope(Launcher& L, const RopeProblem& p, const KCtx& c, int sms) {
    // warps to a token: one, or enough of them to give every SM sixteen
    const int groups = (p.nq + 2 * p.nkv + 7) / 8;
    int parts = (16 * sms + p.T - 1) / p.T;
    if (parts > groups) parts = groups;
    const long long warps = (long long)p.T * parts;
    void* args[] = {(void*)&p, (void*)&parts, (void*)&c};
    return L.launch((const void*)qk_rope_kernel, dim3((unsigned)((warps + kRWarps - 1) / kRWarps)), dim3(kRThreads), 0, args, true);
}

}  // namespace sgp
