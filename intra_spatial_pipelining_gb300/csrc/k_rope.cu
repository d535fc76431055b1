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

// A warp takes chunks of at most 16 rows of one token through a ring of its own in shared memory, filled
// by bulk copies: more is under way than registers would hold.  Four lanes take a row, the warp eight at a
// time; a lane holds 16 elements as two 16-byte pieces such that both elements of each of its pairs are its
// own: frequencies 8 c to 8 c + 7 for lane c of the four, in either layout.  Lane i of the warp computes
// cosine and sine of pair i once for a token.  The angle is a fraction of a turn in 64-bit fixed point,
// position times (frequency / 2 pi) modulo 1, exact however far the position.
// Bound by HBM: 16,384 tokens of 64 + 8 heads from a fused projection into q and caches, 336 MB, 55.2 us
// (0.90 of a copy's rate; 70 with rows in registers and a token to a warp), normed 56.2; with few heads by
// what a chunk costs (32 + 4 heads 32.1, normed 38.6, a copy 24.9); by latency and the host's 9 to 10 us a
// call for a batch of single tokens (2.6 us for one, 4.6 for 512).  Fewer rows to a chunk balance small
// calls, more serve large ones: 32 rows and 12 warps 5.6 for the batch.
constexpr int kRWarps = 16;
constexpr int kRThreads = 32 * kRWarps;
constexpr int kRRows = 16;                      // rows of a chunk
constexpr int kRStages = 4;
constexpr int kRStage = kRRows * 128;

// Two bf16 as two numbers, the lower half first.
__device__ __forceinline__ float2 numbers(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// A lane's words in the order of its pairs and back: word j of the one result holds the first elements of
// two pairs, of the other one the second elements.  With neighbouring elements as pairs these are pairs j
// and j + 4 of its eight, with halves apart pairs 2 j and 2 j + 1, and the words are in order already.
__device__ __forceinline__ void by_pairs(uint32_t& a, uint32_t& b, bool interleaved) {
    if (interleaved) {
        const uint32_t t = __byte_perm(a, b, 0x5410);
        b = __byte_perm(a, b, 0x7632);
        a = t;
    }
}

struct RopeSmem {
    uint64_t full[kRWarps][kRStages];
    unsigned long long turns[32];
    float2 trig[kRWarps][32];
};

// Chunks of a token: of q, of k, of v.
struct RopeChunks {
    int q, k, v;
};

// A warp's chunk.
struct RopePlace {
    int left, t, k;                             // chunks left; token, chunk of the token
};

__global__ void __launch_bounds__(kRThreads, 1) qk_rope_kernel(const __grid_constant__ RopeProblem P, const RopeChunks C, const KCtx ctx) {
    extern __shared__ __align__(128) uint8_t smem[];
    RopeSmem& S = *reinterpret_cast<RopeSmem*>(smem + (size_t)kRWarps * kRStages * kRStage);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    if (tid < kRWarps * kRStages) mbar_init(&S.full[0][0] + tid, 1);
    if (tid < 32) S.turns[tid] = P.turns[tid];
    fence_barrier_init();
    __syncthreads();
    griddep_wait();
    task_begin(ctx);
    // Many tokens go round the warps one by one: what is read and written at a time then lies close
    // together (16,384 tokens 54 us, 61 by equal runs).  Of fewer, whose last round would leave warps idle,
    // the warps take equal runs of chunks (4000 tokens 15.5 us, 17.9 one by one).
    const int per = C.q + C.k + C.v, total = P.T * per, warps = gridDim.x * kRWarps;
    const int w = warp * gridDim.x + blockIdx.x;
    const bool round = P.T >= 4 * warps;
    const int each = total / warps, more = total - each * warps;
    const int left = round ? (w < P.T ? (P.T - 1 - w) / warps + 1 : 0) * per : each + (w < more);
    if (left > 0) {
        uint8_t* ring = smem + (size_t)warp * kRStages * kRStage;
        uint64_t* full = S.full[warp];
        // Going round, a warp begins with another chunk of its tokens than its neighbours (55.8 us without,
        // for the 55.2 above) and has two chunks under way: with four, reads and writes get in each other's
        // way (62).
        const int start = round ? w % per : 0, depth = round ? 2 : kRStages;
        auto next = [&](RopePlace& x) {
            --x.left;
            if (++x.k == per) x.k = 0;
            if (x.k == start) x.t += round ? warps : 1;
        };
        // A token's sequence and slot, and its row in the caches; negative: it has none.
        auto where = [&](int t) { return make_int2(P.seq != nullptr ? P.seq[t] : t, P.slot[t]); };
        auto place = [&](int t, int2 x, bool tell) -> long long {
            const int s = x.x, at = x.y;
            const bool out = s >= P.n_seqs || (s >= 0 && (at < 0 || at >= P.cap));
            if (out && tell) report(ctx, ST_BOUNDS, (uint32_t)t);
            return s < 0 || out ? -1 : (long long)s * P.nkv * P.cap + at;
        };
        const bool in_place = P.k_cache != nullptr && P.k == nullptr;
        auto issue = [&](RopePlace& x, int st) {
            uint8_t* dst = ring + st * kRStage;
            if (x.k >= C.q && x.k < C.q + C.k && in_place) {
                const int j = (x.k - C.q) * kRRows + lane;
                const long long at = place(x.t, where(x.t), false);
                const bool live = lane < kRRows && j < P.nkv && at >= 0;
                const unsigned rows = __popc(__ballot_sync(0xffffffffu, live));
                if (lane == 0) mbar_arrive_expect_tx(&full[st], rows * 128);
                __syncwarp();
                if (live) bulk_load(dst + lane * 128, P.k_cache + (at + (long long)j * P.cap) * 64, 128, &full[st]);
            } else if (lane == 0) {
                const bf16* src;
                int rows, first;
                if (x.k < C.q) {
                    first = x.k * kRRows;
                    rows = P.nq - first;
                    src = P.q + x.t * P.ld_q;
                } else {
                    const bool v = x.k >= C.q + C.k;
                    first = (x.k - C.q - (v ? C.k : 0)) * kRRows;
                    rows = P.nkv - first;
                    src = v ? P.v + x.t * P.ld_v : P.k + x.t * P.ld_k;
                }
                const uint32_t bytes = min(rows, kRRows) * 128;
                mbar_arrive_expect_tx(&full[st], bytes);
                bulk_load(dst, src + first * 64, bytes, &full[st]);
            }
            next(x);
        };
        RopePlace cs;
        cs.left = left;
        const int first = round ? w * per : w * each + min(w, more);
        cs.t = first / per;
        cs.k = round ? start : first - cs.t * per;
        RopePlace ld = cs;
        uint32_t issued = 0, done = 0;
#pragma unroll
        for (int st = 0; st < kRStages; ++st)
            if (ld.left > 0 && st < depth) {
                issue(ld, st);
                ++issued;
            }
        // this lane's two pieces of 8 elements; whether its pairs are rotated, all of them or none
        const bool spin = c < P.rot / 16;
        int c0 = 2 * c, c1 = 2 * c + 1;
        if (!P.interleaved) {
            const int n = P.rot / 16;           // lanes with rotated pieces
            c0 = c < n ? c : 2 * n + 2 * (c - n);
            c1 = c < n ? c + n : c0 + 1;
        }
        // positions and places of the warp's next 32 tokens, one to a lane (8 + 8 heads, 16,384 tokens: 22.5
        // us; 25.0 with one token's loaded ahead)
        int pos = 0, nth = 0;
        int2 put = make_int2(-1, 0);
        auto ahead = [&](int t) {
            const long long mine = t + (long long)lane * (round ? warps : 1);
            if (mine < P.T) {
                pos = P.pos[mine];
                if (P.k_cache != nullptr) put = where((int)mine);
            }
            nth = 0;
        };
        ahead(cs.t);
        // (first, second) -> (first * ff + second * sf, second * ss + first * fs), gains included
        float2 ff[4], sf[4], ss[4], fs[4];
        const bf16* with = nullptr;             // gains that they have in them
        long long at = -1;                      // the token's row in the caches
        int token = -1, st = 0, parity = 0;
        bool fresh = false, failed = false;
        while (cs.left > 0) {
            if (cs.t != token) {
                token = cs.t;
                if (nth == 32) ahead(token);
                if (P.k_cache != nullptr)
                    at = place(token, make_int2(__shfl_sync(0xffffffffu, put.x, nth), __shfl_sync(0xffffffffu, put.y, nth)), lane == 0);
                const unsigned long long turn = S.turns[lane] * (unsigned long long)(long long)__shfl_sync(0xffffffffu, pos, nth);
                ++nth;
                float sn, cn;
                sincospif((float)(int)(turn >> 32) * 0x1p-31f, &sn, &cn);
                __syncwarp();
                S.trig[warp][lane] = lane < P.rot / 2 ? make_float2(cn * P.amplitude, sn * P.amplitude) : make_float2(1.f, 0.f);
                __syncwarp();
                fresh = true;
            }
            // where the chunk goes
            const bf16* gain = P.g_q;
            bf16* dst;
            long long step = 64;
            int rows;
            bool turned = true, kept = true;
            if (cs.k < C.q) {
                const int first = cs.k * kRRows;
                rows = P.nq - first;
                dst = P.q_out + token * P.ld_q_out + first * 64;
            } else {
                turned = cs.k < C.q + C.k;
                const int first = (cs.k - C.q - (turned ? 0 : C.k)) * kRRows;
                rows = P.nkv - first;
                gain = P.g_k;
                if (P.k_cache != nullptr) {
                    kept = at >= 0;
                    step = (long long)P.cap * 64;
                    dst = (turned ? P.k_cache : P.v_cache) + at * 64 + first * step;
                } else {
                    dst = P.k_out + token * P.ld_k_out + first * 64;
                }
            }
            rows = min(rows, kRRows);
            const bool ok = mbar_wait(&full[st], parity, ctx.timeout_ns);
            if (__any_sync(0xffffffffu, !ok)) {
                if (lane == 0) report(ctx, ST_TIMEOUT, 30);
                failed = true;
                break;
            }
            if (turned && (fresh || gain != with)) {
                fresh = false;
                with = gain;
                uint4 g0 = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u), g1 = g0;     // ones
                if (gain != nullptr) {
                    g0 = *reinterpret_cast<const uint4*>(gain + c0 * 8);
                    g1 = *reinterpret_cast<const uint4*>(gain + c1 * 8);
                }
                uint32_t gf[4] = {g0.x, g0.y, g0.z, g0.w}, gs[4] = {g1.x, g1.y, g1.z, g1.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    by_pairs(gf[j], gs[j], P.interleaved);
                    const float2 t0 = S.trig[warp][8 * c + (P.interleaved ? j : 2 * j)];
                    const float2 t1 = S.trig[warp][8 * c + (P.interleaved ? j + 4 : 2 * j + 1)];
                    const float2 f = numbers(gf[j]), s = numbers(gs[j]);
                    ff[j] = make_float2(t0.x * f.x, t1.x * f.y);
                    fs[j] = make_float2(t0.y * f.x, t1.y * f.y);
                    ss[j] = make_float2(t0.x * s.x, t1.x * s.y);
                    sf[j] = make_float2(-t0.y * s.x, -t1.y * s.y);
                }
            }
            if (kept) {
                const uint8_t* row = ring + st * kRStage + g * 128;
                dst += g * step;
#pragma unroll 1
                for (int j = g; j - g < rows; j += 8) {
                    uint4 x0 = *reinterpret_cast<const uint4*>(row + c0 * 16), x1 = *reinterpret_cast<const uint4*>(row + c1 * 16);
                    row += 1024;
                    if (turned && (spin || gain != nullptr)) {
                        uint32_t u[4] = {x0.x, x0.y, x0.z, x0.w}, v[4] = {x1.x, x1.y, x1.z, x1.w};
                        float2 f[4], s[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            by_pairs(u[i], v[i], P.interleaved);
                            f[i] = numbers(u[i]);
                            s[i] = numbers(v[i]);
                        }
                        float2 inv = make_float2(1.f, 1.f);
                        if (gain != nullptr) {
                            float2 sum = mul2(f[0], f[0]);
#pragma unroll
                            for (int i = 1; i < 4; ++i) sum = fma2(f[i], f[i], sum);
#pragma unroll
                            for (int i = 0; i < 4; ++i) sum = fma2(s[i], s[i], sum);
                            float q = sum.x + sum.y;
                            q += __shfl_xor_sync(0xffffffffu, q, 1);
                            q += __shfl_xor_sync(0xffffffffu, q, 2);
                            inv.x = inv.y = rsqrtf(fmaf(q, 1.f / 64.f, P.eps));
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float2 y = mul2(f[i], ff[i]), z = mul2(s[i], ss[i]);
                            if (spin) {         // elsewhere 0 times an infinity would not be 0
                                y = fma2(s[i], sf[i], y);
                                z = fma2(f[i], fs[i], z);
                            }
                            if (gain != nullptr) {
                                y = mul2(y, inv);
                                z = mul2(z, inv);
                            }
                            u[i] = pack_bf16x2(y.x, y.y);
                            v[i] = pack_bf16x2(z.x, z.y);
                            by_pairs(u[i], v[i], P.interleaved);
                        }
                        x0 = make_uint4(u[0], u[1], u[2], u[3]);
                        x1 = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                    if (j < rows) {
                        *reinterpret_cast<uint4*>(dst + c0 * 8) = x0;
                        *reinterpret_cast<uint4*>(dst + c1 * 8) = x1;
                    }
                    dst += 8 * step;
                }
            }
            ++done;
            fence_proxy_async();
            __syncwarp();
            if (ld.left > 0) {
                issue(ld, st);
                ++issued;
            }
            if (++st == depth) {
                st = 0;
                parity ^= 1;
            }
            next(cs);
        }
        if (failed)                             // loads still in flight
            for (uint32_t n = done; n < issued; ++n)
                (void)mbar_wait(&full[n % depth], (n / depth) & 1u, 10000000ull);
    }
    task_end(ctx);
}

}  // namespace

int enqueue_qk_rope(Launcher& L, const RopeProblem& p, const KCtx& c, int sms) {
    const int chunks = (p.nkv + kRRows - 1) / kRRows;
    RopeChunks C;
    C.q = p.q != nullptr ? (p.nq + kRRows - 1) / kRRows : 0;
    C.k = p.k != nullptr || p.k_cache != nullptr ? chunks : 0;
    C.v = p.v != nullptr ? chunks : 0;
    const int total = p.T * (C.q + C.k + C.v);
    const size_t smem = (size_t)kRWarps * kRStages * kRStage + sizeof(RopeSmem);
    void* args[] = {(void*)&p, (void*)&C, (void*)&c};
    return L.launch((const void*)qk_rope_kernel, dim3(total < sms ? total : sms), dim3(kRThreads), smem, args, true);
}

}  // namespace sgp
