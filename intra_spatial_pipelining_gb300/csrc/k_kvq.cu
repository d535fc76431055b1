// A cache held in 8 bits, and decode attention over it.
//
//   codes   k_p = code * scale, one scale for a block of positions, head and tensor; codes are e4m3
//           numbers or 8-bit integers;
//   fold    the full blocks at the front of a bf16 cache become codes, the positions behind them
//           move to its front (or to another cache's);
//   attention   s_p = q . k_p / sqrt(d) over the coded positions, then over the bf16 ones behind
//           them; o = sum softmax(s)_p v_p.
#include "serving.cuh"

namespace sgp {

namespace {

// ---------------------------------------------------------------------------------------
// codes to fp16 (exact: an e4m3 number and an 8-bit integer have at most 8 significant bits)
// ---------------------------------------------------------------------------------------
// the numbers of two bytes, the lower one in the lower half
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
    uint32_t d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(d) : "r"(two));
    return d;
}
// 0x6400 + u is the fp16 number 1024 + u for a byte u; with u = code + 128, 1152 too much
__device__ __forceinline__ uint32_t sub_1152(uint32_t x) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(0x64806480u));
    return d;
}
// codes (b0, b1) and (b2, b3) of a word
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (FMT == KVQ_INT8) {
        w ^= 0x80808080u;
        lo = sub_1152(__byte_perm(w, 0x64646464u, 0x4140));
        hi = sub_1152(__byte_perm(w, 0x64646464u, 0x4342));
    } else {
        lo = e4m3x2_f16x2(w);
        hi = e4m3x2_f16x2(w >> 16);
    }
}

// D(16x8, fp32) += A(16x16, fp16, row) * B(16x8, fp16, col)
__device__ __forceinline__ void mma16816_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// NaN if one of them is
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

__device__ __forceinline__ void bulk_load_once(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t pol) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar)), "l"(pol)
        : "memory");
}

// ---------------------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------------------
constexpr int kQThreads = kKvqWarps * 32;
constexpr int kQTile = 64;                      // coded positions of a tile
constexpr int kQTail = 32;                      // bf16 positions of a tile: as many bytes
constexpr int kQHalf = 4096;                    // K (or V) bytes of a tile
constexpr int kQStages = 2;
constexpr int kQMax = 512;                      // sequences
static_assert(2 * kQThreads >= kQMax, "the plan takes two sequences to a thread");
constexpr float kPShift = 14.f;                 // weights of V are below 2^14: fp16 down to 2^-28 of the largest

// n things cut into `parts` runs, the longer ones first.
struct Cuts {
    int each, more;                             // `more` runs have one thing more
    __device__ __forceinline__ Cuts(int n, int parts) : each(n / parts), more(n - n / parts * parts) {}
    __device__ __forceinline__ int begin(int run) const { return run * each + min(run, more); }
    __device__ __forceinline__ int of(int i) const {
        const int edge = more * (each + 1);
        return i < edge ? i / (each + 1) : more + (i - edge) / max(each, 1);
    }
};

struct alignas(16) KvqSmem {
    uint64_t full[kKvqWarps][kQStages];
    int pre[kQMax + 1];                         // tiles before each sequence
    int held[kQMax], len[kQMax];                // lengths, 0 where out of range
    int sums[kKvqWarps];
};

// A sequence's tiles for one KV head: coded ones from `q0` on (a multiple of the tile), then the
// bf16 ones from `b0` on.
struct Span {
    int low, q0, nq, b0, nb;                    // low: first visible position
};
__device__ __forceinline__ Span span_of(int held, int len, int window) {
    Span s;
    s.low = window > 0 ? max(0, held + len - window) : 0;
    s.q0 = min(s.low, held) & ~(kQTile - 1);
    s.nq = s.low < held ? (held - s.q0 + kQTile - 1) / kQTile : 0;
    s.b0 = max(0, s.low - held) & ~(kQTail - 1);
    s.nb = len > s.b0 ? (len - s.b0 + kQTail - 1) / kQTail : 0;
    return s;
}

// The lengths of sequence t, both 0 where one of them is out of range.
__device__ __forceinline__ int2 lengths_of(const KvqProblem& P, int t, const KCtx& ctx, bool tell) {
    int h = P.held[t], n = P.kv_len != nullptr ? P.kv_len[t] : 0;
    if (h < 0 || h > P.cap || (h & (P.block - 1)) || n < 0 || n > P.tail_cap) {
        if (tell) report(ctx, ST_BOUNDS, (uint32_t)t);
        h = n = 0;
    }
    return make_int2(h, n);
}

// A tile of a share.
struct Place {
    int i, t, kvh, c, per;                      // tile index; sequence, KV head, tile of the pair, tiles a pair
    Span s;
};

// The joined parts of one query head: maximum, sum, and four dims to a thread of sixteen.
struct Join {
    float M = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);

    // raises the maximum; then takes parts whose maxima are not above it
    __device__ __forceinline__ void raise(float top) {
        const float f = ex2(M - (top == -INFINITY ? 0.f : top));
        M = top;
        L *= f;
        a.x *= f;
        a.y *= f;
        a.z *= f;
        a.w *= f;
    }
    __device__ __forceinline__ void take(float2 ml, const float4& v) {
        const float f = ex2(ml.x - (M == -INFINITY ? 0.f : M));
        L = fmaf(f, ml.y, L);
        a.x = fmaf(f, v.x, a.x);
        a.y = fmaf(f, v.y, a.y);
        a.z = fmaf(f, v.z, a.z);
        a.w = fmaf(f, v.w, a.w);
    }
    // n parts, the rows given by a function of the index (two passes: maxima, then sums)
    template <typename F>
    __device__ __forceinline__ void take_all(int n, F row, int sub) {
        float top = M;
#pragma unroll 4
        for (int k = 0; k < n; ++k) top = fmaxf(top, row(k)[64]);
        raise(top);
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const float* r = row(k);
            take(*reinterpret_cast<const float2*>(r + 64), *reinterpret_cast<const float4*>(r + 4 * sub));
        }
    }
    __device__ __forceinline__ void put(float* r, int sub) const {
        *reinterpret_cast<float4*>(r + 4 * sub) = a;
        if (sub == 0) *reinterpret_cast<float2*>(r + 64) = make_float2(M, L);
    }
    __device__ __forceinline__ void finish(const KvqProblem& P, size_t at, int sub) const {
        const float inv = 1.f / L;
        *reinterpret_cast<uint2*>(P.o + at * 64 + 4 * sub) =
            make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
        if (P.lse != nullptr && sub == 0) P.lse[at] = (M + log2f(L)) * 0.6931471805599453f;
    }
    // a sequence without positions: o = 0, lse = -inf
    __device__ __forceinline__ void nothing(const KvqProblem& P, size_t at, int sub) const {
        *reinterpret_cast<uint2*>(P.o + at * 64 + 4 * sub) = make_uint2(0, 0);
        if (P.lse != nullptr && sub == 0) P.lse[at] = -INFINITY;
    }
};

// One query group against one KV head at a time: q^T are the columns of warp-level products,
//     S^T = K q^T   (16 positions x 8 heads, 64 dims),   O^T += V^T P^T   (16 dims x 8 heads, 16 positions),
// K and V decoded to fp16 in registers (exact), fp32 sums.  A scale is a factor of the scores, or of the
// weights before they are rounded for the second product: with m the running maximum of the scores s and mv
// that of s + log2(v_scale), a weight of V is 2^(s + log2(v_scale) - mv + 14), at most 2^14, so that fp16
// holds all that counts however the scales differ, while the sum of the weights goes by m alone.
// Tiles of 64 positions (32 of the bf16 cache, the same bytes) come by bulk copies into a ring of each
// warp's own, two stages; the order of a product's positions and dims is free, so lanes read K and V from
// shared memory as they lie: 16 bytes of one position for K, 8 of each of four for V, whose rows are taken
// such that a quad's lanes read both parities (two-way conflicts instead of four).
// Bound by HBM for long caches: 512 sequences of up to 32,768 positions on one head (int8) 160.8 us, 0.98 of
// a copy's rate (e4m3, whose codes the compiler unpacks with more instructions, 170); 64 sequences x 8 heads
// of up to 8192 49.4, of which 1.3 are the plan, about 4 the shares' uneven ends and 3.5 the join; 10 warps
// instead of 12: 198 and 55.  Beyond 8 heads to a group the instructions bound it (16: 64.6).
//
// WHOLE: a CTA to each pair ((sequence, KV head)), whose warps share its tiles and join their parts in
// shared memory (2 sequences x 8 heads of up to 512 positions: 5.0 us).  Else the tiles of all pairs are cut
// into equal shares, one to a warp; a part that is not a whole pair goes to the workspace, for
// kvq_merge_kernel.  (A join by the last CTA to arrive: as long, since its code is met cold, and shares of
// neighbouring tiles on one SM end less evenly.)
// ALIKE: a tile has one scale (blocks of 64 and more); a form of its own, because with a branch in the loop
// the compiler does not interleave what is around it (the first case above 175.6 us with the branch, 165.9
// without the case).
template <int NT, int FMT, bool WHOLE, bool ALIKE>
__global__ void __launch_bounds__(kQThreads, 1) kvq_attn_kernel(const __grid_constant__ KvqProblem P, const KCtx ctx) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    KvqSmem& S = *reinterpret_cast<KvqSmem*>(smem + (size_t)kKvqWarps * kQStages * 2 * kQHalf);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cq = lane & 3;

    if (tid < kKvqWarps * kQStages) mbar_init(&S.full[0][0] + tid, 1);
    fence_barrier_init();
    griddep_wait();
    task_begin(ctx);
    // This warp's tiles [i0, i1), and the sequence, KV head and tile of the pair that i0 is.  In WHOLE the
    // tiles are counted from the pair's first.
    int i0, i1;
    Place cs;
    if constexpr (WHOLE) {
        cs.t = blockIdx.x / P.nkv;
        cs.kvh = blockIdx.x - cs.t * P.nkv;
        const int2 l = lengths_of(P, cs.t, ctx, cs.kvh == 0 && tid == 0);
        if (tid == 0) {
            S.held[cs.t] = l.x;
            S.len[cs.t] = l.y;
        }
        cs.s = span_of(l.x, l.y, P.window);
        cs.per = cs.s.nq + cs.s.nb;
        const Cuts shares(cs.per, kKvqWarps);
        i0 = cs.i = cs.c = shares.begin(warp);
        i1 = shares.begin(warp + 1);
        __syncthreads();
    } else {
        // tiles before each sequence: two sequences to a thread
        int cnt[2], sum = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int t = 2 * tid + k;
            cnt[k] = 0;
            if (t < P.T) {
                const int2 l = lengths_of(P, t, ctx, blockIdx.x == 0);
                S.held[t] = l.x;
                S.len[t] = l.y;
                const Span s = span_of(l.x, l.y, P.window);
                cnt[k] = (s.nq + s.nb) * P.nkv;
            }
            sum += cnt[k];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) S.sums[warp] = incl;
        __syncthreads();
        int run = incl - sum;
        for (int i = 0; i < warp; ++i) run += S.sums[i];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int t = 2 * tid + k;
            if (t < P.T) {
                S.pre[t] = run;
                // a sequence without positions has no parts
                if (cnt[k] == 0 && blockIdx.x == 0)
                    for (int j = 0; j < P.nkv; ++j) P.parts[t * P.nkv + j] = make_int2(0, 0);
            }
            run += cnt[k];
            if (t == P.T - 1) S.pre[P.T] = run;
        }
        __syncthreads();
        // neighbouring shares are different SMs'
        const Cuts shares(S.pre[P.T], kKvqShares);
        const int w = warp * kKvqCtas + blockIdx.x;
        i0 = shares.begin(w);
        i1 = shares.begin(w + 1);
        if (i0 < i1) {
            int t = 0, hi = P.T;                // largest t with pre[t] <= i0
            while (hi - t > 1) {
                const int mid = (t + hi) >> 1;
                if (S.pre[mid] <= i0) t = mid;
                else hi = mid;
            }
            cs.i = i0;
            cs.t = t;
            cs.s = span_of(S.held[t], S.len[t], P.window);
            cs.per = cs.s.nq + cs.s.nb;
            const int r = i0 - S.pre[t];
            cs.kvh = r / cs.per;
            cs.c = r - cs.kvh * cs.per;
        }
    }
    if (i0 < i1) {
        uint8_t* ring = smem + (size_t)warp * kQStages * 2 * kQHalf;
        uint64_t* full = S.full[warp];
        const uint64_t pol = policy_evict_first();

        auto next = [&](Place& x) {
            ++x.i;
            if (++x.c < x.per || WHOLE) return;
            x.c = 0;
            if (++x.kvh < P.nkv) return;
            x.kvh = 0;
            if (x.i >= i1) return;
            do ++x.t;
            while (S.pre[x.t + 1] <= x.i);
            x.s = span_of(S.held[x.t], S.len[x.t], P.window);
            x.per = x.s.nq + x.s.nb;
        };
        Place ld = cs;
        // Scales of the tiles in flight: lane m holds the key scale of the tile's positions 16 m and
        // up, lane 4 + m the logarithm of their value scale; 1 where no position is visible.
        float sc[kQStages];
        auto issue = [&](int st) -> float {     // tile `ld` into stage st, then the next one
            const size_t pair = (size_t)ld.t * P.nkv + ld.kvh;
            uint8_t* dst = ring + st * 2 * kQHalf;
            float scale = 1.f;
            if (ld.c < ld.s.nq) {
                const int p0 = ld.s.q0 + ld.c * kQTile, rows = min(kQTile, S.held[ld.t] - p0);
                if (lane == 0) {
                    const size_t at = (pair * P.cap + p0) * 64;
                    mbar_arrive_expect_tx(&full[st], rows * 128);
                    bulk_load_once(dst, P.k + at, rows * 64, &full[st], pol);
                    bulk_load_once(dst + kQHalf, P.v + at, rows * 64, &full[st], pol);
                }
                const int p = p0 + (lane & 3) * 16;
                if (lane < 8 && p < p0 + rows && p + 16 > ld.s.low) {
                    const size_t at = pair * (P.cap >> P.block_log2) + (p >> P.block_log2);
                    scale = __ldg((lane < 4 ? P.ks : P.vs) + at);
                }
            } else if (lane == 0) {
                const int p0 = ld.s.b0 + (ld.c - ld.s.nq) * kQTail, rows = min(kQTail, S.len[ld.t] - p0);
                const size_t at = (pair * P.tail_cap + p0) * 64;
                mbar_arrive_expect_tx(&full[st], rows * 256);
                bulk_load_once(dst, P.tk + at, rows * 128, &full[st], pol);
                bulk_load_once(dst + kQHalf, P.tv + at, rows * 128, &full[st], pol);
            }
            next(ld);
            return scale;
        };
        uint32_t issued = 0, done = 0;          // tiles
#pragma unroll
        for (int st = 0; st < kQStages; ++st) {
            sc[st] = 1.f;
            if (ld.i < i1) {
                sc[st] = issue(st);
                ++issued;
            }
        }

        // Queries of a (sequence, KV head): lane (g, c) holds dims 16 c to 16 c + 15 of heads 8 nt + g, as
        // they are and in fp16, times a power of two.
        uint32_t qh[NT][4][2], qb[NT][4][2];
        auto load_q = [&]() {
            const bf16* qa = P.q + ((size_t)cs.t * P.nq + (size_t)cs.kvh * P.G) * 64 + 16 * cq;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int h = nt * 8 + g;
                uint4 a = make_uint4(0, 0, 0, 0), b = a;
                if (h < P.G) {
                    a = *reinterpret_cast<const uint4*>(qa + h * 64);
                    b = *reinterpret_cast<const uint4*>(qa + h * 64 + 8);
                }
                const uint32_t r[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) qb[nt][e >> 1][e & 1] = r[e];
            }
        };
        load_q();
        float qs[NT][2];                        // factor of a score of heads 2 cq, 2 cq + 1
        float m[NT][2], mv[NT][2], l[NT][2], oacc[4][NT][4];
        bool fresh = true, failed = false;
        while (cs.i < i1) {
            const int st = done % kQStages;
            if (fresh) {
                fresh = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t top = 0;           // largest magnitude's bits
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t x = qb[nt][e >> 1][e & 1];
                        top = max(top, max(x & 0x7fffu, (x >> 16) & 0x7fffu));
                    }
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // a power of two takes the largest to [2^14, 2^15): fp16 holds bf16's bits down to
                    // 2^-28 of it, below with an error of 2^-39 of it
                    const int ex = min(max((int)(top >> 7) - 127 - 14, -126), 126);
                    const float up = pow2i(-ex);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t x = qb[nt][kk][e];
                            qh[nt][kk][e] = pack_f16x2(__uint_as_float(x << 16) * up,
                                                       __uint_as_float(x & 0xffff0000u) * up);
                        }
                    const float down = pow2i(ex) * P.scale_log2;
                    qs[nt][0] = __shfl_sync(0xffffffffu, down, 8 * cq);
                    qs[nt][1] = __shfl_sync(0xffffffffu, down, 8 * cq + 4);
                    m[nt][0] = m[nt][1] = mv[nt][0] = mv[nt][1] = -INFINITY;
                    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
                    for (int md = 0; md < 4; ++md)
                        oacc[md][nt][0] = oacc[md][nt][1] = oacc[md][nt][2] = oacc[md][nt][3] = 0.f;
                }
            }
            const bool ok = mbar_wait(&full[st], (done / kQStages) & 1u, ctx.timeout_ns);
            if (__any_sync(0xffffffffu, !ok)) {
                if (lane == 0) report(ctx, ST_TIMEOUT, 20);
                failed = true;
                break;
            }
            uint8_t* kt = ring + st * 2 * kQHalf;
            uint8_t* vt = kt + kQHalf;
            const bool coded = cs.c < cs.s.nq;
            const int held = S.held[cs.t];
            // rows [lo, hi) of the tile are visible; the others of V become 0
            const int p0 = coded ? cs.s.q0 + cs.c * kQTile : held + cs.s.b0 + (cs.c - cs.s.nq) * kQTail;
            const int size = coded ? kQTile : kQTail, rowb = coded ? 64 : 128;
            const int lo = max(0, cs.s.low - p0), hi = min(size, (coded ? held : held + S.len[cs.t]) - p0);
            const bool part = lo > 0 || hi < size;
            if (part) {
                for (int e = lane * 16; e < kQHalf; e += 512) {
                    const int r = e / rowb;
                    if (r < lo || r >= hi) *reinterpret_cast<uint4*>(vt + e) = make_uint4(0, 0, 0, 0);
                }
                __syncwarp();
            }
            // row r of a 16-position product is position rho(r) of its half: the lanes of a quad read
            // V rows of both parities
            const int rho = g ^ ((g >> 1) & 1);
            float s[4][NT][4], lsv[4];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                lsv[mt] = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
            }
            // ---- S^T = K q^T ----
            if (coded) {
                const float own = lane < 4 ? sc[0] : lg2(sc[0]);
                // a lane with a visible position's scale
                const int one = min(lo >> 4, 3);
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    const uint4 k0 = *reinterpret_cast<const uint4*>(kt + (mt * 16 + rho) * 64 + cq * 16);
                    const uint4 k1 = *reinterpret_cast<const uint4*>(kt + (mt * 16 + 8 + rho) * 64 + cq * 16);
                    const uint32_t x0[4] = {k0.x, k0.y, k0.z, k0.w}, x1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        uint32_t a[4];
                        decode4<FMT>(x0[kk], a[0], a[2]);
                        decode4<FMT>(x1[kk], a[1], a[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816_f16(s[mt][nt], a, qh[nt][kk][0], qh[nt][kk][1]);
                    }
                }
                if constexpr (ALIKE) {
                    const float ksc = __shfl_sync(0xffffffffu, own, one);
                    lsv[0] = __shfl_sync(0xffffffffu, own, 4 + one);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float f[2] = {qs[nt][0] * ksc, qs[nt][1] * ksc};
#pragma unroll
                        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[mt][nt][e] *= f[e & 1];
                    }
                } else {
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt) {
                        const float ksc = __shfl_sync(0xffffffffu, own, mt);
                        lsv[mt] = __shfl_sync(0xffffffffu, own, 4 + mt);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[mt][nt][e] *= qs[nt][e & 1] * ksc;
                    }
                }
            } else {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    const uint4* r0 = reinterpret_cast<const uint4*>(kt + (mt * 16 + rho) * 128 + cq * 32);
                    const uint4* r1 = reinterpret_cast<const uint4*>(kt + (mt * 16 + 8 + rho) * 128 + cq * 32);
                    const uint4 a0 = r0[0], b0 = r0[1], a1 = r1[0], b1 = r1[1];
                    const uint32_t x0[8] = {a0.x, a0.y, a0.z, a0.w, b0.x, b0.y, b0.z, b0.w};
                    const uint32_t x1[8] = {a1.x, a1.y, a1.z, a1.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t a[4] = {x0[2 * kk], x1[2 * kk], x0[2 * kk + 1], x1[2 * kk + 1]};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816(s[mt][nt], a, qb[nt][kk][0], qb[nt][kk][1]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[mt][nt][e] *= P.scale_log2;
                }
            }
            // ---- softmax: m is the maximum of the scores, mv that of scores and value scales ----
            uint32_t pk[4][NT][2];              // weights, [position half]
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float top[4][2];                // maxima of 16 positions, of this lane's
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int r = mt * 16 + hf * 8 + rho;
                        if ((part || !coded) && (r < lo || r >= hi))
                            s[mt][nt][2 * hf] = s[mt][nt][2 * hf + 1] = -INFINITY;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) top[mt][e] = fmaxf(s[mt][nt][e], s[mt][nt][2 + e]);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(fmaxf(top[0][e], top[1][e]), fmaxf(top[2][e], top[3][e])), mw;
                    if constexpr (!ALIKE)
                        mw = fmaxf(fmaxf(top[0][e] + lsv[0], top[1][e] + lsv[1]), fmaxf(top[2][e] + lsv[2], top[3][e] + lsv[3]));
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        if constexpr (!ALIKE) mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, o));
                    }
                    if constexpr (ALIKE) mw = mx + lsv[0];
                    const float n = fmaxf(m[nt][e], mx), nv = fmaxf(mv[nt][e], mw);
                    const float sub = n == -INFINITY ? 0.f : n, subv = nv == -INFINITY ? 0.f : nv;
                    const float c = ex2(m[nt][e] - sub), cv = ex2(mv[nt][e] - subv);
                    m[nt][e] = n;
                    mv[nt][e] = nv;
                    // a weight of V is the weight to base m times f (value scales more than 2^112 apart are
                    // not told apart)
                    const float to = sub - subv + kPShift;
                    float f[4];
                    if constexpr (ALIKE) {
                        f[0] = f[1] = f[2] = f[3] = ex2(min_nan(lsv[0] + to, 126.f));
                    } else {
#pragma unroll
                        for (int mt = 0; mt < 4; ++mt) f[mt] = ex2(min_nan(lsv[mt] + to, 126.f));
                    }
                    float sum = 0.f;
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const float x = ex2(s[mt][nt][2 * hf + e] - sub);
                            sum += x;
                            s[mt][nt][2 * hf + e] = x * f[mt];
                        }
                    l[nt][e] = fmaf(l[nt][e], c, sum);
#pragma unroll
                    for (int md = 0; md < 4; ++md) {
                        oacc[md][nt][e] *= cv;
                        oacc[md][nt][2 + e] *= cv;
                    }
                }
#pragma unroll
                for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const float a = s[mt][nt][2 * hf], b = s[mt][nt][2 * hf + 1];
                        pk[mt][nt][hf] = movmatrix_t(coded ? pack_f16x2(a, b) : pack_bf16x2(a, b));
                    }
            }
            // ---- O^T += V^T P^T: lane (g, c) holds dims 8 g to 8 g + 7 ----
            const int r0 = 2 * cq + (cq & 1), r1 = 2 * cq + 1 - (cq & 1);   // rho of rows 2 cq, 2 cq + 1
            if (coded) {
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    uint32_t a[4][4];           // [pair of dims]
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint8_t* v = vt + (mt * 16 + hf * 8) * 64 + g * 8;
                        const uint2 x = *reinterpret_cast<const uint2*>(v + r0 * 64);
                        const uint2 y = *reinterpret_cast<const uint2*>(v + r1 * 64);
                        decode4<FMT>(__byte_perm(x.x, y.x, 0x5140), a[0][2 * hf], a[0][2 * hf + 1]);
                        decode4<FMT>(__byte_perm(x.x, y.x, 0x7362), a[1][2 * hf], a[1][2 * hf + 1]);
                        decode4<FMT>(__byte_perm(x.y, y.y, 0x5140), a[2][2 * hf], a[2][2 * hf + 1]);
                        decode4<FMT>(__byte_perm(x.y, y.y, 0x7362), a[3][2 * hf], a[3][2 * hf + 1]);
                    }
#pragma unroll
                    for (int md = 0; md < 4; ++md)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816_f16(oacc[md][nt], a[md], pk[mt][nt][0], pk[mt][nt][1]);
                }
            } else {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    uint32_t a[4][4];
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint8_t* v = vt + (mt * 16 + hf * 8) * 128 + g * 16;
                        const uint4 x = *reinterpret_cast<const uint4*>(v + r0 * 128);
                        const uint4 y = *reinterpret_cast<const uint4*>(v + r1 * 128);
                        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int md = 0; md < 4; ++md) {
                            a[md][2 * hf] = __byte_perm(xs[md], ys[md], 0x5410);
                            a[md][2 * hf + 1] = __byte_perm(xs[md], ys[md], 0x7632);
                        }
                    }
#pragma unroll
                    for (int md = 0; md < 4; ++md)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816(oacc[md][nt], a[md], pk[mt][nt][0], pk[mt][nt][1]);
                }
            }
            // ---- the stage is free for the tile after the next ----
            ++done;
            sc[0] = sc[1];
            fence_proxy_async();
            __syncwarp();
            if (ld.i < i1) {
                sc[1] = issue(st);
                ++issued;
            }
            // ---- end of the pair, or of the share ----
            const bool pair_ends = cs.c == cs.per - 1;
            if ((!WHOLE && pair_ends) || cs.i == i1 - 1) {
                const int pair = cs.t * P.nkv + cs.kvh, begin = cs.i - cs.c;
                const bool all = pair_ends && begin >= i0;
                const int w = warp * kKvqCtas + blockIdx.x;
                // WHOLE: into the warp's own stages, where nothing is loaded any more
                float* rows = WHOLE ? reinterpret_cast<float*>(ring) : P.acc + (size_t)(w + pair) * P.G * kPartRow;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], o);
                        const int h = nt * 8 + 2 * cq + e;
                        if (h >= P.G) continue;
                        const float ref = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
                        // sum of weights (to base m) times V, dims 8 g to 8 g + 7
                        const float f = ex2(mv[nt][e] - ref - kPShift) * (all ? 1.f / l[nt][e] : 1.f);
                        float x[8];
#pragma unroll
                        for (int md = 0; md < 4; ++md) {
                            x[2 * md] = oacc[md][nt][e] * f;
                            x[2 * md + 1] = oacc[md][nt][2 + e] * f;
                        }
                        if (all) {
                            const size_t at = (size_t)cs.t * P.nq + cs.kvh * P.G + h;
                            *reinterpret_cast<uint4*>(P.o + at * 64 + 8 * g) =
                                make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                           pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
                            if (P.lse != nullptr && g == 0)
                                P.lse[at] = (m[nt][e] + log2f(l[nt][e])) * 0.6931471805599453f;
                        } else {
                            float* r = rows + h * kPartRow;
                            *reinterpret_cast<float4*>(r + 8 * g) = make_float4(x[0], x[1], x[2], x[3]);
                            *reinterpret_cast<float4*>(r + 8 * g + 4) = make_float4(x[4], x[5], x[6], x[7]);
                            if (g == 0) *reinterpret_cast<float2*>(r + 64) = make_float2(m[nt][e], l[nt][e]);
                        }
                    }
                // the share that begins a pair says where its parts are
                if (!WHOLE && begin >= i0 && lane == 0)
                    P.parts[pair] = make_int2(w + pair, Cuts(S.pre[P.T], kKvqShares).of(begin + cs.per - 1) - w + 1);
                fresh = true;
            }
            next(cs);
            if (!WHOLE && fresh && cs.i < i1) load_q();
        }
        if (failed)                             // loads still in flight
            for (uint32_t n = done; n < issued; ++n)
                (void)mbar_wait(&full[n % kQStages], (n / kQStages) & 1u, 10000000ull);
    }

    if constexpr (WHOLE) {
        __syncthreads();
        const int n = min(cs.per, kKvqWarps), sub = tid & 15;   // sixteen threads to a head
        for (int h = tid >> 4; h < P.G; h += kQThreads / 16) {
            const size_t at = (size_t)cs.t * P.nq + cs.kvh * P.G + h;
            Join j;
            if (n > 1) {
                j.take_all(n, [&](int k) {
                    return reinterpret_cast<const float*>(smem + (size_t)k * kQStages * 2 * kQHalf) + h * kPartRow;
                }, sub);
                j.finish(P, at, sub);
            } else if (n == 0) {
                j.nothing(P, at, sub);
            }
        }
    }
    task_end(ctx);
}

// Joins the parts of the pairs that more than one share has worked on, in the shares' order: `heads` heads
// to a CTA, `pieces` groups of sixteen threads to a head.  Latency: two dependent loads behind the first
// kernel's end, 3.5 us.  It is not launched early: waiting CTAs cost the first kernel 0.7 to 1.3 us.
__global__ void __launch_bounds__(512) kvq_merge_kernel(const __grid_constant__ KvqProblem P, const int heads, const int pieces, const KCtx ctx) {
    __shared__ __align__(16) float rows[32][kPartRow];
    griddep_wait();
    task_begin(ctx);
    const int pair = blockIdx.x, t = pair / P.nkv, kvh = pair - t * P.nkv;
    const int2 q = P.parts[pair];
    const int group = threadIdx.x >> 4, sub = threadIdx.x & 15, piece = group / heads;
    const int h = blockIdx.y * heads + group % heads;
    if (q.y == 1) {                             // written already
        task_end(ctx);
        return;
    }
    const size_t at = (size_t)t * P.nq + kvh * P.G + h;
    Join j;
    if (h < P.G) {
        const float* first = P.acc + ((size_t)q.x * P.G + h) * kPartRow;
        const unsigned step = P.G * kPartRow;
        const int k1 = q.y * (piece + 1) / pieces;
        constexpr int kBatch = 8;
#pragma unroll 1
        for (int k = q.y * piece / pieces; k < k1; k += kBatch) {
            float2 ml[kBatch];
            float4 v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const float* r = first + (size_t)step * min(k + i, k1 - 1);
                ml[i] = __ldcg(reinterpret_cast<const float2*>(r + 64));
                v[i] = __ldcg(reinterpret_cast<const float4*>(r + 4 * sub));
            }
            float top = j.M;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) top = fmaxf(top, ml[i].x);
            j.raise(top);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (k + i < k1) j.take(ml[i], v[i]);
        }
    }
    if (pieces > 1) {
        j.put(rows[group], sub);
        __syncthreads();
        if (piece == 0) j.take_all(pieces - 1, [&](int i) { return &rows[group + (i + 1) * heads][0]; }, sub);
    }
    if (piece == 0 && h < P.G) {
        if (q.y == 0) j.nothing(P, at, sub);
        else j.finish(P, at, sub);
    }
    task_end(ctx);
}

// ---------------------------------------------------------------------------------------
// fold
// ---------------------------------------------------------------------------------------
constexpr int kFThreads = 256;
constexpr int kFRows = 32;                      // positions of a warp
constexpr int kFChunk = kFRows * kFThreads / 32;

__device__ __forceinline__ void load32(const void* p, uint4& a, uint4& b) {
    asm volatile("ld.global.L1::no_allocate.L2::evict_first.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p)
                 : "memory");
}

// A sequence's lengths: folded positions, positions in all, coded ones so far; folded < 0: a length
// out of range, or no room.
struct FoldLen {
    int full, len, held;
};
__device__ __forceinline__ FoldLen fold_len(const FoldProblem& P, int t) {
    FoldLen f;
    f.len = P.kv_len[t];
    f.held = P.held[t];
    f.full = f.len & ~(P.block - 1);
    if (f.len < 0 || f.len > P.cap || f.held < 0 || f.held > P.cap_q || (f.held & (P.block - 1)) ||
        f.full > P.cap_q - f.held)
        f.full = -1;
    return f;
}
__device__ __forceinline__ void fold_lengths_out(const FoldProblem& P, int t, const FoldLen& f) {
    P.len_out[t] = f.full < 0 ? f.len : f.len - f.full;
    P.held_out[t] = f.full < 0 ? f.held : f.held + f.full;
}

// Four bf16 numbers over s as integer codes.  A function, because it is hardly ever called.
__device__ __noinline__ uint32_t divide4(uint32_t a, uint32_t b, float s) {
    uint32_t code = 0;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
        const uint32_t w = j < 2 ? a : b;
        const float y = __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
        code |= (__float2int_rn(__fdiv_rn(y, s)) & 0xff) << (8 * j);
    }
    return code;
}

// One warp holds 32 positions of one (sequence, KV head, tensor) in registers, so that they are read once;
// lane l has the dims 16 (l & 3) to 16 (l & 3) + 15 of rows 8 i + l / 4.  Blocks of more positions join
// their warps' maxima in shared memory; magnitudes compare as integers, which sorts infinities and NaN
// above every number.  The first CTA of a (sequence, KV head, tensor) also moves the rest: fewer than 128
// rows, which it holds in registers before it or anyone else overwrites the rows that it reads.
// Bound by HBM: 64 sequences x 8 heads of up to 8192 positions, 797 MB, 124.4 us in e4m3 (0.95 of a copy's
// rate), 134 in int8; 128 threads to a CTA 137.6.  Short ones are latency (64 x 8 of up to 127: 5.7).
template <int FMT>
__global__ void __launch_bounds__(kFThreads, 4) kvq_fold_kernel(const __grid_constant__ FoldProblem P, const KCtx ctx) {
    __shared__ uint32_t tops[kFThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int chunk = blockIdx.x >> 1, value = blockIdx.x & 1, kvh = blockIdx.y, t = blockIdx.z;
    griddep_wait();
    task_begin(ctx);
    const FoldLen f = fold_len(P, t);
    if (chunk == 0 && value == 0 && kvh == 0 && tid == 0) {
        if (f.full < 0) report(ctx, ST_BOUNDS, (uint32_t)t);
        if (P.len_out != P.kv_len) fold_lengths_out(P, t, f);
    }
    if (f.full < 0 || (chunk > 0 && chunk * kFChunk >= f.full)) {
        task_end(ctx);
        return;
    }
    const size_t pair = (size_t)t * P.nkv + kvh;
    const bf16* src = (value ? P.v : P.k) + pair * P.cap * 64;
    const int p0 = chunk * kFChunk + warp * kFRows;
    const bool live = p0 < f.full;
    const int rows = min(kFRows, f.full - p0);  // a multiple of 16
    uint4 x[4][2];
    uint32_t top[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
        if (live && 8 * i < rows) load32(src + (size_t)(p0 + 8 * i + (lane >> 2)) * 64 + (lane & 3) * 16, x[i][0], x[i][1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
        uint32_t hi = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) hi = __vmaxu2(hi, v[e] & 0x7fff7fffu);
        top[i >> 1] = max(top[i >> 1], max(hi & 0xffffu, hi >> 16));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) top[i] = __reduce_max_sync(0xffffffffu, top[i]);
    if (P.block >= 32) top[0] = top[1] = max(top[0], top[1]);
    // rest rows, before the first chunk's rows are overwritten (in place); at most 127
    const int n_rest = f.len - f.full;
    const bool moves = chunk == 0 && (P.moved || f.full > 0);
    uint4 rest[4];
    if (moves) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = tid + i * kFThreads;  // 16-byte pieces, 8 to a row
            if (e < n_rest * 8) rest[i] = *reinterpret_cast<const uint4*>(src + (size_t)(f.full + (e >> 3)) * 64 + (e & 7) * 8);
        }
    }
    if (P.block >= 64 && lane == 0) tops[warp] = top[0];
    if (P.block >= 64 || moves) __syncthreads();
    if (P.block >= 64) {
        const int n = P.block / kFRows, w0 = warp & ~(n - 1);
        for (int i = 0; i < n; ++i) top[0] = max(top[0], tops[w0 + i]);
        top[1] = top[0];
    }
    if (moves) {
        bf16* dst = (value ? P.v_rest : P.k_rest) + pair * P.cap_rest * 64;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = tid + i * kFThreads;
            if (e < n_rest * 8) *reinterpret_cast<uint4*>(dst + (size_t)(e >> 3) * 64 + (e & 7) * 8) = rest[i];
        }
    }
    if (live) {
        float scale[2], mul[2];
        bool fine[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            fine[i] = top[i] < 0x7f80u;         // no infinity, no NaN
            const float amax = fmaxf(__uint_as_float(top[i] << 16), kKvqSmallest);
            if constexpr (FMT == KVQ_INT8) {
                scale[i] = __fdiv_rn(amax, 127.f);
                mul[i] = __frcp_rn(scale[i]);
            } else {
                // 2^e, the least with amax <= 448 2^e = 1.75 2^(e + 8)
                const uint32_t b = __float_as_uint(amax);
                const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
                scale[i] = pow2i(e);
                mul[i] = pow2i(-e);
            }
        }
        uint8_t* code = (value ? P.vq : P.kq) + (pair * P.cap_q + f.held + p0) * 64;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (8 * i >= rows) break;
            const float s = scale[i >> 1], inv = mul[i >> 1];
            const uint32_t v[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
            uint32_t out[4];
            if constexpr (FMT == KVQ_INT8) {
                // The fp32 quotient by a step of Markstein's iteration ("Computation of elementary functions on
                // the IBM RISC System/6000 processor", 1990): the exact remainder of a close one corrects it.
                // For numbers of 8 significant bits over a 127th of another one the nearest integer is then
                // that of the rounded quotient (all of them: tests/test_kvq_cpu.py); halves between codes
                // are common, amax / 2 is 63.5 of them.  Plus 1.5 2^23 the integer is in the lowest byte.
                // (Caches of 64 sequences x 8 heads, up to 8192 positions: 134 us, 160 with a division where
                // it might matter, 262 with one everywhere in question.)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t t[4];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t w = v[2 * e + j];
                        const float2 y = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
                        float2 z = mul2(y, make_float2(inv, inv));
                        z = fma2(fma2(z, make_float2(-s, -s), y), make_float2(inv, inv), z);
                        z = add2(z, make_float2(12582912.f, 12582912.f));
                        t[2 * j] = __float_as_uint(z.x);
                        t[2 * j + 1] = __float_as_uint(z.y);
                    }
                    out[e] = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
                }
                // remainders that would be subnormal
                if (s < 0x1p-64f)
                    for (int e = 0; e < 4; ++e) out[e] = divide4(v[2 * e], v[2 * e + 1], s);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float y[4] = {__uint_as_float(v[2 * e] << 16), __uint_as_float(v[2 * e] & 0xffff0000u),
                                        __uint_as_float(v[2 * e + 1] << 16), __uint_as_float(v[2 * e + 1] & 0xffff0000u)};
                    uint16_t lo, hi;
                    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[1] * inv), "f"(y[0] * inv));
                    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[3] * inv), "f"(y[2] * inv));
                    out[e] = lo | (uint32_t)hi << 16;
                }
            }
            if (!fine[i >> 1]) out[0] = out[1] = out[2] = out[3] = 0;
            *reinterpret_cast<uint4*>(code + (size_t)(8 * i + (lane >> 2)) * 64 + (lane & 3) * 16) =
                make_uint4(out[0], out[1], out[2], out[3]);
        }
        // the block's first warp, or this one for each of its blocks
        float* to = (value ? P.vs : P.ks) + pair * (P.cap_q / P.block) + (f.held + p0) / P.block;
        if (lane == 0 && (p0 & (P.block - 1)) == 0) {
            to[0] = fine[0] ? scale[0] : __int_as_float(0x7fc00000);
            if (P.block == 16 && rows > 16) to[1] = fine[1] ? scale[1] : __int_as_float(0x7fc00000);
        }
    }
    task_end(ctx);
}

__global__ void __launch_bounds__(512) kvq_fold_len_kernel(const __grid_constant__ FoldProblem P, const KCtx ctx) {
    griddep_wait();
    task_begin(ctx);
    if ((int)threadIdx.x < P.T) fold_lengths_out(P, threadIdx.x, fold_len(P, threadIdx.x));
    task_end(ctx);
}

}  // namespace

int enqueue_kvq_attention(Launcher& L, const KvqProblem& p, const KCtx& c) {
    const size_t smem = 128 + (size_t)kKvqWarps * kQStages * 2 * kQHalf + sizeof(KvqSmem);
    void* args[] = {(void*)&p, (void*)&c};
    // [format][more than 8 heads][whole, else blocks of a tile and more]
    static const void* const kern[2][2][3] = {
        {{(const void*)kvq_attn_kernel<1, KVQ_E4M3, false, false>, (const void*)kvq_attn_kernel<1, KVQ_E4M3, false, true>,
          (const void*)kvq_attn_kernel<1, KVQ_E4M3, true, false>},
         {(const void*)kvq_attn_kernel<2, KVQ_E4M3, false, false>, (const void*)kvq_attn_kernel<2, KVQ_E4M3, false, true>,
          (const void*)kvq_attn_kernel<2, KVQ_E4M3, true, false>}},
        {{(const void*)kvq_attn_kernel<1, KVQ_INT8, false, false>, (const void*)kvq_attn_kernel<1, KVQ_INT8, false, true>,
          (const void*)kvq_attn_kernel<1, KVQ_INT8, true, false>},
         {(const void*)kvq_attn_kernel<2, KVQ_INT8, false, false>, (const void*)kvq_attn_kernel<2, KVQ_INT8, false, true>,
          (const void*)kvq_attn_kernel<2, KVQ_INT8, true, false>}}};
    // A CTA to each pair where none can have many tiles, by capacity (lengths are on the device); the more
    // pairs, the longer the other form takes.  Replayed, a CTA to each and shares with a join: 16 pairs of
    // 512 positions 5.0 and 7.9 us, 1024 6.5 and 8.0, 1536 8.2 and 8.0, 2048 9.2 and 8.0, 4096 14.6 and
    // 8.4; 148 pairs of up to 500 5.1 and 8.3, 1000 6.8 and 8.9, 2000 9.6 and 11.4, 3001 13.2 and 13.1.
    const int pairs = p.T * p.nkv;
    const bool whole = pairs <= kKvqCtas && p.cap / kQTile + p.tail_cap / kQTail <= 24 + pairs / 6;
    const int e = L.launch(kern[p.format][p.G > 8][whole ? 2 : p.block >= kQTile], dim3(whole ? pairs : kKvqCtas), dim3(kQThreads), smem, args, true);
    if (e || whole) return e;
    // Parts of a pair: about kKvqShares / pairs when every sequence is as long; two to four to a group (8
    // pairs of 228 parts, 512 of 5, 148 of 13: with eight to a group 0.1, 0 and 0.5 us more).
    int heads = 1, pieces = 1;
    while (pieces < 32 && pairs * pieces * 4 < kKvqShares) pieces *= 2;
    while (heads * 2 * pieces <= 16 && heads < p.G) heads *= 2;
    void* args2[] = {(void*)&p, (void*)&heads, (void*)&pieces, (void*)&c};
    return L.launch((const void*)kvq_merge_kernel, dim3(pairs, (p.G + heads - 1) / heads), dim3(16 * heads * pieces), 0, args2, true);
}

int enqueue_kvq_fold(Launcher& L, const FoldProblem& p, const KCtx& c) {
    void* args[] = {(void*)&p, (void*)&c};
    const void* f = p.format == KVQ_INT8 ? (const void*)kvq_fold_kernel<KVQ_INT8> : (const void*)kvq_fold_kernel<KVQ_E4M3>;
    const int full = p.cap / p.block * p.block, chunks = full > 0 ? (full + kFChunk - 1) / kFChunk : 1;
    const int e = L.launch(f, dim3(2 * chunks, p.nkv, p.T), dim3(kFThreads), 0, args, true);
    if (e || p.kv_len != p.len_out) return e;
    return L.launch((const void*)kvq_fold_len_kernel, dim3(1), dim3(512), 0, args, true);
}

}  // namespace sgp
