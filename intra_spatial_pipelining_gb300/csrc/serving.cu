// C entry points of the serving operators beside the decode layer: attention over shared
// prefixes, accumulated attention weights, cache eviction, low-rank adapters, norms and rotation of
// queries and keys, caches in 8 bits.  Argument checks, workspace layout and launches; nothing here
// keeps state between calls.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "host.h"

using namespace sgp;

namespace {

enum : uint32_t { OP_PREFIX = 16, OP_WEIGHTS = 17, OP_EVICT = 18, OP_LORA = 19,
                OP_ROPE = 20, OP_FOLD = 21, OP_KVQ = 22 };
constexpr size_t kStatusBytes = 256;  // the status word, at the start of every workspace

bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
bool bad16(const void* p) { return !p || misaligned(p, 16); }
bool bad4(const void* p) { return !p || misaligned(p, 4); }
size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

// whether [a, a + na) and [b, b + nb) share a byte
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

struct HostLauncher : Launcher {
    cudaStream_t s;
    explicit HostLauncher(sgp_stream_t st) : s((cudaStream_t)st) {}
    int launch(const void* func, dim3 grid, dim3 block, size_t smem, void** args,
               bool overlap_ok) override {
        return host_launch(s, func, grid, block, smem, args, overlap_ok);
    }
};

// The head fields of the dimensions (the others are not read).
int check_heads(const sgp_dims* d, bool queries) {
    if (!d) return host_fail_arg("dims is NULL");
    if (d->head_dim != 64) return host_fail_arg("head_dim must be 64");
    if (d->n_kv_heads < 1 || d->n_kv_heads > 1024) return host_fail_arg("n_kv_heads out of range");
    if (queries) {
        if (d->n_q_heads < 1 || d->n_q_heads % d->n_kv_heads)
            return host_fail_arg("n_q_heads must be a positive multiple of n_kv_heads");
        if (d->n_q_heads / d->n_kv_heads > 16)
            return host_fail_arg("more than 16 query heads per KV head");
    }
    return SGP_OK;
}

int check_tokens(int T) {
    return T < 1 || T > kHostMaxTokens ? host_fail_arg("n_tokens must be in [1, 512]") : SGP_OK;
}

// The cache fields of a layer (the weights are not read).  align: of the loads of its rows.
int check_cache(const sgp_dims* d, const sgp_layer* l, int T, bool values, size_t align) {
    if (!l) return host_fail_arg("cache is NULL");
    if (!l->k_cache || misaligned(l->k_cache, align) || (values && (!l->v_cache || misaligned(l->v_cache, align))))
        return host_fail_arg("cache pointer NULL or not aligned (16 bytes for attention, 32 for weights and eviction)");
    if (l->kv_cap < 1) return host_fail_arg("kv_cap must be positive");
    if (l->window < 0) return host_fail_arg("window must be >= 0");
    if ((uint64_t)T * d->n_kv_heads * l->kv_cap >= (1ull << 31))
        return host_fail_arg("KV cache rows exceed 2^31");
    return SGP_OK;
}

int check_workspace(const void* ws, size_t have, size_t need) {
    if (!ws || misaligned(ws, 256)) return host_fail_arg("workspace NULL or not 256-byte aligned");
    if (have < need) return host_fail_arg("workspace too small");
    return SGP_OK;
}

int launched(int e, const char* what) {
    if (e == 0) return SGP_OK;
    if (e == SGP_ERR_INVALID_ARG || e == SGP_ERR_CUDA) return e;
    return host_fail_cuda((cudaError_t)e, what);
}

// ---- attention over shared prefixes ----------------------------------------------------
struct PrefixLayout {
    size_t own_ml, own_acc, parts, pre_ml, pre_acc, total;
    int chunk_log2, S_max, tile_seqs;
};

// Own positions of a work item: the longest that still gives the 64 or so streaming CTAs' 768 warps
// about four items each (a shorter one costs its partial, 2 KB written and read for 32 KB streamed
// at 128 positions).  64 sequences x 8 KV heads of up to 1024 positions beside a prefix of 8192:
// chunks of 1024 left the stream at half its rate.
constexpr int kOwnLogMin = 7, kOwnLogMax = 10;
constexpr size_t kOwnItems = 3000;

size_t own_chunks(size_t pairs, int kv_cap, int log2) { return pairs * (size_t)(((kv_cap - 1) >> log2) + 1); }

int own_chunk_log2(size_t pairs, int kv_cap) {
    int b = kOwnLogMax;
    while (b > kOwnLogMin && own_chunks(pairs, kv_cap, b) < kOwnItems) --b;
    return b;
}

// Room for the chunks of every call with at most so many pairs and positions.  A smaller call may cut
// its caches finer, but a chunk is halved only while there are fewer than kOwnItems, which makes fewer
// than twice as many of them.
size_t own_slots(size_t pairs, int kv_cap) {
    return std::max(own_chunks(pairs, kv_cap, kOwnLogMax),
                    std::min(own_chunks(pairs, kv_cap, kOwnLogMin), 2 * (kOwnItems - 1)));
}

PrefixLayout prefix_layout(const sgp_dims& d, int T, int kv_cap, int n_prefixes) {
    PrefixLayout y;
    const int G = d.n_q_heads / d.n_kv_heads;
    const size_t pairs = (size_t)T * d.n_kv_heads;
    y.chunk_log2 = own_chunk_log2(pairs, kv_cap);
    y.S_max = ((kv_cap - 1) >> y.chunk_log2) + 1;
    y.tile_seqs = kPrefixRows / G;
    size_t off = kStatusBytes;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = al256(off + bytes);
        return o;
    };
    // (every size below grows with T, kv_cap and n_prefixes, so that a workspace serves smaller calls)
    const size_t own_rows = own_slots(pairs, kv_cap) * G;
    y.own_ml = take(own_rows * 2 * 4);
    y.own_acc = take(own_rows * 64 * 4);
    // slots: one per share and tile; a group has a started tile at most beside its full ones
    const size_t groups = n_prefixes < T ? n_prefixes : T;
    const size_t tiles = d.n_kv_heads * (groups + T / y.tile_seqs);
    const size_t slots = n_prefixes > 0 ? kPrefixCtas + tiles : 0;
    y.parts = take(pairs * sizeof(PrefixParts));
    y.pre_ml = take(slots * kPrefixRows * 2 * 4);
    y.pre_acc = take(slots * kPrefixRows * 64 * 4);
    y.total = off;
    return y;
}

int prefix_attention(const sgp_dims* d, const sgp_layer* cache, const sgp_prefix* pre,
                     const int32_t* kv_len, const void* q, void* o, float* lse, int T, void* ws,
                     size_t ws_bytes, sgp_stream_t stream) {
    int r;
    if ((r = check_heads(d, true)) || (r = check_tokens(T)) || (r = check_cache(d, cache, T, true, 16)))
        return r;
    if (bad4(kv_len)) return host_fail_arg("kv_len NULL or not aligned");
    if (bad16(q) || bad16(o)) return host_fail_arg("q or o NULL or not 16-byte aligned");
    if (lse && bad4(lse)) return host_fail_arg("lse not aligned");
    const size_t rows = (size_t)T * d->n_q_heads;
    if (overlap(q, rows * 128, o, rows * 128) && q != o) return host_fail_arg("q and o overlap");
    const int n = pre ? pre->n_prefixes : 0;
    if (n < 0 || n > kPrefixMax) return host_fail_arg("n_prefixes must be in [0, 512]");
    if (n > 0) {
        if (bad16(pre->k) || bad16(pre->v))
            return host_fail_arg("prefix pointer NULL or not 16-byte aligned");
        if (bad4(pre->len) || bad4(pre->prefix_of))
            return host_fail_arg("prefix len or prefix_of NULL or not aligned");
        if (pre->cap < 1) return host_fail_arg("prefix cap must be positive");
        if ((uint64_t)n * d->n_kv_heads * pre->cap >= (1ull << 31))
            return host_fail_arg("prefix rows exceed 2^31");
    }
    const PrefixLayout y = prefix_layout(*d, T, cache->kv_cap, n);
    if ((r = check_workspace(ws, ws_bytes, y.total))) return r;
    if (!host_driver_ready()) return SGP_ERR_UNSUPPORTED;
    uint8_t* w = static_cast<uint8_t*>(ws);
    HostLauncher L(stream);
    const KCtx c = host_ctx(ws, OP_PREFIX);
    PrefixProblem p;
    memset(&p, 0, sizeof(p));
    const uint64_t own_rows = (uint64_t)T * d->n_kv_heads * cache->kv_cap;
    if ((r = host_tmap_pair(&p.tmK, &p.tmV, cache->k_cache, cache->v_cache, 64, own_rows, 64, 64))) return r;
    if (n > 0) {
        const uint64_t pre_rows = (uint64_t)n * d->n_kv_heads * pre->cap;
        if ((r = host_tmap_pair(&p.tmPK, &p.tmPV, pre->k, pre->v, 64, pre_rows, 64, kPrefixKeys))) return r;
        p.prefix = {pre->prefix_of, pre->len, n, pre->cap};
    }
    p.q = static_cast<const bf16*>(q);
    p.kv_len = kv_len;
    p.pre_ml = reinterpret_cast<float*>(w + y.pre_ml);
    p.pre_acc = reinterpret_cast<float*>(w + y.pre_acc);
    p.own_ml = reinterpret_cast<float*>(w + y.own_ml);
    p.own_acc = reinterpret_cast<float*>(w + y.own_acc);
    p.parts = reinterpret_cast<PrefixParts*>(w + y.parts);
    p.o = static_cast<bf16*>(o);
    p.lse = lse;
    p.T = T;
    p.nq = d->n_q_heads;
    p.nkv = d->n_kv_heads;
    p.G = d->n_q_heads / d->n_kv_heads;
    p.kv_cap = cache->kv_cap;
    p.window = cache->window;
    p.tile_seqs = y.tile_seqs;
    p.chunk_log2 = y.chunk_log2;
    p.tile_inv = ((1u << 22) + y.tile_seqs - 1) / y.tile_seqs;
    p.S_max = y.S_max;
    p.scale_log2 = 1.4426950408889634f / sqrtf((float)d->head_dim);
    return launched(enqueue_prefix(L, p, c), "prefix attention");
}

int attention_weights(const sgp_dims* d, const sgp_layer* cache, const int32_t* kv_len,
                      const void* q, const float* lse, float* acc, int T, void* ws,
                      size_t ws_bytes, sgp_stream_t stream) {
    int r;
    if ((r = check_heads(d, true)) || (r = check_tokens(T)) || (r = check_cache(d, cache, T, false, 32)))
        return r;
    if (cache->window != 0) return host_fail_arg("attention weights of a sliding-window layer");
    if (bad4(kv_len) || bad4(lse) || bad4(acc)) return host_fail_arg("kv_len, lse or acc NULL or not aligned");
    if (bad16(q)) return host_fail_arg("q NULL or not 16-byte aligned");
    if ((r = check_workspace(ws, ws_bytes, 64))) return r;
    WeightsProblem p{static_cast<const bf16*>(q), static_cast<const bf16*>(cache->k_cache), lse, kv_len,
                     acc, T, d->n_q_heads, d->n_kv_heads, d->n_q_heads / d->n_kv_heads, cache->kv_cap,
                     1.4426950408889634f / sqrtf((float)d->head_dim)};
    HostLauncher L(stream);
    return launched(enqueue_weights(L, p, host_ctx(ws, OP_WEIGHTS), host_sms()), "attention weights");
}

// ---- eviction ----------------------------------------------------------------------------
size_t evict_bytes(const sgp_dims& d, int T, int budget) {
    return kStatusBytes + al256((size_t)T * 4) + al256((size_t)T * d.n_kv_heads * budget * 4);
}

int kv_evict(const sgp_dims* d, const sgp_layer* from, const sgp_layer* to, const sgp_evict* e,
             const int32_t* kv_len, int32_t* kv_len_out, const float* acc, float* acc_out,
             int32_t* kept, int T, void* ws, size_t ws_bytes, sgp_stream_t stream) {
    int r;
    if ((r = check_heads(d, false)) || (r = check_tokens(T)) ||
        (r = check_cache(d, from, T, true, 32)) || (r = check_cache(d, to, T, true, 32)))
        return r;
    if (!e) return host_fail_arg("policy is NULL");
    if (e->budget < 1 || e->budget > to->kv_cap)
        return host_fail_arg("budget must be in [1, kv_cap of the target]");
    if (e->n_sink < 0 || e->n_recent < 0 || (int64_t)e->n_sink + e->n_recent > e->budget)
        return host_fail_arg("n_sink + n_recent must be in [0, budget]");
    if (bad4(kv_len) || bad4(kv_len_out) || bad4(acc) || bad4(acc_out) || (kept && bad4(kept)))
        return host_fail_arg("kv_len, acc or kept NULL or not aligned");
    if (kv_len != kv_len_out && overlap(kv_len, (size_t)T * 4, kv_len_out, (size_t)T * 4))
        return host_fail_arg("kv_len and kv_len_out overlap without being the same");
    const size_t pairs = (size_t)T * d->n_kv_heads;
    const size_t n_from = pairs * from->kv_cap, n_to = pairs * to->kv_cap;
    const bool in_place = from->k_cache == to->k_cache;
    if (in_place) {
        if (from->v_cache != to->v_cache || acc != acc_out || from->kv_cap != to->kv_cap)
            return host_fail_arg("in place: k, v, acc and kv_cap must all be the same");
    } else if (overlap(from->k_cache, n_from * 128, to->k_cache, n_to * 128) ||
               overlap(from->v_cache, n_from * 128, to->v_cache, n_to * 128) ||
               overlap(from->k_cache, n_from * 128, to->v_cache, n_to * 128) ||
               overlap(from->v_cache, n_from * 128, to->k_cache, n_to * 128) ||
               overlap(acc, n_from * 4, acc_out, n_to * 4)) {
        return host_fail_arg("source and target overlap");
    }
    if (overlap(to->k_cache, n_to * 128, to->v_cache, n_to * 128))
        return host_fail_arg("the target's k and v overlap");
    if ((r = check_workspace(ws, ws_bytes, evict_bytes(*d, T, e->budget)))) return r;
    uint8_t* w = static_cast<uint8_t*>(ws);
    EvictProblem p;
    memset(&p, 0, sizeof(p));
    p.k = static_cast<const bf16*>(from->k_cache);
    p.v = static_cast<const bf16*>(from->v_cache);
    p.acc = acc;
    p.kv_len = kv_len;
    p.k_out = static_cast<bf16*>(to->k_cache);
    p.v_out = static_cast<bf16*>(to->v_cache);
    p.acc_out = acc_out;
    p.kv_len_out = kv_len_out;
    p.count = reinterpret_cast<int*>(w + kStatusBytes);
    p.kept = reinterpret_cast<int*>(w + kStatusBytes + al256((size_t)T * 4));
    p.user_kept = kept;
    p.T = T;
    p.nkv = d->n_kv_heads;
    p.cap = from->kv_cap;
    p.cap_out = to->kv_cap;
    p.budget = e->budget;
    p.n_sink = e->n_sink;
    p.n_recent = e->n_recent;
    p.in_place = in_place;
    HostLauncher L(stream);
    return launched(enqueue_evict(L, p, host_ctx(ws, OP_EVICT)), "eviction");
}

int lora_apply(const sgp_lora* a, const int32_t* adapter_of, const void* x, int64_t ld_x,
               const void* y_in, int64_t ld_y_in, void* y_out, int64_t ld_y_out, int T, void* ws,
               size_t ws_bytes, sgp_stream_t stream) {
    int r;
    if (!a) return host_fail_arg("adapters are NULL");
    if ((r = check_tokens(T))) return r;
    if (a->n_adapters < 1 || a->n_adapters > 4096) return host_fail_arg("n_adapters must be in [1, 4096]");
    if (a->in < 32 || a->in > (1 << 20) || a->in % 32 || a->out < 32 || a->out > (1 << 20) || a->out % 32)
        return host_fail_arg("in and out must be multiples of 32, up to 2^20");
    if (a->max_rank < 8 || a->max_rank > 128 || a->max_rank % 8)
        return host_fail_arg("max_rank must be a multiple of 8 in [8, 128]");
    if (bad16(a->a) || bad16(a->b) || bad16(x) || bad16(y_in) || bad16(y_out))
        return host_fail_arg("pointer NULL or not 16-byte aligned");
    if (bad4(adapter_of) || (a->scale && bad4(a->scale)) || (a->rank && bad4(a->rank)))
        return host_fail_arg("adapter_of NULL, or an index or scale pointer not aligned");
    if (ld_x < a->in || ld_y_in < a->out || ld_y_out < a->out || ld_x % 8 || ld_y_in % 8 || ld_y_out % 8 ||
        ld_x > (1ll << 40) || ld_y_in > (1ll << 40) || ld_y_out > (1ll << 40))
        return host_fail_arg("row strides must be multiples of 8, at least the row length");
    auto span = [&](int64_t ld, int n) { return ((size_t)(T - 1) * ld + n) * 2; };
    if (y_in == y_out ? ld_y_in != ld_y_out
                      : overlap(y_in, span(ld_y_in, a->out), y_out, span(ld_y_out, a->out)))
        return host_fail_arg("y_in and y_out overlap");
    if (overlap(x, span(ld_x, a->in), y_out, span(ld_y_out, a->out)))
        return host_fail_arg("x and y_out overlap");
    if ((r = check_workspace(ws, ws_bytes, 64))) return r;
    LoraProblem p{static_cast<const bf16*>(x), static_cast<const bf16*>(y_in), static_cast<bf16*>(y_out),
                  static_cast<const bf16*>(a->a), static_cast<const bf16*>(a->b), a->scale, a->rank,
                  adapter_of, ld_x, ld_y_in, ld_y_out, T, a->n_adapters, a->in, a->out, a->max_rank};
    HostLauncher L(stream);
    return launched(enqueue_lora(L, p, host_ctx(ws, OP_LORA)), "adapters");
}

// ---- norms and rotation ------------------------------------------------------------------
// Whether rows of `wa` elements, lda apart, share a byte with rows of `wb`, ldb apart (T of each).
// Rows of one stride may interleave; of two strides only the whole spans are compared.
bool rows_overlap(const void* a, int64_t lda, int64_t wa, const void* b, int64_t ldb, int64_t wb, int T) {
    if (!overlap(a, ((size_t)(T - 1) * lda + wa) * 2, b, ((size_t)(T - 1) * ldb + wb) * 2)) return false;
    if (lda != ldb) return true;
    const int64_t step = 2 * lda;
    const int64_t off = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
    const int64_t d = ((off % step) + step) % step;     // b's rows begin d bytes behind a's
    return d < 2 * wa || d + 2 * wb > step;
}

int check_rows(const void* p, int64_t ld, int width, const char* what) {
    if (bad16(p)) return host_fail_arg(what);
    if (ld < width || ld % 8 || ld > (1ll << 40)) return host_fail_arg("row strides must be multiples of 8, at least the row length");
    return SGP_OK;
}

int qk_rope(const sgp_dims* d, const sgp_rope* rope, const void* g_q, const void* g_k, float eps,
            const int32_t* pos, const void* q, int64_t ld_q, void* q_out, int64_t ld_q_out, const void* k,
            int64_t ld_k, void* k_out, int64_t ld_k_out, const void* v, int64_t ld_v,
            const sgp_layer* cache, bool append, int n_seqs, const int32_t* seq, const int32_t* slot, int T,
            void* ws, size_t ws_bytes, sgp_stream_t stream) {
    int r;
    if ((r = check_heads(d, true))) return r;
    if (!rope) return host_fail_arg("rope is NULL");
    if (rope->rot_dim < 16 || rope->rot_dim > 64 || rope->rot_dim % 16) return host_fail_arg("rot_dim must be 16, 32, 48 or 64");
    if (rope->layout != SGP_ROPE_HALF && rope->layout != SGP_ROPE_INTERLEAVED) return host_fail_arg("unknown layout of the rotation");
    if (!std::isfinite(rope->amplitude)) return host_fail_arg("amplitude is not finite");
    if (!(eps >= 0.f) || std::isinf(eps)) return host_fail_arg("eps must be >= 0 and finite");
    if (T < 1 || T > (1 << 20)) return host_fail_arg("n_tokens must be in [1, 2^20]");
    if ((g_q && bad16(g_q)) || (g_k && bad16(g_k))) return host_fail_arg("g_q or g_k not 16-byte aligned");
    if (bad4(pos)) return host_fail_arg("pos NULL or not aligned");
    const int wq = d->n_q_heads * 64, wk = d->n_kv_heads * 64;
    if (!q != !q_out) return host_fail_arg("q without q_out, or q_out without q");
    if (q && ((r = check_rows(q, ld_q, wq, "q not 16-byte aligned")) || (r = check_rows(q_out, ld_q_out, wq, "q_out not 16-byte aligned"))))
        return r;
    if (k && (r = check_rows(k, ld_k, wk, "k not 16-byte aligned"))) return r;
    if (v && (r = check_rows(v, ld_v, wk, "v not 16-byte aligned"))) return r;
    if (append) {
        if (!cache) return host_fail_arg("cache is NULL");
        if (n_seqs < 1) return host_fail_arg("n_seqs must be positive");
        if (bad16(cache->k_cache) || (v && bad16(cache->v_cache)) || cache->kv_cap < 1)
            return host_fail_arg("cache pointer NULL or not 16-byte aligned, or kv_cap not positive");
        const uint64_t per = (uint64_t)d->n_kv_heads * cache->kv_cap;
        if (per >= (1ull << 31) || per * n_seqs >= (1ull << 31)) return host_fail_arg("KV cache rows exceed 2^31");
        if (bad4(slot) || (seq && bad4(seq))) return host_fail_arg("slot NULL, or slot or seq not aligned");
        const size_t bytes = (size_t)per * n_seqs * 128;
        const struct { const void* p; int64_t ld; int w; } rows[] = {{q, ld_q, wq}, {q_out, ld_q_out, wq}, {k, ld_k, wk}, {v, ld_v, wk}};
        for (const auto& x : rows)
            for (const void* c : {(const void*)cache->k_cache, v ? (const void*)cache->v_cache : nullptr})
                if (x.p && c && overlap(x.p, ((size_t)(T - 1) * x.ld + x.w) * 2, c, bytes))
                    return host_fail_arg("rows and caches overlap");
        if (v && overlap(cache->k_cache, bytes, cache->v_cache, bytes)) return host_fail_arg("k_cache and v_cache overlap");
    } else {
        if (!k != !k_out) return host_fail_arg("k without k_out, or k_out without k");
        if (!q && !k) return host_fail_arg("neither q nor k");
        if (k && (r = check_rows(k_out, ld_k_out, wk, "k_out not 16-byte aligned"))) return r;
        if (k && !(k == k_out && ld_k == ld_k_out) && rows_overlap(k, ld_k, wk, k_out, ld_k_out, wk, T))
            return host_fail_arg("k and k_out overlap");
        if (q && k && (rows_overlap(q, ld_q, wq, k_out, ld_k_out, wk, T) || rows_overlap(q_out, ld_q_out, wq, k_out, ld_k_out, wk, T)))
            return host_fail_arg("k_out overlaps q or q_out");
    }
    if (q && !(q == q_out && ld_q == ld_q_out) && rows_overlap(q, ld_q, wq, q_out, ld_q_out, wq, T))
        return host_fail_arg("q and q_out overlap");
    if (q && ((k && rows_overlap(k, ld_k, wk, q_out, ld_q_out, wq, T)) || (v && rows_overlap(v, ld_v, wk, q_out, ld_q_out, wq, T))))
        return host_fail_arg("q_out overlaps k or v");
    if ((r = check_workspace(ws, ws_bytes, 64))) return r;
    RopeProblem p;
    memset(&p, 0, sizeof(p));
    for (int i = 0; i < rope->rot_dim / 2; ++i) {
        if (!std::isfinite(rope->freq[i])) return host_fail_arg("a frequency is not finite");
        double turn = rope->freq[i] * 0.15915494309189533577;   // 1 / 2 pi
        turn -= std::floor(turn);                               // in [0, 1]
        p.turns[i] = turn < 1.0 ? (unsigned long long)(turn * 18446744073709551616.0) : 0;
    }
    p.pos = pos;
    p.q = static_cast<const bf16*>(q);
    p.q_out = static_cast<bf16*>(q_out);
    p.k = static_cast<const bf16*>(k);
    p.k_out = static_cast<bf16*>(k_out);
    p.v = static_cast<const bf16*>(v);
    p.g_q = static_cast<const bf16*>(g_q);
    p.g_k = static_cast<const bf16*>(g_k);
    if (append) {
        p.k_cache = static_cast<bf16*>(cache->k_cache);
        p.v_cache = static_cast<bf16*>(cache->v_cache);
        p.cap = cache->kv_cap;
    }
    p.seq = seq;
    p.slot = slot;
    p.ld_q = ld_q;
    p.ld_q_out = ld_q_out;
    p.ld_k = ld_k;
    p.ld_k_out = ld_k_out;
    p.ld_v = ld_v;
    p.T = T;
    p.nq = d->n_q_heads;
    p.nkv = d->n_kv_heads;
    p.n_seqs = n_seqs;
    p.rot = rope->rot_dim;
    p.interleaved = rope->layout == SGP_ROPE_INTERLEAVED;
    p.eps = eps;
    p.amplitude = rope->amplitude;
    HostLauncher L(stream);
    return launched(enqueue_qk_rope(L, p, host_ctx(ws, OP_ROPE), host_sms()), "norms and rotation");
}

int rope_init(sgp_rope* rope, int rot_dim, int layout, double theta, int scaling, double factor,
              double context, double turns_low, double turns_high, float amplitude) {
    const double two_pi = 6.28318530717958647693;
    if (!rope) return host_fail_arg("rope is NULL");
    if (rot_dim < 16 || rot_dim > 64 || rot_dim % 16) return host_fail_arg("rot_dim must be 16, 32, 48 or 64");
    if (layout != SGP_ROPE_HALF && layout != SGP_ROPE_INTERLEAVED) return host_fail_arg("unknown layout of the rotation");
    if (scaling < SGP_ROPE_PLAIN || scaling > SGP_ROPE_BY_INDEX) return host_fail_arg("unknown scaling");
    if (!(theta > 1.0) || std::isinf(theta)) return host_fail_arg("theta must be above 1");
    if (!std::isfinite(amplitude)) return host_fail_arg("amplitude is not finite");
    if (scaling != SGP_ROPE_PLAIN && (!(factor > 0.0) || std::isinf(factor))) return host_fail_arg("factor must be positive");
    if (scaling >= SGP_ROPE_BY_TURNS &&
        (!(context > 0.0) || std::isinf(context) || !(turns_low > 0.0) || !(turns_high > turns_low) || std::isinf(turns_high)))
        return host_fail_arg("context must be positive and 0 < turns_low < turns_high");
    memset(rope, 0, sizeof(*rope));
    rope->rot_dim = rot_dim;
    rope->layout = layout;
    rope->amplitude = amplitude;
    // the index at which a pair makes `t` turns in the context
    auto index_of = [&](double t) { return rot_dim / 2 * std::log(context / (two_pi * t)) / std::log(theta); };
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = std::pow(theta, -2.0 * i / rot_dim);
        double keep = scaling == SGP_ROPE_PLAIN ? 1.0 : 0.0;
        if (scaling == SGP_ROPE_BY_TURNS)
            keep = (context * f / two_pi - turns_low) / (turns_high - turns_low);
        else if (scaling == SGP_ROPE_BY_INDEX)
            keep = 1.0 - (i - index_of(turns_high)) / (index_of(turns_low) - index_of(turns_high));
        keep = std::min(1.0, std::max(0.0, keep));
        rope->freq[i] = keep == 1.0 ? f : f * keep + f / factor * (1.0 - keep);
    }
    return SGP_OK;
}

// ---- caches in 8 bits --------------------------------------------------------------------
int check_kvq(const sgp_dims* d, const sgp_kvq* c, int T) {
    if (!c) return host_fail_arg("the 8-bit cache is NULL");
    if (bad16(c->k) || bad16(c->v)) return host_fail_arg("codes NULL or not 16-byte aligned");
    if (bad4(c->k_scale) || bad4(c->v_scale)) return host_fail_arg("scales NULL or not aligned");
    if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128)
        return host_fail_arg("block must be 16, 32, 64 or 128");
    if (c->cap < c->block || c->cap % c->block) return host_fail_arg("cap must be a positive multiple of block");
    if (c->format != SGP_KVQ_E4M3 && c->format != SGP_KVQ_INT8) return host_fail_arg("unknown format of the codes");
    if ((uint64_t)T * d->n_kv_heads * c->cap >= (1ull << 31)) return host_fail_arg("rows of codes exceed 2^31");
    return SGP_OK;
}

int kvq_fold(const sgp_dims* d, const sgp_layer* from, const sgp_kvq* to, const sgp_layer* rest,
             const int32_t* kv_len, const int32_t* kvq_len, int32_t* kv_len_out, int32_t* kvq_len_out, int T,
             void* ws, size_t ws_bytes, sgp_stream_t stream) {
    int r;
    if ((r = check_heads(d, false)) || (r = check_tokens(T)) || (r = check_cache(d, from, T, true, 32)) ||
        (r = check_cache(d, rest, T, true, 16)) || (r = check_kvq(d, to, T)))
        return r;
    if (bad4(kv_len) || bad4(kvq_len) || bad4(kv_len_out) || bad4(kvq_len_out))
        return host_fail_arg("a length array is NULL or not aligned");
    const size_t n_len = (size_t)T * 4;
    const bool same = kv_len == kv_len_out && kvq_len == kvq_len_out;
    if (overlap(kv_len, n_len, kvq_len, n_len) || overlap(kv_len_out, n_len, kvq_len_out, n_len) ||
        (!same && (overlap(kv_len, n_len, kv_len_out, n_len) || overlap(kvq_len, n_len, kvq_len_out, n_len) ||
                   overlap(kv_len, n_len, kvq_len_out, n_len) || overlap(kvq_len, n_len, kv_len_out, n_len))))
        return host_fail_arg("length arrays overlap: both in place, or all apart");
    const size_t pairs = (size_t)T * d->n_kv_heads;
    const size_t n_from = pairs * from->kv_cap * 128, n_rest = pairs * rest->kv_cap * 128;
    const size_t n_code = pairs * to->cap * 64, n_scale = pairs * (to->cap / to->block) * 4;
    const bool in_place = from->k_cache == rest->k_cache;
    if (in_place) {
        if (from->v_cache != rest->v_cache || from->kv_cap != rest->kv_cap)
            return host_fail_arg("in place: k, v and kv_cap must all be the same");
    } else if (rest->kv_cap < std::min(to->block - 1, from->kv_cap)) {
        return host_fail_arg("no room for the rest");
    }
    // what is written overlaps nothing else; from's k and v may be one cache unless in place
    const struct { const void* p; size_t n; } all[] = {{from->k_cache, n_from}, {from->v_cache, n_from},
        {to->k, n_code}, {to->v, n_code}, {to->k_scale, n_scale}, {to->v_scale, n_scale},
        {rest->k_cache, n_rest}, {rest->v_cache, n_rest}};
    const int count = in_place ? 6 : 8;
    for (int i = 0; i < count; ++i)
        for (int j = std::max(i + 1, in_place ? 1 : 2); j < count; ++j)
            if (overlap(all[i].p, all[i].n, all[j].p, all[j].n)) return host_fail_arg("caches, codes or scales overlap");
    if ((r = check_workspace(ws, ws_bytes, 64))) return r;
    FoldProblem p{static_cast<const bf16*>(from->k_cache), static_cast<const bf16*>(from->v_cache),
                  static_cast<uint8_t*>(to->k), static_cast<uint8_t*>(to->v), to->k_scale, to->v_scale,
                  static_cast<bf16*>(rest->k_cache), static_cast<bf16*>(rest->v_cache), kv_len, kvq_len,
                  kv_len_out, kvq_len_out, T, d->n_kv_heads, from->kv_cap, to->cap, rest->kv_cap, to->block,
                  to->format == SGP_KVQ_INT8 ? KVQ_INT8 : KVQ_E4M3, !in_place};
    HostLauncher L(stream);
    return launched(enqueue_kvq_fold(L, p, host_ctx(ws, OP_FOLD)), "fold");
}

size_t kvq_parts(const sgp_dims& d, int T) { return al256((size_t)T * d.n_kv_heads * sizeof(int2)); }

size_t kvq_bytes(const sgp_dims& d, int T) {
    const size_t slots = kKvqShares + (size_t)T * d.n_kv_heads;
    return kStatusBytes + kvq_parts(d, T) + slots * (d.n_q_heads / d.n_kv_heads) * kPartRow * 4;
}

int kvq_attention(const sgp_dims* d, const sgp_kvq* kvq, const int32_t* kvq_len, const sgp_layer* cache,
                  const int32_t* kv_len, const void* q, void* o, float* lse, int T, void* ws, size_t ws_bytes,
                  sgp_stream_t stream) {
    int r;
    if ((r = check_heads(d, true)) || (r = check_tokens(T)) || (r = check_kvq(d, kvq, T))) return r;
    if (cache && (r = check_cache(d, cache, T, true, 16))) return r;
    if (cache && (int64_t)kvq->cap + cache->kv_cap >= (1ll << 31)) return host_fail_arg("positions of a sequence exceed 2^31");
    if (bad4(kvq_len) || (cache && bad4(kv_len))) return host_fail_arg("kvq_len or kv_len NULL or not aligned");
    if (bad16(q) || bad16(o)) return host_fail_arg("q or o NULL or not 16-byte aligned");
    if (lse && bad4(lse)) return host_fail_arg("lse not aligned");
    const size_t rows = (size_t)T * d->n_q_heads;
    if (q != o && overlap(q, rows * 128, o, rows * 128)) return host_fail_arg("q and o overlap");
    if ((r = check_workspace(ws, ws_bytes, kvq_bytes(*d, T)))) return r;
    uint8_t* w = static_cast<uint8_t*>(ws);
    KvqProblem p;
    memset(&p, 0, sizeof(p));
    p.k = static_cast<const uint8_t*>(kvq->k);
    p.v = static_cast<const uint8_t*>(kvq->v);
    p.ks = kvq->k_scale;
    p.vs = kvq->v_scale;
    p.held = kvq_len;
    if (cache) {
        p.tk = static_cast<const bf16*>(cache->k_cache);
        p.tv = static_cast<const bf16*>(cache->v_cache);
        p.kv_len = kv_len;
        p.tail_cap = cache->kv_cap;
        p.window = cache->window;
    }
    p.q = static_cast<const bf16*>(q);
    p.o = static_cast<bf16*>(o);
    p.lse = lse;
    p.parts = reinterpret_cast<int2*>(w + kStatusBytes);
    p.acc = reinterpret_cast<float*>(w + kStatusBytes + kvq_parts(*d, T));
    p.T = T;
    p.nq = d->n_q_heads;
    p.nkv = d->n_kv_heads;
    p.G = d->n_q_heads / d->n_kv_heads;
    p.cap = kvq->cap;
    p.block = kvq->block;
    while ((1 << p.block_log2) < p.block) ++p.block_log2;
    p.format = kvq->format == SGP_KVQ_INT8 ? KVQ_INT8 : KVQ_E4M3;
    p.scale_log2 = 1.4426950408889634f / sqrtf((float)d->head_dim);
    HostLauncher L(stream);
    return launched(enqueue_kvq_attention(L, p, host_ctx(ws, OP_KVQ)), "attention over an 8-bit cache");
}

// No exception leaves a C entry point (recording an error text allocates).
template <typename F>
int guarded(F f) {
    try {
        return f();
    } catch (...) {
        return SGP_ERR_OOM;
    }
}

}  // namespace

// =======================================================================================
// C ABI
// =======================================================================================
extern "C" size_t sgp_prefix_attention_workspace_bytes(const sgp_dims* d, int n_tokens,
                                                       int kv_cap, int n_prefixes) {
    size_t bytes = 0;
    guarded([&] {
        if (check_heads(d, true) == SGP_OK && check_tokens(n_tokens) == SGP_OK && kv_cap >= 1 &&
            n_prefixes >= 0 && n_prefixes <= kPrefixMax)
            bytes = prefix_layout(*d, n_tokens, kv_cap, n_prefixes).total;
        return SGP_OK;
    });
    return bytes;
}

extern "C" int sgp_prefix_attention(const sgp_dims* dims, const sgp_layer* cache,
                                    const sgp_prefix* prefix, const int32_t* kv_len, const void* q,
                                    void* o, float* lse, int n_tokens, void* workspace,
                                    size_t ws_bytes, sgp_stream_t stream) {
    return guarded([&] {
        return prefix_attention(dims, cache, prefix, kv_len, q, o, lse, n_tokens, workspace, ws_bytes,
                                stream);
    });
}

extern "C" int sgp_attention_weights(const sgp_dims* dims, const sgp_layer* cache,
                                     const int32_t* kv_len, const void* q, const float* lse,
                                     float* acc, int n_tokens, void* workspace, size_t ws_bytes,
                                     sgp_stream_t stream) {
    return guarded([&] {
        return attention_weights(dims, cache, kv_len, q, lse, acc, n_tokens, workspace, ws_bytes, stream);
    });
}

extern "C" size_t sgp_kv_evict_workspace_bytes(const sgp_dims* d, int n_tokens, int budget) {
    size_t bytes = 0;
    guarded([&] {
        if (check_heads(d, false) == SGP_OK && check_tokens(n_tokens) == SGP_OK && budget >= 1)
            bytes = evict_bytes(*d, n_tokens, budget);
        return SGP_OK;
    });
    return bytes;
}

extern "C" int sgp_kv_evict(const sgp_dims* dims, const sgp_layer* from, const sgp_layer* to,
                            const sgp_evict* policy, const int32_t* kv_len, int32_t* kv_len_out,
                            const float* acc, float* acc_out, int32_t* kept, int n_tokens,
                            void* workspace, size_t ws_bytes, sgp_stream_t stream) {
    return guarded([&] {
        return kv_evict(dims, from, to, policy, kv_len, kv_len_out, acc, acc_out, kept, n_tokens,
                        workspace, ws_bytes, stream);
    });
}

extern "C" int sgp_lora_apply(const sgp_lora* lora, const int32_t* adapter_of, const void* x,
                              int64_t ld_x, const void* y_in, int64_t ld_y_in, void* y_out,
                              int64_t ld_y_out, int n_tokens, void* workspace, size_t ws_bytes,
                              sgp_stream_t stream) {
    return guarded([&] {
        return lora_apply(lora, adapter_of, x, ld_x, y_in, ld_y_in, y_out, ld_y_out, n_tokens, workspace,
                          ws_bytes, stream);
    });
}

extern "C" int sgp_rope_init(sgp_rope* rope, int rot_dim, int layout, double theta, int scaling,
                             double factor, double context, double turns_low, double turns_high,
                             float amplitude) {
    return guarded([&] {
        return rope_init(rope, rot_dim, layout, theta, scaling, factor, context, turns_low, turns_high,
                         amplitude);
    });
}

extern "C" int sgp_qk_rope(const sgp_dims* dims, const sgp_rope* rope, const void* g_q, const void* g_k,
                           float eps, const int32_t* pos, const void* q, int64_t ld_q, void* q_out,
                           int64_t ld_q_out, const void* k, int64_t ld_k, void* k_out, int64_t ld_k_out,
                           int n_tokens, void* workspace, size_t ws_bytes, sgp_stream_t stream) {
    return guarded([&] {
        return qk_rope(dims, rope, g_q, g_k, eps, pos, q, ld_q, q_out, ld_q_out, k, ld_k, k_out, ld_k_out,
                       nullptr, 0, nullptr, false, 0, nullptr, nullptr, n_tokens, workspace, ws_bytes,
                       stream);
    });
}

extern "C" int sgp_qk_rope_append(const sgp_dims* dims, const sgp_rope* rope, const void* g_q,
                                  const void* g_k, float eps, const int32_t* pos, const void* q,
                                  int64_t ld_q, void* q_out, int64_t ld_q_out, const void* k, int64_t ld_k,
                                  const void* v, int64_t ld_v, const sgp_layer* cache, int n_seqs,
                                  const int32_t* seq, const int32_t* slot, int n_tokens, void* workspace,
                                  size_t ws_bytes, sgp_stream_t stream) {
    return guarded([&] {
        return qk_rope(dims, rope, g_q, g_k, eps, pos, q, ld_q, q_out, ld_q_out, k, ld_k, nullptr, 0, v, ld_v,
                       cache, true, n_seqs, seq, slot, n_tokens, workspace, ws_bytes, stream);
    });
}

extern "C" int sgp_kvq_fold(const sgp_dims* dims, const sgp_layer* from, const sgp_kvq* to,
                            const sgp_layer* rest, const int32_t* kv_len, const int32_t* kvq_len,
                            int32_t* kv_len_out, int32_t* kvq_len_out, int n_tokens, void* workspace,
                            size_t ws_bytes, sgp_stream_t stream) {
    return guarded([&] {
        return kvq_fold(dims, from, to, rest, kv_len, kvq_len, kv_len_out, kvq_len_out, n_tokens, workspace,
                        ws_bytes, stream);
    });
}

extern "C" size_t sgp_kvq_attention_workspace_bytes(const sgp_dims* d, int n_tokens) {
    size_t bytes = 0;
    guarded([&] {
        if (check_heads(d, true) == SGP_OK && check_tokens(n_tokens) == SGP_OK)
            bytes = kvq_bytes(*d, n_tokens);
        return SGP_OK;
    });
    return bytes;
}

extern "C" int sgp_kvq_attention(const sgp_dims* dims, const sgp_kvq* kvq, const int32_t* kvq_len,
                                 const sgp_layer* cache, const int32_t* kv_len, const void* q, void* o,
                                 float* lse, int n_tokens, void* workspace, size_t ws_bytes,
                                 sgp_stream_t stream) {
    return guarded([&] {
        return kvq_attention(dims, kvq, kvq_len, cache, kv_len, q, o, lse, n_tokens, workspace, ws_bytes,
                             stream);
    });
}
