// Problem descriptions of the serving operators and their enqueue functions.
#pragma once

#include "kernels.h"

namespace sgp {

// Prefixes that sequences of a batch share (lengths and membership as device arrays).
struct PrefixRef {
    const int* of;          // [T]: prefix of a sequence, -1: none
    const int* len;         // [n]
    int n, cap;
};

// Attention of the batch's query heads over the prefixes they share and over the sequences' own
// caches, in one launch of kPrefixCtas CTAs of which some take the prefixes and the others the own
// caches (split by the two parts' work, see k_prefix.cu); every part leaves partials.
//
// Prefixes: sequences with the same prefix form a group; a row is one (sequence, query head) of
// the group and KV head.  A tile is `tile_seqs` sequences' rows (at most kPrefixRows), a step is
// one tile against kPrefixKeys positions.  The steps of all (group, KV head, tile) in order, with
// some units for the beginning of each tile, are cut into equal shares, one per CTA; share s's part
// of tile i leaves its partial in slot s + i.
// Own caches: chunks of 2^chunk_log2 positions of a (sequence, KV head), equal runs of them to a warp.
constexpr int kPrefixRows = 256;
constexpr int kPrefixKeys = 128;
// Fixed, so that results never depend on the SM count: one per SM of a 152-SM part.
constexpr int kPrefixCtas = 152;
constexpr int kPrefixMax = 512;     // sequences, and prefixes, per call

// The parts of a (sequence, KV head): n_pre slots from `slot` on, the sequence's rows from `row`
// on in each, and n_own own chunks.
struct PrefixParts {
    int slot, row, n_pre, n_own;
};

struct PrefixProblem {
    CUtensorMap tmPK, tmPV; // prefixes as 2-D [n * nkv * cap][64], box {64, kPrefixKeys}, SW128
    CUtensorMap tmK, tmV;   // own caches as 2-D [T * nkv * kv_cap][64], box {64, 64}, SW128
    const bf16* q;          // [T][nq * 64]
    const int* kv_len;      // [T]
    PrefixRef prefix;       // n = 0: none
    float* pre_ml;          // [slot][kPrefixRows][2]  (max, sum)
    float* pre_acc;         // [slot][kPrefixRows][64]
    float* own_ml;          // [T * nkv][S_max][G][2]
    float* own_acc;         // [T * nkv][S_max][G][64]
    PrefixParts* parts;     // [T * nkv]
    bf16* o;                // [T][nq * 64]
    float* lse;             // [T][nq] or NULL
    int T, nq, nkv, G, kv_cap, window, tile_seqs, chunk_log2, S_max;
    unsigned tile_inv;      // 2^22 / tile_seqs, rounded up
    float scale_log2;
};

// acc[t][j][p] += sum over the group's heads of exp(scale q.k_p - lse)
struct WeightsProblem {
    const bf16* q;          // [T][nq * 64]
    const bf16* k;          // [T][nkv][cap][64]
    const float* lse;       // [T][nq]
    const int* kv_len;      // [T]
    float* acc;             // [T][nkv][cap]
    int T, nq, nkv, G, cap;
    float scale_log2;
};

// Which positions stay, then the move of their rows.
struct EvictProblem {
    const bf16* k;          // [T][nkv][cap][64]
    const bf16* v;
    const float* acc;       // [T][nkv][cap]
    const int* kv_len;      // [T]
    bf16* k_out;            // [T][nkv][cap_out][64]
    bf16* v_out;
    float* acc_out;         // [T][nkv][cap_out]
    int* kv_len_out;        // [T]
    int* kept;              // [T][nkv][budget] positions in order
    int* user_kept;         // the same, filled up with -1, or NULL
    int* count;             // [T] positions that stay, -1: a length out of range
    int T, nkv, cap, cap_out, budget, n_sink, n_recent;
    int in_place;
};

// y_out = y_in + scale_a B_a (A_a x), a = the sequence's adapter
struct LoraProblem {
    const bf16* x;          // [T] rows, ld_x apart
    const bf16* y_in;       // [T] rows, ld_y_in apart
    bf16* y_out;
    const bf16* a;          // [n][max_rank][in]
    const bf16* b;          // [n][out][max_rank]
    const float* scale;     // [n] or NULL
    const int* rank;        // [n] or NULL
    const int* adapter_of;  // [T], -1: none
    long long ld_x, ld_y_in, ld_y_out;
    int T, n, in, out, max_rank;
};

// Norms and rotation of queries and keys (see k_rope.cu); NULL where a part is not wanted.
struct RopeProblem {
    unsigned long long turns[32];   // frequency / 2 pi of every pair, in 2^-64 turns per position
    const int* pos;         // [T]
    const bf16* q;          // [T] rows, ld_q apart
    bf16* q_out;
    const bf16* k;          // [T] rows; NULL with caches: the key stands in its slot
    bf16* k_out;            // without caches
    const bf16* v;          // [T] rows that go to the cache as they are
    const bf16* g_q;        // [64] or NULL: no norm
    const bf16* g_k;
    bf16* k_cache;          // [n_seqs][nkv][cap][64] or NULL
    bf16* v_cache;
    const int* seq;         // [T] or NULL (t), negative: none
    const int* slot;        // [T]
    long long ld_q, ld_q_out, ld_k, ld_k_out, ld_v;
    int T, nq, nkv, n_seqs, cap, rot, interleaved;
    float eps, amplitude;
};

// A cache in 8 bits (see k_kvq.cu).  The attention's tiles are cut into kKvqShares equal shares, one to a
// warp; the part of pair i ((sequence, KV head)) that share w has worked on is in slot w + i.  Fixed, so
// that results never depend on the SM count.
enum { KVQ_E4M3 = 0, KVQ_INT8 = 1 };
constexpr int kKvqWarps = 12, kKvqCtas = 152, kKvqShares = kKvqWarps * kKvqCtas;
constexpr int kPartRow = 68;            // 64 dims, maximum, sum
constexpr float kKvqSmallest = 0x1p-110f;   // a block's largest magnitude counts as at least this

struct KvqProblem {
    const uint8_t* k;       // [T][nkv][cap][64] codes
    const uint8_t* v;
    const float* ks;        // [T][nkv][cap / block]
    const float* vs;
    const int* held;        // [T] coded positions
    const bf16* tk;         // [T][nkv][tail_cap][64]
    const bf16* tv;
    const int* kv_len;      // [T] bf16 positions, or NULL: none
    const bf16* q;          // [T][nq * 64]
    bf16* o;
    float* lse;             // [T][nq] or NULL
    float* acc;             // [slot][G][kPartRow]
    int2* parts;            // [T * nkv] first slot, slots (1: written already)
    int T, nq, nkv, G, cap, tail_cap, window, block, block_log2, format;
    float scale_log2;
};

struct FoldProblem {
    const bf16* k;          // [T][nkv][cap][64]
    const bf16* v;
    uint8_t* kq;            // [T][nkv][cap_q][64]
    uint8_t* vq;
    float* ks;              // [T][nkv][cap_q / block]
    float* vs;
    bf16* k_rest;           // [T][nkv][cap_rest][64]
    bf16* v_rest;
    const int* kv_len;      // [T]
    const int* held;
    int* len_out;
    int* held_out;
    int T, nkv, cap, cap_q, cap_rest, block, format;
    int moved;              // the rest goes to another cache
};

int enqueue_qk_rope(Launcher& L, const RopeProblem& p, const KCtx& c, int sms);
int enqueue_kvq_attention(Launcher& L, const KvqProblem& p, const KCtx& c);
int enqueue_kvq_fold(Launcher& L, const FoldProblem& p, const KCtx& c);
int enqueue_prefix(Launcher& L, const PrefixProblem& p, const KCtx& c);
int enqueue_weights(Launcher& L, const WeightsProblem& p, const KCtx& c, int sms);
int enqueue_evict(Launcher& L, const EvictProblem& p, const KCtx& c);
int enqueue_lora(Launcher& L, const LoraProblem& p, const KCtx& c);

}  // namespace sgp
