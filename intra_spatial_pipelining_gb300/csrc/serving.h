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

int enqueue_prefix(Launcher& L, const PrefixProblem& p, const KCtx& c);
int enqueue_weights(Launcher& L, const WeightsProblem& p, const KCtx& c, int sms);
int enqueue_evict(Launcher& L, const EvictProblem& p, const KCtx& c);
int enqueue_lora(Launcher& L, const LoraProblem& p, const KCtx& c);

}  // namespace sgp
