// full_tile.cuh -- arguments and launchers of the attention stream (full_tile.cu): cross attention, the shared prefixes of a
// decode batch, and runs of drafted tokens over their sequence's cache.
#pragma once

#include "prefill.cuh"

namespace pkv {

// Chunks, each a run of query tokens and the keys they all attend to:
//   cross attention: sequence s, query tokens [cu_q[s], cu_q[s + 1]), keys [0, kv_lens[s]) of table row s;
//   shared prefixes: group g, tokens = sequences [cu_q[g], cu_q[g + 1]), keys [0, kv_lens[g]) of its first sequence's row;
//   draft trees: as cross attention, but the run's tokens are the last of the keys, and each sees those that its mask names.
// An item is one or two query tiles (128 rows each: token x query head of the group) of one KV head of a chunk.
struct FullArgs {
    // partial records (O unnormalised, m in log2 units, l): one row per (token, query head) for an item's first piece, then
    // 256 rows for every CTA, for the piece with which its share starts inside an item
    float* rec_o;        // [rows][128]
    float2* rec_ml;      // [rows]
    int64_t extra_row;   // first row of the CTAs': total_q_tokens * Hq
    const float* q_scale;  // one-byte caches: [rows] of (token, query head), what the operands' scores are multiplied by
    int* share;          // stream units per CTA; 0: `points`
    int* points;         // [CTAs + 1] where the CTAs' parts of the stream start, when they differ
    int4* cuts;          // [CTAs] {first token, tokens | head << 16, U0, U1} of the item that the CTA's share starts inside
                         // of: shares that start in (U0, U1) of the stream start with a later piece of it; U1 = 0: none
    int4* seq_plan;      // shared prefixes: [sequences] {first key tile's unit of KV head 0's item, units per item, row in the
                         // item, units of its key tiles}
    const int* prefix_blocks;  // [sequences] as the decode of the own blocks found them: > 0 if the row is to be joined
    const int32_t* lens;       // [sequences] context lengths
    int num_seqs;
    int64_t own_row;           // first row of the own blocks' records
    bool prefix;         // shared prefixes: every item leaves records
    bool tree = false;   // draft trees
    int mask_words = 0;  // 64-bit words of a token's mask
    const uint64_t* tree_mask = nullptr;  // [tokens][mask_words]; none: each run is a chain
    const void* v_cache = nullptr;        // draft trees
};

size_t paged_full_smem_bytes(int narrow, bool tree = false);
cudaError_t launch_paged_full(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                              const PrefillArgs& a, const FullArgs& f, int narrow, int grid, bool prepared,
                              cudaStream_t stream);
// Before the stream: the queries' operands (one-byte caches), counters cleared.
cudaError_t launch_full_prepare(const void* q, void* ops, float* scale, int64_t rows, int* counters, int64_t n_counters,
                                int narrow, int sms, cudaStream_t stream);
// Joins the pieces of the cut items (cross attention).
cudaError_t launch_join_cuts(const PrefillArgs& a, const FullArgs& f, int grid, cudaStream_t stream);
// Joins every row of a sequence with a prefix: its pieces, and the record of the sequence's own blocks.
cudaError_t launch_join_rows(const PrefillArgs& a, const FullArgs& f, cudaStream_t stream);

}  // namespace pkv
