// full_tile.cuh -- arguments and launchers of the unmasked attention tile (full_tile.cu): cross attention, and the
// shared prefixes of a decode batch.
#pragma once

#include "prefill.cuh"

namespace pkv {

// Partial records: base rows (one per query token and query head: an item's first piece), then 256 rows for every CTA
// (the piece with which a CTA's share starts inside an item).
struct FullArgs {
    float* rec_o;        // [rows][128] unnormalised O
    float2* rec_ml;      // [rows] (running maximum in log2 units, sum)
    int64_t extra_row;   // first row of the CTAs' own pieces: total_q_tokens * Hq
    int4* cuts;          // [CTAs] the item that CTA c's share starts inside of (CutItem)
    int4* seq_plan;      // prefix form: [num_seqs] (SeqPlan), else nullptr
    int* share;          // key tiles per CTA
    bool prefix;         // chunks are groups: chunk g's table row is that of its first token (sequence)
};

// cuts[c] = {first query token's row of q, valid rows | h << 16, U0, U1}: CTA c's share starts strictly inside the item
// whose key tiles are stream positions [U0, U1); U1 = 0: it does not.
// seq_plan[s] = {U0 of the tile's head 0, key tiles per item, row of the sequence's first query head in its tile, 0}.

size_t paged_full_smem_bytes(int narrow);
cudaError_t launch_paged_full(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                              const PrefillArgs& a, const FullArgs& f, int narrow, int grid, cudaStream_t stream);
cudaError_t launch_full_combine(const PrefillArgs& a, const FullArgs& f, int grid, cudaStream_t stream);

}  // namespace pkv
