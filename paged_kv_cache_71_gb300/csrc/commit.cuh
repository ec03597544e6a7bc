// commit.cuh -- arguments and launcher of the commit of accepted draft tokens (commit.cu).
#pragma once

#include "pkv_device.cuh"

namespace pkv {

constexpr int kMaxLayers = PKV_MAX_LAYERS;
constexpr int kMaxCommitRun = PKV_MAX_COMMIT_RUN;

struct CommitArgs {
    uint4* k[kMaxLayers];
    uint4* v[kMaxLayers];
    const int32_t* tables;
    const int32_t* cu_q;
    const int32_t* past_lens;
    const int32_t* parents;
    const int32_t* draft;
    const int32_t* target;
    int32_t* accepted;
    int32_t* num_accepted;
    int32_t* seq_lens;
    int32_t* next_tokens;
    int32_t* keep_blocks;  // nullable
    int32_t* err;          // nullable
    int layers, MB, shift, NB, tokens, vecs;  // shift: log2 of the block size; vecs: 16-byte pieces of a token's K row
    int per_cta;                              // layers that one CTA moves (set by the launcher)
};

cudaError_t launch_commit_tree(CommitArgs& a, int num_seqs, int sms, cudaStream_t stream);

}  // namespace pkv
