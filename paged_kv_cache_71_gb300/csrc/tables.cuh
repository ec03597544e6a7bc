// tables.cuh -- arguments and launchers of the step-planning kernels (tables.cu).
#pragma once

#include "pkv_device.cuh"

namespace pkv {

struct ExtendArgs {
    int32_t* tables;             // [N][MB], entries of the new blocks are written
    const int32_t* past_lens;    // [N]
    const int32_t* new_lens;     // [N]
    const int32_t* free_blocks;  // stack of free ids, the top at *free_count - 1
    const int32_t* free_count;
    int32_t* seq_lens;           // [N], may be past_lens
    int32_t* new_free_count;     // may be free_count
    int32_t* cu_q;               // [N + 1], nullable
    int32_t* q_starts;           // [N], nullable
    int64_t* slots;              // [max_tokens]
    int32_t* err;                // nullable
    int N, MB, shift, NB, max_tokens;  // shift: log2 of the block size
    int runs = 1;                      // consecutive slots of a thread (set by the launcher)
};

struct ReleaseArgs {
    const int32_t* tables;
    const int32_t* past_lens;
    const uint8_t* finished;     // [N], non-zero: the sequence hands its blocks back
    const int32_t* keep_blocks;  // [N], nullable: leading blocks that are not the sequence's own
    int32_t* free_blocks;        // [NB]
    const int32_t* free_count;
    int32_t* seq_lens;           // [N], may be past_lens
    int32_t* new_free_count;     // may be free_count
    int32_t* err;
    int N, MB, shift, NB;
};

constexpr int kMaxTableSeqs = 8192;

cudaError_t launch_extend_sequences(const ExtendArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_release_sequences(const ReleaseArgs& a, int sms, cudaStream_t stream);

}  // namespace pkv
