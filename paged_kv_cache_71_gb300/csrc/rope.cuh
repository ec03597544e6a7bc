// rope.cuh -- arguments and launcher of the rotary cache write (rope.cu).
#pragma once

#include "pkv_device.cuh"

namespace pkv {

struct RopeArgs {
    const uint8_t *q, *k, *v;  // q and q_out, and k and v, may be NULL (head counts 0 then)
    uint8_t *q_out, *k_cache, *v_cache;
    int64_t q_stride, k_stride, v_stride, q_out_stride;  // elements from token to token
    const int32_t* positions;
    const int64_t* slots;  // nullable: every token's queries are rotated
    const float* inv_freq;
    float factor;          // what cos and sin are multiplied by
    int tokens, Hq, Hkv, d_shift, rot;  // Hkv: 0 without keys; d_shift: log2 of the head dimension
    bool interleaved;
    int64_t pool_slots;
    float k_scale, v_scale;
    const float *k_head, *v_head;
    int32_t* err;
};

cudaError_t launch_rope_and_cache(const RopeArgs& a, int src_dtype, int dst_dtype, int sms, cudaStream_t stream);

}  // namespace pkv
