// rope.cu -- rotary positions on the way into the paged cache (pkv_rope_and_cache): the queries of each token are rotated,
// its key is rotated, converted and written to its slot, its value converted and written, in one pass over the three.
//
// Token at position p, pair i of the rotated part of a head, f = inv_freq[i], a = factor:
//   (x, y) -> (a (x cos(p f) - y sin(p f)), a (y cos(p f) + x sin(p f)))
// in fp32, rounded once to the type of the output or the cache.
//
// Angles: p f loses its fraction of a turn in fp32 long before p reaches a long context's end, so the angle is kept in turns
// as a 64-bit fraction: phase = f / (2 pi) * 2^64, once per CTA and frequency by an integer product with 2^64 / (2 pi), and
// p * phase mod 2^64 is the reduced angle, off by at most |p| 2^-63 turns.  Its upper 32 bits (2^-32 turns) go to
// sincospi.  Every (token, pair) is computed once for all heads of a CTA, through shared memory.
//
// Bound by HBM (large calls) or launch latency.  A thread's unit is 8 elements of one head, two groups of four (of the
// first and the second half of the pairs, or eight neighbours), 16 threads to a head of 128: loads and stores of a warp cover
// whole 32-byte sectors in either pairing, and the rotated part may be any multiple of 8.
#include <algorithm>

#include "rope.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;      // units of a thread in flight
constexpr int kMaxTokens = 4;  // tokens of a CTA

// f turns per radian times 2^64, mod 2^64, for a finite f: the mantissa times floor(2^64 / (2 pi)), shifted by the exponent.
// (Frequencies of 2^24 and more, far beyond the one radian per position that models use, lose bits.)
__device__ __forceinline__ uint64_t turns(float f) {
    constexpr uint64_t kPerRadian = 0x28be60db9391054aull;  // floor(2^64 / (2 pi))
    const uint32_t u = __float_as_uint(f);
    const int e = (u >> 23) & 255;
    const uint64_t m = e ? (u & 0x7fffffu) | 0x800000u : (u & 0x7fffffu);
    const int right = 150 - max(e, 1);  // f = m * 2^-right
    const uint64_t lo = m * kPerRadian, hi = __umul64hi(m, kPerRadian);
    uint64_t t;
    if (right <= 0) t = right > -64 ? lo << -right : 0;
    else if (right < 64) t = (lo >> right) | (hi << (64 - right));
    else t = right < 128 ? hi >> (right - 64) : 0;
    return u >> 31 ? 0 - t : t;
}

template <int T>
__device__ __forceinline__ float4 load4(const uint8_t* base, int64_t elem) {
    if constexpr (T == PKV_F32) return *reinterpret_cast<const float4*>(base + elem * 4);
    const uint2 w = *reinterpret_cast<const uint2*>(base + elem * 2);
    const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
    return make_float4(a.x, a.y, b.x, b.y);
}

template <int T>
__device__ __forceinline__ void store4(uint8_t* base, int64_t elem, float4 x, float scale) {
    if constexpr (T == PKV_F32) {
        *reinterpret_cast<float4*>(base + elem * 4) = x;
    } else if constexpr (T == PKV_BF16) {
        const uint32_t a = float_to_bf16_bits(x.x) | static_cast<uint32_t>(float_to_bf16_bits(x.y)) << 16;
        const uint32_t b = float_to_bf16_bits(x.z) | static_cast<uint32_t>(float_to_bf16_bits(x.w)) << 16;
        *reinterpret_cast<uint2*>(base + elem * 2) = make_uint2(a, b);
    } else {  // the cache write's conversions: an IEEE division, then round to nearest even, saturated
        const float y[4] = {x.x / scale, x.y / scale, x.z / scale, x.w / scale};
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w |= static_cast<uint32_t>(T == PKV_INT8 ? float_to_s8_sym(y[i]) : float_to_e4m3_sat(y[i])) << (8 * i);
        *reinterpret_cast<uint32_t*>(base + elem) = w;
    }
}

}  // namespace

// Grid: x runs of `per_cta` tokens, y parts of the heads (queries, keys and values in a row).
template <int SRC, int DST>
__global__ void __launch_bounds__(kThreads) rope_and_cache_kernel(const RopeArgs a, int per_cta) {
    __shared__ __align__(16) float2 turn[kMaxTokens * 64];  // cos, sin of each token's pairs
    __shared__ int64_t slot_of[kMaxTokens];  // -1: nothing of the token is written
    const int tid = threadIdx.x, t0 = blockIdx.x * per_cta, n = min(per_cta, a.tokens - t0);
    const int half = a.rot >> 1;
    if (tid < n) {
        int64_t s = a.slots ? a.slots[t0 + tid] : 0;
        if (s >= a.pool_slots) {
            if (blockIdx.y == 0) raise_error(a.err, PKV_DEVERR_BAD_SLOT);
            s = -1;
        }
        slot_of[tid] = s;
    }
    for (int i = tid; i < n * half; i += kThreads) {
        const int t = i / half, p = i - t * half;
        const float f = __ldg(a.inv_freq + p);
        const uint64_t phase = turns(f) * static_cast<uint64_t>(static_cast<int64_t>(a.positions[t0 + t]));
        float s, c;
        sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
        if (!(fabsf(f) <= 3.402823466e38f)) c = s = __int_as_float(0x7fc00000);
        turn[t * 64 + p] = make_float2(c * a.factor, s * a.factor);
    }
    __syncthreads();
    const int u_shift = a.d_shift - 3, u = tid & ((1 << u_shift) - 1);  // this thread's unit of its heads
    const int step = kThreads >> u_shift, heads = a.Hq + 2 * a.Hkv;
    const int part = (heads + gridDim.y - 1) / gridDim.y, h0 = blockIdx.y * part, nh = min(part, heads - h0);
    if (nh <= 0) return;
    const bool turned = 8 * u < a.rot;
    const int first = turned && !a.interleaved ? 4 * u : 8 * u, second = turned && !a.interleaved ? half + 4 * u : 8 * u + 4;
    int t = 0, h = tid >> u_shift;
    while (true) {
        while (h >= nh && t < n) {
            h -= nh;
            ++t;
        }
        if (t >= n) break;
        float4 x[kUnits], y[kUnits];
        int tok[kUnits], head[kUnits];
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            while (h >= nh && t < n) {
                h -= nh;
                ++t;
            }
            tok[k] = t;
            head[k] = h0 + h;
            if (t < n && slot_of[t] >= 0) {
                const bool is_q = head[k] < a.Hq, is_k = head[k] < a.Hq + a.Hkv;
                const uint8_t* src = is_q ? a.q : is_k ? a.k : a.v;
                const int64_t at = (t0 + t) * (is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride) +
                                   (static_cast<int64_t>(head[k] - (is_q ? 0 : is_k ? a.Hq : a.Hq + a.Hkv)) << a.d_shift);
                x[k] = load4<SRC>(src, at + first);
                y[k] = load4<SRC>(src, at + second);
            } else {
                tok[k] = -1;
            }
            h += step;
        }
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            if (tok[k] < 0) continue;
            const bool is_q = head[k] < a.Hq, is_k = head[k] < a.Hq + a.Hkv;
            if (turned && is_k) {
                const float4* cs = reinterpret_cast<const float4*>(&turn[tok[k] * 64 + 4 * u]);
                const float4 c0 = cs[0], c1 = cs[1];  // cos, sin of pairs 4 u .. 4 u + 3
                const float4 p = x[k], q = y[k];
                if (a.interleaved) {
                    x[k] = make_float4(p.x * c0.x - p.y * c0.y, p.y * c0.x + p.x * c0.y, p.z * c0.z - p.w * c0.w, p.w * c0.z + p.z * c0.w);
                    y[k] = make_float4(q.x * c1.x - q.y * c1.y, q.y * c1.x + q.x * c1.y, q.z * c1.z - q.w * c1.w, q.w * c1.z + q.z * c1.w);
                } else {
                    x[k] = make_float4(p.x * c0.x - q.x * c0.y, p.y * c0.z - q.y * c0.w, p.z * c1.x - q.z * c1.y, p.w * c1.z - q.w * c1.w);
                    y[k] = make_float4(q.x * c0.x + p.x * c0.y, q.y * c0.z + p.y * c0.w, q.z * c1.x + p.z * c1.y, q.w * c1.z + p.w * c1.w);
                }
            }
            if (is_q) {
                const int64_t at = (t0 + tok[k]) * a.q_out_stride + (static_cast<int64_t>(head[k]) << a.d_shift);
                store4<SRC>(a.q_out, at + first, x[k], 1.f);
                store4<SRC>(a.q_out, at + second, y[k], 1.f);
            } else {
                const int kv = head[k] - (is_k ? a.Hq : a.Hq + a.Hkv);
                uint8_t* dst = is_k ? a.k_cache : a.v_cache;
                const float* hs = is_k ? a.k_head : a.v_head;
                const float scale = hs ? __ldg(hs + kv) : is_k ? a.k_scale : a.v_scale;
                const int64_t at = (slot_of[tok[k]] * a.Hkv + kv) << a.d_shift;
                store4<DST>(dst, at + first, x[k], scale);
                store4<DST>(dst, at + second, y[k], scale);
            }
        }
    }
}

cudaError_t launch_rope_and_cache(const RopeArgs& a, int src_dtype, int dst_dtype, int sms, cudaStream_t stream) {
    const int heads = a.Hq + 2 * a.Hkv, at_once = kThreads >> (a.d_shift - 3);
    // one token per CTA until every SM has its fill of CTAs; below that, parts of a token's heads
    const int fill = sms * (2048 / kThreads);
    const int per_cta = std::min(kMaxTokens, std::max(1, a.tokens / fill));
    const int runs = (a.tokens + per_cta - 1) / per_cta;
    const int parts = std::max(1, std::min((heads + at_once - 1) / at_once, fill / runs));
    const dim3 grid(runs, parts);
#define PKV_ROPE(S_, D_)                                                              \
    if (src_dtype == S_ && dst_dtype == D_) {                                         \
        rope_and_cache_kernel<S_, D_><<<grid, kThreads, 0, stream>>>(a, per_cta);     \
        return cudaGetLastError();                                                    \
    }
    PKV_ROPE(PKV_F32, PKV_F32)
    PKV_ROPE(PKV_F32, PKV_BF16)
    PKV_ROPE(PKV_F32, PKV_FP8_E4M3)
    PKV_ROPE(PKV_F32, PKV_INT8)
    PKV_ROPE(PKV_BF16, PKV_F32)
    PKV_ROPE(PKV_BF16, PKV_BF16)
    PKV_ROPE(PKV_BF16, PKV_FP8_E4M3)
    PKV_ROPE(PKV_BF16, PKV_INT8)
#undef PKV_ROPE
    return cudaErrorInvalidValue;
}

}  // namespace pkv
