// rope.cu -- rotary positions on the way into the paged cache (pkv_rope_and_cache): the queries of each token are rotated,
// its key is rotated, converted and written to its slot, its value converted and written, in one pass over the three.
//
// Token at position p, pair i of the rotated part of a head, f = inv_freq[i], a = factor:
//   (x, y) -> (a (x cos(p f) - y sin(p f)), a (y cos(p f) + x sin(p f)))
// in fp32, rounded once to the type of the output or the cache.
//
// Angles: p f loses its fraction of a turn in fp32 long before p reaches a long context's end, so the angle is kept in turns
// as a 64-bit fraction: phase = f / (2 pi) * 2^64, by an integer product with 2^96 / (2 pi), and p * phase mod 2^64 is the
// reduced angle, off by less than 1.51 |p| 2^-64 turns for f below 2^24.  Its upper 32 bits (2^-32 turns) go to sincospi.
// Every (token, pair) is computed once for all heads of a CTA, through shared memory.
//
// Bound by HBM (large calls) or launch latency.  A thread's unit is two 16-byte groups of one head's elements, of the first and
// the second half of the pairs or one behind the other (two 8-byte groups of bf16 where the rotated part is no multiple of
// 16): a warp's loads and stores cover whole 128-byte lines.  A thread has all of its units (up to four) on their way before
// the angles are computed, whose loads, sines and barrier they cover.
#include <algorithm>

#include "rope.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;      // most units of a thread
constexpr int kMaxTokens = 4;  // most tokens of a CTA
// CTAs that an SM's registers have to hold.  No bound, 3, 4, 5: 8192 bf16 prompt tokens (32 / 8 heads) 41.7 / 34.4 / 32.3 / 32.7
// us, 1013 tokens of 64 / 8 heads into an FP8 cache 11.2 / 9.3 / 7.8 / 9.6 (floors 29.7 and 5.8; 2 us of each is the launch; one
// batch over and over: the drafts' 39 MB stay in L2, and take 10.3 us instead of 7.7 where they do not, the prompt 32.6 for 32.3).
constexpr int kCtas = 4;

// f turns per radian times 2^64, mod 2^64, for a finite f below 2^24: the mantissa times the first 96 bits of 1 / (2 pi), shifted
// by the exponent (a reduction after Payne and Hanek).  Off by less than 1.51: one for the bits shifted out, half of 1.004
// for those of the product that are not computed.  With the constant's first 64 bits alone the error was half of f more, so
// that at position 2^31 - 1 f = 1000 was off by 4e-7 radians, 2^23 by 3e-3; 8192 tokens of 8 / 1 heads took 9.8 us, with 96
// bits 10.0.  (Larger f, far beyond the one radian per position that models use, lose bits.)
__device__ __forceinline__ uint64_t turns(float f) {
    constexpr uint64_t kPerRadian = 0x28be60db9391054aull;  // floor(2^96 / (2 pi)), its upper 64 bits
    constexpr uint32_t kPerRadianLow = 0x7f09d5f4u;
    const uint32_t u = __float_as_uint(f);
    const int e = (u >> 23) & 255;
    const uint32_t m = e ? (u & 0x7fffffu) | 0x800000u : (u & 0x7fffffu);
    const int right = 150 - max(e, 1);  // f = m * 2^-right
    const uint64_t top = m * kPerRadian, lo = top + __umulhi(m, kPerRadianLow);
    const uint64_t hi = __umul64hi(m, kPerRadian) + (lo < top);
    uint64_t t;
    if (right <= 0) t = right > -64 ? lo << -right : 0;
    else if (right < 64) t = (lo >> right) | (hi << (64 - right));
    else t = right < 128 ? hi >> (right - 64) : 0;
    return u >> 31 ? 0 - t : t;
}

// V elements of type T as they lie in memory: 16 bytes, or 8
template <int T, int V>
struct Group {
    static constexpr int kWords = V * (T == PKV_F32 ? 4 : 2) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const uint8_t* base, int64_t elem) {
        const uint8_t* p = base + elem * (T == PKV_F32 ? 4 : 2);
        if constexpr (kWords == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(p);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            w[0] = x.x, w[1] = x.y;
        }
    }
    __device__ __forceinline__ void values(float (&f)[V]) const {
        if constexpr (T == PKV_F32) {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 x = bf16x2_to_float2(w[i]);
                f[2 * i] = x.x;
                f[2 * i + 1] = x.y;
            }
        }
    }
};

// f / scale, as the cache write divides (IEEE).  Of a power of two the product with its inverse, which is the same number:
// 8192 tokens of 16 / 8 heads of 64 into an FP8 cache, in L2, 16.3 us by division, 13.0 by product (12.5 with two codes a
// conversion; 15.4 where q, k and v come from HBM).
template <int V>
__device__ __forceinline__ void divide(float (&f)[V], float scale) {
    const uint32_t u = __float_as_uint(scale), e = u >> 23;
    if ((u & 0x7fffffu) == 0 && e >= 1 && e <= 253) {
        const float inv = __uint_as_float((254 - e) << 23);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] *= inv;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] /= scale;
    }
}

template <int T, int V>
__device__ __forceinline__ void store_group(uint8_t* base, int64_t elem, const float (&f)[V]) {
    constexpr int kBytes = T == PKV_F32 ? 4 : T == PKV_BF16 ? 2 : 1, kWords = V * kBytes / 4;
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        if constexpr (T == PKV_F32) {
            w[i] = __float_as_uint(f[i]);
        } else if constexpr (T == PKV_BF16) {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
        } else if constexpr (T == PKV_FP8_E4M3) {  // the cache write's conversions: round to nearest even, saturated
            uint16_t lo, hi;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f[4 * i + 1]), "f"(f[4 * i]));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f[4 * i + 3]), "f"(f[4 * i + 2]));
            w[i] = lo | static_cast<uint32_t>(hi) << 16;
        } else {
            w[i] = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[i] |= static_cast<uint32_t>(float_to_s8_sym(f[4 * i + k])) << (8 * k);
        }
    }
    uint8_t* p = base + elem * kBytes;
    if constexpr (kWords == 8) {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else if constexpr (kWords == 4) {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (kWords == 2) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
        *reinterpret_cast<uint32_t*>(p) = w[0];
    }
}

}  // namespace

// Grid: x runs of `per_cta` tokens, y parts of the heads (queries, keys and values in a row).  V: elements of a group.
template <int SRC, int DST, int V>
__global__ void __launch_bounds__(kThreads, kCtas) rope_and_cache_kernel(const RopeArgs a, int per_cta) {
    // cos, sin of each token's pairs, two pairs to 16 bytes; those that the threads of a head read at a time side by side
    __shared__ float4 turn[kMaxTokens][32];
    __shared__ int64_t slot_of[kMaxTokens];  // -1: nothing of the token is written
    constexpr int kQuads = V / 2;            // 16-byte pieces of `turn` that a unit needs
    constexpr int kPlaces = 32 / kQuads;     // units of a head of 128
    const int tid = threadIdx.x, t0 = blockIdx.x * per_cta, n = min(per_cta, a.tokens - t0);
    const int half = a.rot >> 1, u_shift = a.d_shift - (V == 8 ? 4 : 3);
    const int u = tid & ((1 << u_shift) - 1);  // this thread's unit of its heads
    const int heads = a.Hq + 2 * a.Hkv, part = (heads + gridDim.y - 1) / gridDim.y;
    const int h0 = blockIdx.y * part, nh = min(part, heads - h0), rows = n * nh;
    if (nh <= 0) return;
    const bool turned = 2 * V * u < a.rot;
    const int first = turned && !a.interleaved ? V * u : 2 * V * u, second = turned && !a.interleaved ? half + V * u : first + V;
    const int row0 = tid >> u_shift, step = kThreads >> u_shift;
    auto token_of = [&](int row) { return (row >= nh) + (row >= 2 * nh) + (row >= 3 * nh); };
    Group<SRC, V> x[kUnits], y[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const int row = row0 + k * step;
        if (row >= rows) break;
        const int t = token_of(row), h = h0 + row - t * nh;
        const bool is_q = h < a.Hq, is_k = h < a.Hq + a.Hkv;
        const uint8_t* src = is_q ? a.q : is_k ? a.k : a.v;
        const int64_t at = (t0 + t) * (is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride) +
                           (static_cast<int64_t>(h - (is_q ? 0 : is_k ? a.Hq : a.Hq + a.Hkv)) << a.d_shift);
        x[k].load(src, at + first);
        y[k].load(src, at + second);
    }
    if (tid >= kThreads - n) {  // (the last threads: the first ones have the angles)
        const int t = kThreads - 1 - tid;
        int64_t s = a.slots ? a.slots[t0 + t] : 0;
        if (s >= a.pool_slots) {
            if (blockIdx.y == 0) raise_error(a.err, PKV_DEVERR_BAD_SLOT);
            s = -1;
        }
        slot_of[t] = s;
    }
    for (int i = tid; i < n * half; i += kThreads) {
        const int t = i / half, p = i - t * half;
        const float f = __ldg(a.inv_freq + p);
        const uint64_t phase = turns(f) * static_cast<uint64_t>(static_cast<int64_t>(a.positions[t0 + t]));
        float s, c;
        sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
        if (!(fabsf(f) <= 3.402823466e38f)) c = s = __int_as_float(0x7fc00000);
        const int quad = p >> 1;
        reinterpret_cast<float2*>(&turn[t][(quad % kQuads) * kPlaces + quad / kQuads])[p & 1] = make_float2(c * a.factor, s * a.factor);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
        const int row = row0 + k * step;
        if (row >= rows) break;
        const int t = token_of(row), h = h0 + row - t * nh;
        const int64_t slot = slot_of[t];
        if (slot < 0) continue;
        const bool is_q = h < a.Hq, is_k = h < a.Hq + a.Hkv;
        float p[V], q[V];
        x[k].values(p);
        y[k].values(q);
        if (turned && is_k) {
#pragma unroll
            for (int i = 0; i < kQuads; ++i) {
                const float4 cs = turn[t][i * kPlaces + u];  // pairs V u + 2 i and the next
                const float c[2] = {cs.x, cs.z}, s[2] = {cs.y, cs.w};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float *l, *r;  // the pair
                    if (a.interleaved) {
                        l = i < kQuads / 2 ? &p[4 * i + 2 * e] : &q[4 * (i - kQuads / 2) + 2 * e];
                        r = l + 1;
                    } else {
                        l = &p[2 * i + e];
                        r = &q[2 * i + e];
                    }
                    const float lv = *l, rv = *r;
                    *l = lv * c[e] - rv * s[e];
                    *r = rv * c[e] + lv * s[e];
                }
            }
        }
        if (is_q) {
            const int64_t at = (t0 + t) * a.q_out_stride + (static_cast<int64_t>(h) << a.d_shift);
            store_group<SRC, V>(a.q_out, at + first, p);
            store_group<SRC, V>(a.q_out, at + second, q);
        } else {
            const int kv = h - (is_k ? a.Hq : a.Hq + a.Hkv);
            uint8_t* dst = is_k ? a.k_cache : a.v_cache;
            if constexpr (DST == PKV_FP8_E4M3 || DST == PKV_INT8) {
                const float* hs = is_k ? a.k_head : a.v_head;
                const float scale = hs ? __ldg(hs + kv) : is_k ? a.k_scale : a.v_scale;
                divide(p, scale);
                divide(q, scale);
            }
            const int64_t at = (slot * a.Hkv + kv) << a.d_shift;
            store_group<DST, V>(dst, at + first, p);
            store_group<DST, V>(dst, at + second, q);
        }
    }
}

cudaError_t launch_rope_and_cache(const RopeArgs& a, int src_dtype, int dst_dtype, int sms, cudaStream_t stream) {
    // bf16 groups of 16 bytes need whole units in the rotated part
    const int V = src_dtype == PKV_BF16 && a.rot % 16 == 0 ? 8 : 4;
    const int units = (a.Hq + 2 * a.Hkv) << (a.d_shift - (V == 8 ? 4 : 3));  // of a token
    // as many tokens as four units a thread hold, or parts of a token; one unit a thread while that leaves SMs without a CTA
    int per_cta = std::max(1, std::min({kMaxTokens, kThreads * kUnits / units, (a.tokens + sms - 1) / sms}));
    const int runs = (a.tokens + per_cta - 1) / per_cta;
    int parts = (units + kThreads * kUnits - 1) / (kThreads * kUnits);
    if (per_cta == 1 && static_cast<int64_t>(runs) * parts < 2 * sms) parts = (units + kThreads - 1) / kThreads;
    const int heads = a.Hq + 2 * a.Hkv, at_once = kThreads / (units / heads);  // (a part is whole heads)
    parts = std::max(parts, (heads + at_once * kUnits - 1) / (at_once * kUnits));
    const dim3 grid(runs, parts);
#define PKV_ROPE_V(S_, D_, V_)                                                            \
    if (src_dtype == S_ && dst_dtype == D_ && V == V_) {                                  \
        rope_and_cache_kernel<S_, D_, V_><<<grid, kThreads, 0, stream>>>(a, per_cta);     \
        return cudaGetLastError();                                                        \
    }
#define PKV_ROPE(D_) PKV_ROPE_V(PKV_F32, D_, 4) PKV_ROPE_V(PKV_BF16, D_, 8) PKV_ROPE_V(PKV_BF16, D_, 4)
    PKV_ROPE(PKV_F32)
    PKV_ROPE(PKV_BF16)
    PKV_ROPE(PKV_FP8_E4M3)
    PKV_ROPE(PKV_INT8)
#undef PKV_ROPE
#undef PKV_ROPE_V
    return cudaErrorInvalidValue;
}

}  // namespace pkv
