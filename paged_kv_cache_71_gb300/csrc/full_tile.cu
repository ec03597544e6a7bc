// full_tile.cu -- attention of many query rows over a paged K/V range without a mask: cross attention to an encoder's
// states (pkv_paged_cross_attention) and the shared prefixes of a decode batch (pkv_paged_attention_decode_prefix).
//
// A chunk is a run of query tokens that attend to the same keys: a sequence's tokens and its encoder states, or a group
// of sequences (one token each) and their common prefix.  For KV head h its rows are (token, query head of h's group),
// stacked; an item is a pair of 128-row query tiles of one KV head against all of the chunk's keys, and runs on the
// tcgen05 tile of prefill_tile.cuh: S = Q K^T, an online softmax, O += P V, with K and V read once per 256 rows.
//
// Work split: the items' key tiles (64 keys) are laid end to end and cut into equal shares, one per CTA (SM).  An item
// that is cut leaves a partial (O, m, l) record for each of its pieces; they join as
//   M = max m_i,  l = sum 2^(m_i - M) l_i,  O = sum 2^(m_i - M) O_i / l
// in full_combine_kernel (cross attention) or at the end of the suffix decode (decode_mma.cuh).
#include "full_tile.cuh"
#include "prefill_tile.cuh"

namespace pkv {

namespace {

// Fewest key tiles in a share: a piece costs the tile's set-up (TMEM, barriers, Q) and a record whatever its length.
constexpr int kMinShare = 4;

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

}  // namespace

template <int NARROW>
__global__ void __launch_bounds__(kThreads, 1)
    paged_full_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const PrefillArgs a, const FullArgs f) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int* part = reinterpret_cast<int*>(smem + Plan<NARROW>::kOffMeta + kMetaPart);
    int* pre = reinterpret_cast<int*>(smem + Plan<NARROW>::kOffMeta + kMetaCount);  // [nseq + 1] key tiles before chunk s
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x, ncta = gridDim.x;
    const int rows_q = kRows / a.G, cta_q = 2 * rows_q;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- chunk s: query tokens [q0, q1), keys; nothing to do for a malformed chunk
    auto chunk = [&](int s, int& q0, int& q1, int& kv, bool report) {
        q0 = a.cu_q[s];
        q1 = a.cu_q[s + 1];
        kv = a.kv_lens[s];
        const bool bad_q = q0 < 0 || q1 < q0 || q1 > a.NQ;
        const bool bad_k = kv < 0 || kv > a.MB * a.S || (f.prefix && kv % a.S != 0);
        if ((bad_q || bad_k) && report) raise_error(a.err, PKV_DEVERR_BAD_LENGTH);
        if (bad_q) q1 = q0 = 0;
        if (bad_k) kv = -1;
    };
    const int per = (a.nseq + kThreads - 1) / kThreads;
    const int c_lo = min(tid * per, a.nseq), c_hi = min(c_lo + per, a.nseq);
    int sum = 0;
    for (int c = c_lo; c < c_hi; ++c) {
        int q0, q1, kv;
        chunk(c, q0, q1, kv, cta == 0);
        const int w = kv > 0 ? ceil_div(q1 - q0, cta_q) * a.Hkv * ceil_div(kv, kKeys) : 0;
        pre[c + 1] = w;
        sum += w;
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < warp; ++w) run += part[w];
    for (int c = c_lo; c < c_hi; ++c) {
        run += pre[c + 1];
        pre[c + 1] = run;
    }
    if (tid == 0) pre[0] = 0;
    __syncthreads();
    const int T = pre[a.nseq];
    const int share = max(kMinShare, ceil_div(T, ncta));

    // ---- what the joining of the pieces needs to know, and the rows without keys
    if (cta == 0 && tid == 0) *f.share = share;
    if (f.prefix) {
        for (int g = cta; g < a.nseq; g += ncta) {
            int q0, q1, kv;
            chunk(g, q0, q1, kv, false);
            const int kt = kv > 0 ? ceil_div(kv, kKeys) : 0;
            for (int i = tid; i < q1 - q0; i += kThreads)
                f.seq_plan[q0 + i] = make_int4(pre[g] + (i / cta_q) * a.Hkv * kt, kt, (i % cta_q) * a.G, 0);
        }
    } else {
        for (int s = cta; s < a.nseq; s += ncta) {
            int q0, q1, kv;
            chunk(s, q0, q1, kv, false);
            if (kv != 0) continue;
            uint4* o = reinterpret_cast<uint4*>(a.out) + static_cast<size_t>(q0) * a.Hq * 16;
            for (size_t i = tid; i < static_cast<size_t>(q1 - q0) * a.Hq * 16; i += kThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    }

    // ---- this CTA's share of the stream, item by item
    int x = min(static_cast<int64_t>(cta) * share, static_cast<int64_t>(T));
    const int x_end = min(static_cast<int64_t>(x) + share, static_cast<int64_t>(T));
    if (tid == 0) f.cuts[cta] = make_int4(0, 0, 0, 0);
    while (x < x_end) {
        int lo = 0, hi = a.nseq - 1;  // the chunk whose key tiles hold x
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= x) lo = mid; else hi = mid - 1;
        }
        int q0, q1, kv;
        chunk(lo, q0, q1, kv, false);
        const int kt = ceil_div(kv, kKeys), item = (x - pre[lo]) / kt;
        const int tile = item / a.Hkv, h = item % a.Hkv;
        const int U0 = pre[lo] + item * kt, U1 = U0 + kt;
        FullJob job;
        job.q_base = q0;
        job.NQ = q1 - q0;
        job.i0 = tile * cta_q;
        job.kv_len = kv;
        job.table = a.block_table + static_cast<size_t>(f.prefix ? q0 : lo) * a.MB;
        job.j0 = x - U0;
        job.n_tiles = min(U1, x_end) - x;
        if (f.prefix || job.n_tiles < kt) {
            const bool head = job.j0 == 0;  // an item's first piece has the rows' own records
            job.rec_by_token = head;
            const size_t row = head ? 0 : static_cast<size_t>(f.extra_row) + static_cast<size_t>(cta) * (2 * kRows);
            job.rec_o = f.rec_o + row * 128;
            job.rec_ml = f.rec_ml + row;
            if (!head && tid == 0)
                f.cuts[cta] = make_int4(q0 + job.i0, min(cta_q, job.NQ - job.i0) | (h << 16), U0, U1);
        }
        prefill_tile<NARROW, NARROW == 2, true, true>(qmap, kmap, vmap, a, 0, h, 0, smem_raw, job);
        x += job.n_tiles;
    }
}

// Joins the pieces of every cut item: block (c, part) takes rows [32 part, 32 part + 32) of the item whose second piece
// starts CTA c's share; one warp per row, four head dims per lane.
__global__ void __launch_bounds__(256) full_combine_kernel(const PrefillArgs a, const FullArgs f) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 cut = f.cuts[c];
    const int share = *f.share, U0 = cut.z, U1 = cut.w;
    if (U1 == 0 || U0 / share != c - 1) return;
    const int valid = (cut.y & 0xffff) * a.G, h = cut.y >> 16;
    const int c_last = (U1 - 1) / share;
    const float out_mul = a.v_head ? __ldg(a.v_head + h) : a.out_mul;
    for (int r = blockIdx.y * 32 + warp; r < min(valid, blockIdx.y * 32 + 32); r += 8) {
        const size_t tok = static_cast<size_t>(cut.x) + r / a.G;
        const size_t row = tok * a.Hq + static_cast<size_t>(h) * a.G + r % a.G;
        float2 ml = f.rec_ml[row];
        float4 o = reinterpret_cast<const float4*>(f.rec_o + row * 128)[lane];
        for (int k = c; k <= c_last; ++k) {
            const size_t rk = static_cast<size_t>(f.extra_row) + static_cast<size_t>(k) * 256 + r;
            const float2 mk = f.rec_ml[rk];
            const float4 ok = reinterpret_cast<const float4*>(f.rec_o + rk * 128)[lane];
            const float m = fmaxf(ml.x, mk.x), w0 = ex2_approx(ml.x - m), w1 = ex2_approx(mk.x - m);
            ml = make_float2(m, ml.y * w0 + mk.y * w1);
            o.x = o.x * w0 + ok.x * w1;
            o.y = o.y * w0 + ok.y * w1;
            o.z = o.z * w0 + ok.z * w1;
            o.w = o.w * w0 + ok.w * w1;
        }
        const float inv = ml.y > 0.f ? out_mul / ml.y : 0.f;
        reinterpret_cast<uint2*>(a.out)[row * 32 + lane] = make_uint2(bf16x2_rn(o.x * inv, o.y * inv),
                                                                      bf16x2_rn(o.z * inv, o.w * inv));
    }
}

template <int NARROW>
static cudaError_t launch_full(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                               const PrefillArgs& a, const FullArgs& f, int grid, cudaStream_t stream) {
    const size_t smem = prefill_ws_smem_bytes(NARROW);
    auto kern = paged_full_kernel<NARROW>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    kern<<<grid, kThreads, smem, stream>>>(qmap, kmap, vmap, a, f);
    return cudaGetLastError();
}

cudaError_t launch_paged_full(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                              const PrefillArgs& a, const FullArgs& f, int narrow, int grid, cudaStream_t stream) {
    switch (narrow) {
        case 0: return launch_full<0>(qmap, kmap, vmap, a, f, grid, stream);
        case 1: return launch_full<1>(qmap, kmap, vmap, a, f, grid, stream);
        case 2: return launch_full<2>(qmap, kmap, vmap, a, f, grid, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_full_combine(const PrefillArgs& a, const FullArgs& f, int grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 8);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, full_combine_kernel, a, f);
}

}  // namespace pkv
