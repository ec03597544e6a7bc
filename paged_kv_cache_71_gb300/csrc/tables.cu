// tables.cu -- block tables, lengths and slot maps of a serving step, planned on the GPU from the request lengths.
//
// The rules are those of the host block manager: a sequence of L tokens holds nb(L) = ceil(L / S) blocks, position p
// lives in slot table[p / S] * S + p % S ("3.3 批处理与内存管理", sections "PagedAttention：块表" and "代码"), free ids
// form a stack and a sequence takes a new id from its top whenever its last block is full.  Sequence s, with L_s
// tokens and n_s more to come, takes e_s = nb(L_s + n_s) - nb(L_s) blocks; with E the exclusive sum of e over the
// batch and F free ids, its i-th new block is free[F - 1 - (E_s + i)] -- what taking the blocks one by one in order
// would give, known for every block at once.  Releasing is the mirror image: block i of the finished sequence s goes to
// free[F + E_s + i].
//
// The work is a scan over the batch and then independent writes.  Every CTA scans the whole batch for itself (at most 8
// sequences a thread), keeps the sums in shared memory and writes its part, so one launch does the call without the CTAs
// having to wait for one another.  Lengths and the free count may be updated in place, which nobody may do while a CTA
// still reads them: with one CTA it is the last thing it does, with several a second small kernel does it after them.
#include <algorithm>

#include "tables.cuh"

namespace pkv {

namespace {

// Sums that stay at kMany once they reach it: they are past every limit then, and the order of the additions does not matter.
constexpr uint32_t kMany = 0x7fffffffu;
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return min(a + b, kMany); }

// Block-wide exclusive sums of two values per thread; the totals in ta, tb.  (Short rolled code: a step runs once, so that
// what it executes comes through the instruction cache cold.)
__device__ __forceinline__ void block_scan2(uint32_t& a, uint32_t& b, uint32_t& ta, uint32_t& tb, uint2* warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    uint32_t xa = a, xb = b;
    uint32_t ia = 0, ib = 0, ca = 0, cb = 0;
#pragma unroll 1
    for (int level = 0; level < 2; ++level) {  // within the warp, then over the warps' sums
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t ya = __shfl_up_sync(kFull, xa, o), yb = __shfl_up_sync(kFull, xb, o);
            if (lane >= o) {
                xa = add_sat(xa, ya);
                xb = add_sat(xb, yb);
            }
        }
        if (level == 0) {
            ia = __shfl_up_sync(kFull, xa, 1);
            ib = __shfl_up_sync(kFull, xb, 1);
            if (lane == 0) ia = ib = 0;
            if (lane == 31) warps[warp] = make_uint2(xa, xb);
            __syncthreads();
            const uint2 w = lane < nw ? warps[lane] : make_uint2(0u, 0u);
            xa = w.x;
            xb = w.y;
        }
    }
    ta = __shfl_sync(kFull, xa, 31);
    tb = __shfl_sync(kFull, xb, 31);
    ca = __shfl_sync(kFull, xa, max(0, warp - 1));
    cb = __shfl_sync(kFull, xb, max(0, warp - 1));
    a = warp ? add_sat(ca, ia) : ia;
    b = warp ? add_sat(cb, ib) : ib;
}

// Largest s in [0, n) with P[s] <= x (P[0] = 0 <= x, P non-decreasing).
__device__ __forceinline__ int find_run(const int* P, int n, int x) {
    int lo = 0, hi = n - 1;
#pragma unroll 1
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (P[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

}  // namespace

// The scan of an extend step; the sums before each sequence go to tok and blk ([N + 1]) when the step is possible.
struct ExtendScan {
    int F, T, E;  // free blocks before the step, its tokens and its blocks (0 for a refused step)
    bool ok;
};
__device__ __forceinline__ ExtendScan scan_extend(const ExtendArgs& a, int* tok, int* blk, int* past, bool report) {
    __shared__ uint2 warps[32];
    const int tid = threadIdx.x, N = a.N, mask = (1 << a.shift) - 1;
    const int per = (N + blockDim.x - 1) / blockDim.x;
    const int lo = min(tid * per, N), hi = min(lo + per, N);
    const int F = *a.free_count;
    const int cap = a.MB << a.shift;
    uint32_t nt = 0, nb = 0;
    bool bad = false;
#pragma unroll 1
    for (int s = lo; s < hi; ++s) {
        const int L = a.past_lens[s], n = a.new_lens[s];
        if (L < 0 || n < 0 || L > cap || n > cap - L) {
            bad = true;
            continue;
        }
        const int e = ((L + n + mask) >> a.shift) - ((L + mask) >> a.shift);
        past[s] = L;
        tok[s] = n;
        blk[s] = e;
        nt = add_sat(nt, n);
        nb = add_sat(nb, e);
    }
    uint32_t total_t, total_b;
    block_scan2(nt, nb, total_t, total_b, warps);
    bad = __syncthreads_or(bad);
    const bool no_room = F < 0 || F > a.NB || total_b > static_cast<uint32_t>(F);
    const bool ok = !bad && !no_room && total_t <= static_cast<uint32_t>(a.max_tokens);
    if (ok) {
#pragma unroll 1
        for (int s = lo; s < hi; ++s) {
            const int n = tok[s], e = blk[s];
            tok[s] = static_cast<int>(nt);
            blk[s] = static_cast<int>(nb);
            nt += n;
            nb += e;
        }
        if (tid == 0) {
            tok[N] = static_cast<int>(total_t);
            blk[N] = static_cast<int>(total_b);
        }
    } else if (report && tid == 0) {
        raise_error(a.err, (bad || total_t > static_cast<uint32_t>(a.max_tokens) ? PKV_DEVERR_BAD_LENGTH : 0) | (no_room ? PKV_DEVERR_BAD_SLOT : 0));
    }
    __syncthreads();
    return {F, ok ? static_cast<int>(total_t) : 0, ok ? static_cast<int>(total_b) : 0, ok};
}

// The lengths and the free count after the step, in place perhaps: for a CTA after which nobody reads the old ones.
__device__ __forceinline__ void write_extend_state(const ExtendArgs& a, const ExtendScan& r, const int* tok, const int* past) {
#pragma unroll 1
    for (int s = threadIdx.x; s < a.N; s += blockDim.x)
        a.seq_lens[s] = r.ok ? past[s] + (tok[s + 1] - tok[s]) : a.past_lens[s];  // a refused step leaves them
    if (threadIdx.x == 0) *a.new_free_count = r.F - r.E;
}

__global__ void __launch_bounds__(1024) extend_sequences_kernel(const ExtendArgs a, bool write_state) {
    extern __shared__ int smem[];
    int* tok = smem;              // [N + 1] exclusive sums of the new tokens
    int* blk = tok + a.N + 1;     // [N + 1] exclusive sums of the new blocks
    int* past = blk + a.N + 1;    // [N]
    const int tid = threadIdx.x, N = a.N, mask = (1 << a.shift) - 1;
    const int width = static_cast<int>(gridDim.x * blockDim.x), at = static_cast<int>(blockIdx.x * blockDim.x) + tid;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const ExtendScan r = scan_extend(a, tok, blk, past, blockIdx.x == 0);
    const int F = r.F, T = r.T, E = r.E;

    // ---- the new blocks' table entries and the new tokens' slots.  A refused step has neither: every slot is -1.
    auto free_id = [&](int e) {  // the e-th block taken by the step; -1 if the stack's entry is no block
        const int id = __ldg(a.free_blocks + (F - 1 - e));
        return id >= 0 && id < a.NB ? id : -1;
    };
#pragma unroll 1
    for (int e = at; e < E; e += width) {
        const int s = find_run(blk, N, e);
        const int id = free_id(e);
        if (id < 0) raise_error(a.err, PKV_DEVERR_BAD_BLOCK);
        a.tables[static_cast<size_t>(s) * a.MB + ((past[s] + mask) >> a.shift) + (e - blk[s])] = id;
    }
    const int lane = tid & 31, runs = a.runs;
#pragma unroll 1
    for (int64_t i = static_cast<int64_t>(at >> 5) * (32 * runs); i < a.max_tokens; i += static_cast<int64_t>(width) * runs) {
        int s = -1;
#pragma unroll 1
        for (int t = static_cast<int>(i) + lane, u = 0; u < runs && t < a.max_tokens; ++u, t += 32) {
            int64_t slot = -1;
            if (t < T) {
                if (s < 0 || tok[s + 1] <= t) s = find_run(tok, N, t);
                const int L = past[s], p = L + t - tok[s], j = p >> a.shift, j_new = (L + mask) >> a.shift;
                int id;
                if (j >= j_new) {
                    id = free_id(blk[s] + j - j_new);
                } else {
                    id = a.tables[static_cast<size_t>(s) * a.MB + j];
                    if (id < 0 || id >= a.NB) {
                        id = -1;
                        raise_error(a.err, PKV_DEVERR_BAD_BLOCK);
                    }
                }
                if (id >= 0) slot = (static_cast<int64_t>(id) << a.shift) + (p & mask);
            }
            a.slots[t] = slot;
        }
    }

    // ---- the step's index arrays, and its state
#pragma unroll 1
    for (int s = at; s <= N; s += width) {
        if (a.cu_q) a.cu_q[s] = r.ok ? tok[s] : 0;
        if (a.q_starts && s < N) a.q_starts[s] = r.ok ? past[s] : a.past_lens[s];
    }
    if (write_state && blockIdx.x == 0) write_extend_state(a, r, tok, past);
}

// In place, after every CTA of extend_sequences_kernel.
__global__ void __launch_bounds__(1024) extend_state_kernel(const ExtendArgs a) {
    extern __shared__ int smem[];
    int* tok = smem;
    int* past = tok + 2 * (a.N + 1);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const ExtendScan r = scan_extend(a, tok, tok + a.N + 1, past, false);
    write_extend_state(a, r, tok, past);
}

// The scan of a release; the sums before each sequence go to blk ([N + 1]), the lengths after it to len ([N]).
struct ReleaseScan {
    int F, E;
    bool ok;
};
__device__ __forceinline__ ReleaseScan scan_release(const ReleaseArgs& a, int* blk, int* len, bool report) {
    __shared__ uint2 warps[32];
    const int tid = threadIdx.x, N = a.N, mask = (1 << a.shift) - 1;
    const int per = (N + blockDim.x - 1) / blockDim.x;
    const int lo = min(tid * per, N), hi = min(lo + per, N);
    const int F = *a.free_count;
    const int cap = a.MB << a.shift;
    uint32_t n = 0, none = 0;
    bool bad = false;
#pragma unroll 1
    for (int s = lo; s < hi; ++s) {
        const int L = a.past_lens[s], k = a.keep_blocks ? a.keep_blocks[s] : 0;
        const bool done = a.finished[s] != 0;
        if (L < 0 || L > cap || k < 0) {
            bad = true;
            continue;
        }
        len[s] = done ? 0 : L;
        blk[s] = done ? max(0, ((L + mask) >> a.shift) - k) : 0;
        n = add_sat(n, blk[s]);
    }
    uint32_t total, zero;
    block_scan2(n, none, total, zero, warps);
    bad = __syncthreads_or(bad);
    const bool no_room = F < 0 || F > a.NB || total > static_cast<uint32_t>(a.NB - F);
    const bool ok = !bad && !no_room;
    if (ok) {
#pragma unroll 1
        for (int s = lo; s < hi; ++s) {
            const int e = blk[s];
            blk[s] = static_cast<int>(n);
            n += e;
        }
        if (tid == 0) blk[N] = static_cast<int>(total);
    } else if (report && tid == 0) {
        raise_error(a.err, (bad ? PKV_DEVERR_BAD_LENGTH : 0) | (no_room ? PKV_DEVERR_BAD_SLOT : 0));
    }
    __syncthreads();
    return {F, ok ? static_cast<int>(total) : 0, ok};
}

__device__ __forceinline__ void write_release_state(const ReleaseArgs& a, const ReleaseScan& r, const int* len) {
#pragma unroll 1
    for (int s = threadIdx.x; s < a.N; s += blockDim.x) a.seq_lens[s] = r.ok ? len[s] : a.past_lens[s];
    if (threadIdx.x == 0) *a.new_free_count = r.F + r.E;
}

__global__ void __launch_bounds__(1024) release_sequences_kernel(const ReleaseArgs a, bool write_state) {
    extern __shared__ int smem[];
    int* blk = smem;
    int* len = blk + a.N + 1;
    const int width = static_cast<int>(gridDim.x * blockDim.x), at = static_cast<int>(blockIdx.x * blockDim.x + threadIdx.x);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const ReleaseScan r = scan_release(a, blk, len, blockIdx.x == 0);
#pragma unroll 1
    for (int e = at; e < r.E; e += width) {
        const int s = find_run(blk, a.N, e);
        const int k = a.keep_blocks ? __ldg(a.keep_blocks + s) : 0;
        int id = __ldg(a.tables + static_cast<size_t>(s) * a.MB + k + (e - blk[s]));
        if (id < 0 || id >= a.NB) {
            id = -1;
            raise_error(a.err, PKV_DEVERR_BAD_BLOCK);
        }
        a.free_blocks[r.F + e] = id;
    }
    if (write_state && blockIdx.x == 0) write_release_state(a, r, len);
}

// In place, after every CTA of release_sequences_kernel.
__global__ void __launch_bounds__(1024) release_state_kernel(const ReleaseArgs a) {
    extern __shared__ int smem[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const ReleaseScan r = scan_release(a, smem, smem + a.N + 1, false);
    write_release_state(a, r, smem + a.N + 1);
}

namespace {

// Items (slots, or table entries) per CTA while there are SMs, a thread each.  With 4096, 8192 slots took 6.0 us instead of
// 4.6 and a release of 64 sequences 4.4 instead of 3.7.
constexpr int64_t kPerCta = 1024;
// Most consecutive slots (32 apart) of a thread, which are mostly the same sequence's: 1.06 M slots took 7.8 us with 8 and 16,
// 8.9 with 4, and 9.8 with 1.
constexpr int64_t kRuns = 8;

struct Shape {
    int grid, block;
};
Shape shape_of(int N, int64_t items, int sms) {
    return {static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(sms, (items + kPerCta - 1) / kPerCta))),
            N <= 256 && items <= 1024 ? 256 : 1024};
}

// Dynamic shared memory that every kernel may have without being allowed more: 48 KB less the static part (256 bytes, the
// scan's), rounded down.
constexpr size_t kFreeSmem = 47 * 1024;

// The kernel, and behind it the state kernel when the state is updated in place and there is more than one CTA to read it.
// `most`: dynamic shared memory of the largest batch.  A limit is always raised to that, so that no call lowers it between
// another host thread's raising and launching.
template <class Kernel, class State, class Args>
cudaError_t launch(Kernel kern, State state, const Args& a, bool in_place, Shape shape, size_t smem, size_t most,
                   cudaStream_t stream) {
    if (smem > kFreeSmem) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(state, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
        if (e != cudaSuccess) return e;
    }
    const bool second = in_place && shape.grid > 1;
    kern<<<shape.grid, shape.block, smem, stream>>>(a, !second);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !second) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(1024);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, state, a);
}

}  // namespace

static size_t extend_smem(int N) { return (3 * static_cast<size_t>(N) + 2) * 4; }
static size_t release_smem(int N) { return (2 * static_cast<size_t>(N) + 1) * 4; }

cudaError_t launch_extend_sequences(const ExtendArgs& a, int sms, cudaStream_t stream) {
    const bool in_place = a.seq_lens == a.past_lens || a.new_free_count == a.free_count;
    const Shape shape = shape_of(a.N, a.max_tokens, sms);
    ExtendArgs b = a;
    const int64_t threads = static_cast<int64_t>(shape.grid) * shape.block;
    // (a small step's slots are half padding, which would leave half of one CTA's warps idle: 256 slots 4.6 instead of 3.7 us)
    b.runs = shape.grid == 1 ? 1 : static_cast<int>(std::max<int64_t>(1, std::min(kRuns, (a.max_tokens + threads - 1) / threads)));
    return launch(extend_sequences_kernel, extend_state_kernel, b, in_place, shape, extend_smem(a.N),
                  extend_smem(kMaxTableSeqs), stream);
}

cudaError_t launch_release_sequences(const ReleaseArgs& a, int sms, cudaStream_t stream) {
    const bool in_place = a.seq_lens == a.past_lens || a.new_free_count == a.free_count;
    return launch(release_sequences_kernel, release_state_kernel, a, in_place,
                  shape_of(a.N, static_cast<int64_t>(a.N) * a.MB, sms), release_smem(a.N), release_smem(kMaxTableSeqs), stream);
}

}  // namespace pkv
