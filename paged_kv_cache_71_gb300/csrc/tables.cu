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
// The work is a scan over the batch and then independent writes, so a call is bound by latency until its writes fill
// some SMs.  One CTA, or for many writes one cluster of CTAs, runs the whole call: every CTA scans the whole batch for
// itself (at most 8 sequences a thread), keeps the sums in shared memory and writes its part; the cluster barrier,
// which every CTA passes only after its last read of the lengths, lets the first CTA then write them in place.
#include <algorithm>

#include "tables.cuh"

namespace pkv {

namespace {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Block-wide exclusive sums of two values per thread (the first in 64 bits); returns the totals in ta, tb.
__device__ __forceinline__ void block_scan2(int64_t& a, int& b, int64_t& ta, int& tb, int64_t* wa, int* wb) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int64_t ia = a;
    int ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ya = __shfl_up_sync(kFull, ia, o);
        const int yb = __shfl_up_sync(kFull, ib, o);
        if (lane >= o) {
            ia += ya;
            ib += yb;
        }
    }
    if (lane == 31) {
        wa[warp] = ia;
        wb[warp] = ib;
    }
    __syncthreads();
    int64_t ca = lane < nw ? wa[lane] : 0;
    int cb = lane < nw ? wb[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ya = __shfl_up_sync(kFull, ca, o);
        const int yb = __shfl_up_sync(kFull, cb, o);
        if (lane >= o) {
            ca += ya;
            cb += yb;
        }
    }
    ta = __shfl_sync(kFull, ca, 31);
    tb = __shfl_sync(kFull, cb, 31);
    const int64_t pa = __shfl_sync(kFull, ca, warp == 0 ? 0 : warp - 1);
    const int pb = __shfl_sync(kFull, cb, warp == 0 ? 0 : warp - 1);
    a = ia - a + (warp ? pa : 0);
    b = ib - b + (warp ? pb : 0);
}

// Largest s in [0, n) with P[s] <= x (P[0] = 0 <= x, P non-decreasing).
__device__ __forceinline__ int find_run(const int* P, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (P[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

constexpr int kRun = 4;  // consecutive items per thread: one search serves them

}  // namespace

__global__ void __launch_bounds__(1024) extend_sequences_kernel(const ExtendArgs a) {
    extern __shared__ int smem[];
    __shared__ int64_t wa[32];
    __shared__ int wb[32];
    int* tok = smem;              // [N + 1] exclusive sums of the new tokens
    int* blk = tok + a.N + 1;     // [N + 1] exclusive sums of the new blocks
    int* past = blk + a.N + 1;    // [N]
    const int tid = threadIdx.x, N = a.N, S = 1 << a.shift, mask = S - 1;
    const uint32_t rank = cluster_rank();
    const int width = static_cast<int>(cluster_size() * blockDim.x), at = static_cast<int>(rank * blockDim.x) + tid;

    // ---- the scan: new tokens and new blocks before each sequence
    const int per = (N + blockDim.x - 1) / blockDim.x;
    const int lo = min(tid * per, N), hi = min(lo + per, N);
    const int F = *a.free_count;
    const int64_t cap = static_cast<int64_t>(a.MB) << a.shift;
    int64_t nt = 0;
    int nb = 0;
    bool bad = false;
    for (int s = lo; s < hi; ++s) {
        const int L = a.past_lens[s], n = a.new_lens[s];
        if (L < 0 || n < 0 || static_cast<int64_t>(L) + n > cap) {
            bad = true;
            continue;
        }
        past[s] = L;
        nt += n;
        nb += ((L + n + mask) >> a.shift) - ((L + mask) >> a.shift);
    }
    int64_t total_t;
    int total_b;
    block_scan2(nt, nb, total_t, total_b, wa, wb);
    bad = __syncthreads_or(bad);
    const bool no_room = F < 0 || F > a.NB || total_b > F;
    const bool ok = !bad && !no_room && total_t <= a.max_tokens;
    if (ok) {
        for (int s = lo; s < hi; ++s) {
            const int L = past[s], n = a.new_lens[s];
            tok[s] = static_cast<int>(nt);
            blk[s] = nb;
            nt += n;
            nb += ((L + n + mask) >> a.shift) - ((L + mask) >> a.shift);
        }
        if (tid == 0) {
            tok[N] = static_cast<int>(total_t);
            blk[N] = total_b;
        }
    } else if (rank == 0 && tid == 0) {
        raise_error(a.err, (bad || total_t > a.max_tokens ? PKV_DEVERR_BAD_LENGTH : 0) | (no_room ? PKV_DEVERR_BAD_SLOT : 0));
    }
    __syncthreads();

    // ---- the new blocks' table entries and the new tokens' slots.  A refused step has neither: every slot is -1.
    const int T = ok ? static_cast<int>(total_t) : 0, E = ok ? total_b : 0;
    auto free_id = [&](int e) {  // the e-th block taken by the step; -1 (and an error) if the stack's entry is no block
        const int id = __ldg(a.free_blocks + (F - 1 - e));
        return id >= 0 && id < a.NB ? id : -1;
    };
    for (int e = at; e < E; e += width) {
        const int s = find_run(blk, N, e);
        const int id = free_id(e);
        if (id < 0) raise_error(a.err, PKV_DEVERR_BAD_BLOCK);
        a.tables[static_cast<size_t>(s) * a.MB + ((past[s] + mask) >> a.shift) + (e - blk[s])] = id;
    }
    for (int64_t i = static_cast<int64_t>(at) * kRun; i < a.max_tokens; i += static_cast<int64_t>(width) * kRun) {
        const int t0 = static_cast<int>(i);
        int s = t0 < T ? find_run(tok, N, t0) : N;
        int64_t out[kRun];
        int j_seen = -1, s_seen = -1, id = -1;
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            const int t = t0 + u;
            out[u] = -1;
            if (t >= T) continue;
            while (tok[s + 1] <= t) ++s;  // tok[N] = T > t
            const int L = past[s], p = L + t - tok[s], j = p >> a.shift, j_new = (L + mask) >> a.shift;
            if (j != j_seen || s != s_seen) {  // a block's first token here
                if (j >= j_new) {
                    id = free_id(blk[s] + j - j_new);
                } else {
                    id = a.tables[static_cast<size_t>(s) * a.MB + j];
                    if (id < 0 || id >= a.NB) {
                        id = -1;
                        raise_error(a.err, PKV_DEVERR_BAD_BLOCK);
                    }
                }
                j_seen = j;
                s_seen = s;
            }
            if (id >= 0) out[u] = (static_cast<int64_t>(id) << a.shift) + (p & mask);
        }
        if (t0 + kRun <= a.max_tokens && (reinterpret_cast<uintptr_t>(a.slots) & 15u) == 0) {
#pragma unroll
            for (int u = 0; u < kRun; u += 2)
                *reinterpret_cast<longlong2*>(a.slots + t0 + u) = make_longlong2(out[u], out[u + 1]);
        } else {
#pragma unroll
            for (int u = 0; u < kRun; ++u)
                if (t0 + u < a.max_tokens) a.slots[t0 + u] = out[u];
        }
    }

    // ---- the state, which may be the input arrays: written once no CTA reads them any more
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    for (int s = tid; s < N; s += blockDim.x) {
        const int L = ok ? past[s] : a.past_lens[s];  // a refused step leaves the lengths as they are
        if (a.q_starts) a.q_starts[s] = L;
        if (a.cu_q) a.cu_q[s] = ok ? tok[s] : 0;
        a.seq_lens[s] = ok ? L + (tok[s + 1] - tok[s]) : L;
    }
    if (tid == 0) {
        if (a.cu_q) a.cu_q[N] = T;
        *a.new_free_count = F - E;
    }
}

__global__ void __launch_bounds__(1024) release_sequences_kernel(const ReleaseArgs a) {
    extern __shared__ int smem[];
    __shared__ int64_t wa[32];
    __shared__ int wb[32];
    int* blk = smem;            // [N + 1] exclusive sums of the released blocks
    int* len = blk + a.N + 1;   // [N] the lengths after the call
    const int tid = threadIdx.x, N = a.N, mask = (1 << a.shift) - 1;
    const uint32_t rank = cluster_rank();
    const int width = static_cast<int>(cluster_size() * blockDim.x), at = static_cast<int>(rank * blockDim.x) + tid;

    const int per = (N + blockDim.x - 1) / blockDim.x;
    const int lo = min(tid * per, N), hi = min(lo + per, N);
    const int F = *a.free_count;
    const int64_t cap = static_cast<int64_t>(a.MB) << a.shift;
    auto count = [&](int s, bool& bad) {  // blocks that sequence s hands back
        const int L = a.past_lens[s], k = a.keep_blocks ? a.keep_blocks[s] : 0;
        if (L < 0 || L > cap || k < 0) {
            bad = true;
            return 0;
        }
        len[s] = a.finished[s] ? 0 : L;
        return a.finished[s] ? max(0, ((L + mask) >> a.shift) - k) : 0;
    };
    int64_t n64 = 0;
    int none = 0;
    bool bad = false;
    for (int s = lo; s < hi; ++s) n64 += count(s, bad);
    int64_t total;
    int zero;
    block_scan2(n64, none, total, zero, wa, wb);
    bad = __syncthreads_or(bad);
    const bool no_room = F < 0 || F > a.NB || total > a.NB - F;
    const bool ok = !bad && !no_room;
    if (ok) {
        for (int s = lo; s < hi; ++s) {
            blk[s] = static_cast<int>(n64);
            n64 += count(s, bad);
        }
        if (tid == 0) blk[N] = static_cast<int>(total);
    } else if (rank == 0 && tid == 0) {
        raise_error(a.err, (bad ? PKV_DEVERR_BAD_LENGTH : 0) | (no_room ? PKV_DEVERR_BAD_SLOT : 0));
    }
    __syncthreads();
    const int E = ok ? static_cast<int>(total) : 0;
    for (int64_t i = static_cast<int64_t>(at) * kRun; i < E; i += static_cast<int64_t>(width) * kRun) {
        int s = find_run(blk, N, static_cast<int>(i));
#pragma unroll
        for (int u = 0; u < kRun; ++u) {
            const int e = static_cast<int>(i) + u;
            if (e >= E) break;
            while (blk[s + 1] <= e) ++s;  // blk[N] = E > e
            const int k = a.keep_blocks ? a.keep_blocks[s] : 0;
            int id = a.tables[static_cast<size_t>(s) * a.MB + k + (e - blk[s])];
            if (id < 0 || id >= a.NB) {
                id = -1;
                raise_error(a.err, PKV_DEVERR_BAD_BLOCK);
            }
            a.free_blocks[F + e] = id;
        }
    }
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    for (int s = tid; s < N; s += blockDim.x) a.seq_lens[s] = ok ? len[s] : a.past_lens[s];
    if (tid == 0) *a.new_free_count = F + E;
}

namespace {

// One CTA for a step of few writes; one cluster of kCluster CTAs for more.  A CTA of 1024 threads writes kSingle items
// about as fast as the cluster starts up and synchronises.
constexpr int kCluster = 8;
constexpr int64_t kSingle = 8192;

template <class Kernel, class Args>
cudaError_t launch(Kernel kern, const Args& a, int64_t items, size_t smem, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const int ncta = items > kSingle ? kCluster : 1;
    cfg.gridDim = dim3(ncta);
    cfg.blockDim = dim3(a.N <= 256 && items <= 1024 ? 256 : 1024);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ncta;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_extend_sequences(const ExtendArgs& a, cudaStream_t stream) {
    const size_t smem = (3 * static_cast<size_t>(a.N) + 2) * 4;
    return launch(extend_sequences_kernel, a, a.max_tokens, smem, stream);
}

cudaError_t launch_release_sequences(const ReleaseArgs& a, cudaStream_t stream) {
    const size_t smem = (2 * static_cast<size_t>(a.N) + 1) * 4;
    return launch(release_sequences_kernel, a, static_cast<int64_t>(a.N) * a.MB, smem, stream);
}

}  // namespace pkv
