// commit.cu -- the accepted path of each sequence's draft tree, and its K/V moved to consecutive slots in every layer
// (pkv_commit_tree).
//
// The path: token 0 of the run, then from token c the first later token i with parents[i] = c and draft[i] = target[c], until
// there is none.  A CTA stages its sequence's run in shared memory and warp 0 walks it, 32 candidates at a time; the walk is
// repeated by every CTA of the sequence (about 1 us) instead of a second launch.
//
// The move: the j-th token of the path, at run index i >= j, goes from position past + i to past + j.  Moves of a sequence
// may chain (a place that one token leaves is taken by a later one), so they happen as if in order of j: a thread owns a
// 16-byte column of the token rows, takes up to kBatch of them with loads before the stores, and what an earlier batch
// overwrote lies at run indexes below its last j, which no later token comes from (i >= j).
//
// Bound by latency: the launch, the run's loads, the walk, the table's, then a thread's loads and stores, few of them at a time
// where little moves.  256 ragged trees of 32 layers (bf16, 8 heads of 128; 78 MB, 11.5 us at the measured copy rate) from graphs:
// 19.3 us with pools that are not in L2 (six batches in turn), 14.7 with one batch over and over, most of which stays there.
// 8 trees 3.6 / 3.3 us.
#include <algorithm>

#include "commit.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;
// CTAs that an SM holds at a time (48 registers, 25 KB of shared memory).  The work split for 2, 3, 4, 5, 6, 8, 10, 16 of them: the 256
// trees, not in L2, 31.5 / 24.0 / 21.3 / 19.2 / 19.2 / 20.7 / 20.1 / 20.4 us, 48 trees of 64 in 80 layers (FP8, 20 MB)
// 11.0 / 9.5 / 8.9 / 8.4 / 8.5 / 8.3 / 9.8 / 9.8.
constexpr int kCtas = 5;

}  // namespace

__global__ void __launch_bounds__(kThreads, kCtas) commit_tree_kernel(const __grid_constant__ CommitArgs a) {
    __shared__ int parent[kMaxCommitRun], draft[kMaxCommitRun], target[kMaxCommitRun];
    __shared__ int path[kMaxCommitRun], from[kMaxCommitRun], to[kMaxCommitRun];
    __shared__ int counts[2];  // tokens of the path, moves
    const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const bool writes = blockIdx.y == 0;
    const int q0 = a.cu_q[s], q1 = a.cu_q[s + 1], past = a.past_lens[s];
    const bool bad_q = q0 < 0 || q1 < q0 || q1 > a.tokens;
    const int n = bad_q ? 0 : q1 - q0;
    const bool bad = bad_q || past < 0 || n > kMaxCommitRun || static_cast<int64_t>(past) + n > (static_cast<int64_t>(a.MB) << a.shift);
    if (bad || n == 0) {
        if (writes) {
            if (tid == 0) {
                if (bad) raise_error(a.err, PKV_DEVERR_BAD_LENGTH);
                a.num_accepted[s] = 0;
                a.seq_lens[s] = past;
                a.next_tokens[s] = -1;
                if (a.keep_blocks) a.keep_blocks[s] = past > 0 ? ((past - 1) >> a.shift) + 1 : 0;
            }
            for (int i = tid; i < n; i += kThreads) a.accepted[q0 + i] = -1;
        }
        return;
    }
    for (int i = tid; i < n; i += kThreads) {
        parent[i] = a.parents[q0 + i];
        draft[i] = a.draft[q0 + i];
        target[i] = a.target[q0 + i];
    }
    __syncthreads();
    if (tid < 32) {
        int cur = 0, count = 1;
        if (lane == 0) path[0] = 0;
        for (int base = 0; base < n; base += 32) {  // the next token of the path lies behind the last one
            const int i = base + lane;
            while (true) {
                const bool fits = i > cur && i < n && parent[i] == cur && draft[i] == target[cur];
                const unsigned some = __ballot_sync(0xffffffffu, fits);
                if (!some) break;
                cur = base + __ffs(some) - 1;
                if (lane == 0) path[count] = cur;
                ++count;
            }
        }
        __syncwarp();
        int moves = 0;
        for (int base = 0; base < count; base += 32) {
            const int j = base + lane;
            bool move = j < count && path[j] != j;
            int src = 0, dst = 0;
            if (move) {
                const int p = past + path[j], d = past + j, mask = (1 << a.shift) - 1;
                const int64_t row = static_cast<int64_t>(s) * a.MB;
                const int sb = a.tables[row + (p >> a.shift)], db = a.tables[row + (d >> a.shift)];
                if (sb < 0 || sb >= a.NB || db < 0 || db >= a.NB) {
                    move = false;
                    if (writes) raise_error(a.err, PKV_DEVERR_BAD_BLOCK);
                }
                src = (sb << a.shift) + (p & mask);
                dst = (db << a.shift) + (d & mask);
            }
            const unsigned which = __ballot_sync(0xffffffffu, move);
            if (move) {
                const int at = moves + __popc(which & ((1u << lane) - 1));
                from[at] = src;
                to[at] = dst;
            }
            moves += __popc(which);
        }
        if (lane == 0) {
            counts[0] = count;
            counts[1] = moves;
        }
    }
    __syncthreads();
    const int count = counts[0], moves = counts[1];
    if (writes) {
        for (int i = tid; i < n; i += kThreads) a.accepted[q0 + i] = i < count ? path[i] : -1;
        if (tid == 0) {
            a.num_accepted[s] = count;
            a.seq_lens[s] = past + count;
            a.next_tokens[s] = target[path[count - 1]];
            if (a.keep_blocks) a.keep_blocks[s] = ((past + count - 1) >> a.shift) + 1;
        }
    }
    if (moves == 0) return;
    const int l0 = blockIdx.y * a.per_cta, nl = min(a.per_cta, a.layers - l0);
    for (int i = tid; i < nl * 2 * a.vecs; i += kThreads) {
        const int row = i / a.vecs, vec = i - row * a.vecs;
        uint4* base = ((row & 1) ? a.v : a.k)[l0 + (row >> 1)] + vec;
        for (int m = 0; m < moves; m += kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (m + k < moves) x[k] = base[static_cast<int64_t>(from[m + k]) * a.vecs];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (m + k < moves) base[static_cast<int64_t>(to[m + k]) * a.vecs] = x[k];
        }
    }
}

cudaError_t launch_commit_tree(CommitArgs& a, int num_seqs, int sms, cudaStream_t stream) {
    // as many CTAs as the SMs hold at a time, a layer each at least
    const int64_t fill = static_cast<int64_t>(sms) * kCtas;
    a.per_cta = static_cast<int>(std::max<int64_t>(1, (static_cast<int64_t>(num_seqs) * a.layers + fill - 1) / fill));
    a.per_cta = std::min(a.per_cta, a.layers);
    const dim3 grid(num_seqs, (a.layers + a.per_cta - 1) / a.per_cta);
    commit_tree_kernel<<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace pkv
