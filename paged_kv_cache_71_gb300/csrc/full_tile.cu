// full_tile.cu -- attention of many query rows over a paged K/V range without a mask: cross attention to an encoder's
// states (pkv_paged_cross_attention) and the shared prefixes of a decode batch (pkv_paged_attention_decode_prefix).
//
// Chunks and items are described in full_tile.cuh.  An item reads its keys once for all of its rows, in tiles of 64:
// S = Q K^T, P = 2^(S - m) with the running maximum m (log2 units), O += P V.
//
// Work split: the items are laid end to end in units, a key tile that serves two query tiles counting two and one that
// serves a single one counting one, item_units more for every item, rounded up to an even number, and cut into equal
// shares, one per CTA (SM); a cut in an item's first item_units falls before it.  An item that is cut, and every item of a
// shared prefix, leaves a partial record for each of its pieces; they join as
//   M = max m_i,  l = sum 2^(m_i - M) l_i,  O = sum 2^(m_i - M) O_i / l
// in a kernel launched beside this one: join_cuts_kernel (cross attention), join_rows_kernel (shared prefixes).
//
// (Cross attention with many long items: whole items in rounds first, see kRounds.)
//
// A CTA runs its share as one stream: TMEM, barriers and the K/V rings live through all of its items, and the copies of
// the next item's keys run while the current one ends.  Two groups, A and B (128 softmax threads, one per query row, a
// score and a P V warp, a Q slot, two score buffers and an output accumulator in TMEM each), work side by side: on an
// item's two query tiles, or, when it has one, on alternate key tiles of the same rows; the item's owner (A and B in turn)
// then joins the two accumulators.
//   * warps 0-3 and 4-7: the groups' softmax.  A group's first thread also copies its next item's Q, once the scores of
//     its last key tile of the current item are there (nothing reads the old Q any more);
//   * warps 9 and 13: the groups' scores (tcgen05), one key tile ahead of P V, which warps 11 and 15 issue.  One warp for
//     both groups' scores and one for both groups' P V, tried first, took 1044 cycles per issue (waits, loop and issue in
//     turn), 2090 per key tile of two query tiles;
//   * warps 8 and 10: copy the K and V tiles (TMA, one block of the block table per copy, one lane per block);
//   * INT8 caches: warps 16-19 widen the codes to f16, two warps per operand, half of the rows each.
// Hand-offs are mbarriers; every wait is bounded.  On a timeout a role records the error and does nothing more, the CTA
// drains its own MMAs and copies (bounded) and frees TMEM.
//
// What bounds it: a key tile of two query tiles takes 1780 cycles (bf16) where its MMAs need 1296 (scores 128 x 64 x 16 from
// shared memory 48.7 cycles each, P V 128 x 128 x 16 with P in TMEM 64.6).  The rest is the chain of hand-offs through the two
// score buffers (P over the scores that it was made of): softmax 1370 cycles, P seen by its warp 370, P V 570, the next scores
// 1030.  Half of the score MMAs, half of the P V MMAs or no exponentials at all take 4 to 6% off, no more.  Tried and slower:
// P in columns of its own beside one score buffer per group (+11%) or three between the groups (+20%), one arrival per warp
// instead of one per thread (+3%).
#include <algorithm>

#include "full_tile.cuh"
#include "prefill_tile.cuh"

namespace pkv {

namespace {

// Fewest units in a share (even): a piece costs a record and its joining whatever its length.  128 sequences over 800 INT8
// tokens took 33 us with 4, 29 with 8, 33 with 16.
constexpr int kMinShare = 8;
// What an item costs beside its key tiles, which count w units each (w: query tiles).  4 units for either kind, tried first,
// left the SMs with many short items of two query tiles behind: 12 prompts over long states took 810 us against 785.
__device__ constexpr int item_units(int w) { return 4 * w; }
constexpr int kBatch = 128;    // items that a CTA lists at a time
constexpr int kEmpty = 512;    // chunks without keys that it lists
// Cross attention, at least two items for every CTA, and long ones: the items, ordered by KV head, are first handed out whole,
// one per CTA and round, so that the query tiles of one head run side by side over the same keys; what is left (an item or
// two per CTA) is cut so that all CTAs end together.  Cut from the start, the stream's places lie anywhere in a head's keys
// and every query tile reads them from DRAM: 3.9 GB instead of 1.3 for 12 prompts of 1000 tokens over states of 4500
// (790 us; 717 with rounds; both in short loops, see kRegsSoftmax), and 2048 rows over 8192 keys in 8 sequences 472 us instead of 430.  With shorter items the
// keys stay in L2 anyway, and the rounds' plan (4 us) is not worth it.
constexpr int kRounds = 64;      // most rounds
constexpr int kRoundUnits = 64;  // fewest units per item, on average

template <int NARROW>
struct FullPlan {
    static constexpr int kStages = NARROW == 0 ? 4 : NARROW == 1 ? 8 : 2;  // K and V ring depth (what the MMAs read)
    static constexpr int kStage = NARROW == 1 ? kStgSlot : 2 * kKvHalf;
    static constexpr int kSlots = NARROW == 2 ? 4 : 0;                     // INT8: staging slots per operand
    static constexpr int kCopies = NARROW == 2 ? kSlots : kStages;         // depth of the ring that TMA writes
    static constexpr int kOffK = 4 * kQHalf;                               // the Q slots of A and B first
    static constexpr int kOffV = kOffK + kStages * kStage;
    static constexpr int kOffStg = kOffV + kStages * kStage;
    static constexpr int kOffMeta = kOffStg + 2 * kSlots * kStgSlot;
    static constexpr int kThreads = NARROW == 2 ? 640 : 512;
    // registers per thread after the split: 256 x 176 + 256 x 80 = 256 x 184 + 256 x 72 = 512 x 128, what the launch gives;
    // 256 x 168 + 384 x 48 = 640 x 96.  bf16 168 / 176 / 184 / 192 / 200 softmax registers: cross_prompts 706 / 703 / 714 /
    // 701 / 702 us (in loops below 0.1 s; 749 in loops of seconds), 256 queries over 32768 keys 206 / 203 / 209 / 207 / 207;
    // FP8: those queries 246 / 252 / 241 / 247 / 250.
    static constexpr int kRegsSoftmax = NARROW == 2 ? 168 : NARROW == 1 ? 184 : 176;
    static constexpr int kRegsOther = NARROW == 2 ? 48 : NARROW == 1 ? 72 : 80;
};

// mbarriers
constexpr int kFKFull = 0, kFKEmpty = 8, kFVFull = 16, kFVEmpty = 24;  // + stage
constexpr int kFS = 32, kFP = 36, kFPV = 40;        // + 2 * group + buffer: scores written, P written, P V done
constexpr int kFQ = 44, kFO = 48;                   // + group: Q landed, O complete
constexpr int kFMl = 50, kFTaken = 52;              // + owner: the other group's (m, l) are in shared memory; owner has its O
constexpr int kFZero = 54;                          // V rows past the last key zeroed (items of two query tiles)
constexpr int kFVThere = 55;                        // + group: V with rows past the last key has landed
constexpr int kFDrain = 57;
constexpr int kFStg = 58, kFStgFree = 66;           // + 4 * (V ? 1 : 0) + slot
constexpr int kFBars = 74;
constexpr int kFTmem = 8 * kFBars, kFAbort = kFTmem + 4;  // byte offsets
constexpr int kFPart = kFAbort + 4;                 // per-warp sums of the plan's scan: units [32], items [32]
constexpr int kFMine = kFPart + 256;                // ints: x0, x1; the lister's chunk, item, first unit; items listed, more,
                                                    // the first item's index; + group: the V stage with rows to be zeroed
constexpr int kFItems = 912;
constexpr int kFMlOut = kFItems + 32 * kBatch;      // (m, l) of the other group's rows, [owner][128]
constexpr int kFUnits = kFMlOut + 2 * 128 * 8;      // the chunks' first units, [kMaxSeqs + 1]
constexpr int kFFirst = kFUnits + 4 * (kMaxSeqs + 1);  // and first items
constexpr int kFEnd = kFFirst + 4 * (kMaxSeqs + 1);
static_assert(kFMine + 52 <= kFItems, "meta slots overlap");

// One CTA's part of an item
struct Item {
    int q_row, tokens;  // the item's first row of q, its query tokens
    int keys, table;    // keys of the chunk, the block table entry of the first
    int j0, n;          // first key tile, key tiles
    int head_pair;      // KV head, two query tiles << 16
    int rec;            // 0: the result goes to out; 1: a record at the rows of (token, query head); 2: at the CTA's
};
static_assert(sizeof(Item) == 32, "item size");

// A chunk's work
struct Chunk {
    int q0, tokens, keys, table;
    int kt, w, ku;  // key tiles, units per key tile, units per item
    int items;
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Most units of a stream.  Only query ranges that overlap (malformed) can have more, the host bounds the others; the room up
// to INT_MAX, where sums of units stop, is for what is added to a total (the CTAs, an item's length).
constexpr int kMostUnits = 0x7fffffff - 4096;
__device__ __forceinline__ int add_units(int a, int b) {
    return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b), 0x7fffffffu));
}

__device__ __forceinline__ void store_v8(float* p, const float* v) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

}  // namespace


namespace {

// Bounded wait of a warp for a phase of an mbarrier; the warp is converged afterwards.
__device__ __forceinline__ bool warp_wait(uint32_t b, uint32_t parity, uint64_t limit_ns) {
    return __all_sync(kFull, mbar_wait_bounded(b, parity, limit_ns));
}

}  // namespace

template <int NARROW>
__global__ void __launch_bounds__(FullPlan<NARROW>::kThreads, 1)
    paged_full_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const PrefillArgs a, const FullArgs f) {
    using PL = FullPlan<NARROW>;
    constexpr int kStages = PL::kStages, kStage = PL::kStage, kCopies = PL::kCopies, kNT = PL::kThreads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem), bar = sb + PL::kOffMeta;
    uint8_t* meta = smem + PL::kOffMeta;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(meta + kFTmem);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(meta + kFAbort);
    int* part = reinterpret_cast<int*>(meta + kFPart);
    int* first_unit = reinterpret_cast<int*>(meta + kFUnits);
    int* first_item = reinterpret_cast<int*>(meta + kFFirst);
    volatile int* mine = reinterpret_cast<volatile int*>(meta + kFMine);
    Item* items = reinterpret_cast<Item*>(meta + kFItems);
    float2* ml_out = reinterpret_cast<float2*>(meta + kFMlOut);
    int* empty = reinterpret_cast<int*>(ml_out);  // while the plan is made: chunks without keys
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x, ncta = gridDim.x;
    const int g_shift = 31 - __clz(a.G);  // G divides 128
    const int rows_q = kRows >> g_shift, cta_q = 2 * rows_q, cta_shift = 8 - g_shift;
    const int n_chunks = a.nseq;

    if (tid < kFBars) {
        const int i = tid;
        int count = 1;
        if (i >= kFP && i < kFP + 4) count = 128;
        if (i >= kFMl && i <= kFZero) count = 128;
        if ((i >= kFKEmpty && i < kFVFull) || (i >= kFVEmpty && i < kFS)) count = 2;
        if (i == kFDrain) count = 4;
        if (NARROW == 2 && (i < kFKEmpty || (i >= kFVFull && i < kFVEmpty) || i >= kFStgFree)) count = 2;
        mbar_init(bar + 8 * i, count);
        fence_mbar_init();
    }
    if (tid == 0) {
        *abort_flag = 0;
        mine[11] = 0;
        prefetch_tensormap(&qmap);
    }
    if (warp == 8 && lane == 0) prefetch_tensormap(&kmap);
    if (warp == 10 && lane == 0) prefetch_tensormap(&vmap);
    if (warp == 11) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }

    __syncthreads();
    // ---- the plan.  A malformed chunk has nothing to do.
    auto load_chunk = [&](int c, bool report) {
        Chunk k;
        const int q0 = a.cu_q[c], q1 = a.cu_q[c + 1], kv = a.kv_lens[c];
        const bool bad_q = q0 < 0 || q1 < q0 || q1 > a.NQ;
        const bool bad = bad_q || kv < 0 || kv > a.MB * a.S || (f.prefix && (kv & (a.S - 1)) != 0);
        if (bad && report) raise_error(a.err, PKV_DEVERR_BAD_LENGTH);
        k.q0 = bad_q ? 0 : q0;
        k.tokens = bad_q ? 0 : q1 - q0;
        k.keys = bad ? -1 : kv;
        k.table = (f.prefix ? k.q0 : c) * a.MB;
        k.w = k.tokens > rows_q ? 2 : 1;
        k.kt = (max(k.keys, 0) + kKeys - 1) / kKeys;
        k.ku = k.kt > 0 ? (k.kt * k.w + item_units(k.w) + 1) & ~1 : 0;
        k.items = k.kt > 0 ? ((k.tokens + cta_q - 1) >> cta_shift) * a.Hkv : 0;
        return k;
    };
    // What [x0, x1) holds of item m (KV head and query tiles) of a chunk whose first unit is `start`, into the list.
    auto put_item = [&](int slot, const Chunk& k, int start, int m, int x0, int x1, int rounds, bool first) {
        const int n_tiles = (k.tokens + cta_q - 1) >> cta_shift;
        const int tile = rounds ? m % n_tiles : m / a.Hkv, h = rounds ? m / n_tiles : m - tile * a.Hkv, t0 = tile << cta_shift;
        const int Uk = start + m * k.ku, j0 = max(0, x0 - Uk - item_units(k.w)) >> (k.w - 1);
        Item it;
        it.q_row = k.q0 + t0;
        it.tokens = min(cta_q, k.tokens - t0);
        it.keys = k.keys;
        it.table = k.table;
        it.j0 = j0;
        it.n = min(k.kt, (min(Uk + k.ku, x1) - Uk - item_units(k.w)) >> (k.w - 1)) - j0;
        it.head_pair = h | ((it.tokens > rows_q ? 1 : 0) << 16);
        it.rec = !(f.prefix || it.n < k.kt) ? 0 : j0 > 0 ? 2 : 1;
        items[slot] = it;
        if (first) f.cuts[cta] = j0 > 0 ? make_int4(it.q_row, it.tokens | (h << 16), Uk + item_units(k.w), Uk + k.ku) : make_int4(0, 0, 0, 0);
    };
    // Items of a chunk that start before x1, but the last of them if x1 is among its first units.
    auto items_before = [&](const Chunk& k, int start, int x1) {
        return k.items == 0 || start + item_units(k.w) >= x1 ? 0 : min(k.items, ceil_div(x1 - start - item_units(k.w), k.ku));
    };
    // Each thread takes a contiguous run of chunks: (0) the sums of their units and items; (1) with what comes before
    // known, the place where this CTA's share starts; (2) the first batch of its items.
    {
        const int per = ceil_div(n_chunks, kNT);
        const int c_lo = min(tid * per, n_chunks), c_hi = min(c_lo + per, n_chunks);
        int sum = 0, count = 0, before = 0, items_at = 0, x0 = 0, x1 = 0;  // units and items; of the chunks before this thread's
        Chunk k = {};
        int rounds = 0;  // of whole items, one per CTA
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            int run = before, index = items_at;
#pragma unroll 1
            for (int c = c_lo; c < c_hi; ++c) {
                if (pass == 0 || per > 1) k = load_chunk(c, pass == 0 && cta == 0);
                const int units = k.items * k.ku;
                if (pass == 0) {
                    sum = add_units(sum, units);
                    count += k.items;
                    if (!f.prefix && k.keys == 0 && k.tokens > 0) {
                        const int e = atomicAdd(const_cast<int*>(mine) + 11, 1);
                        if (e < kEmpty) empty[e] = c;
                    }
                } else if (pass == 1) {
                    first_unit[c] = run;
                    if (run <= x0 && x0 < run + units && x0 < x1) {  // where this CTA starts
                        const int m = (x0 - run) / k.ku;
                        mine[2] = c;
                        mine[3] = m;
                        mine[4] = run;
                        mine[7] = index + m;
                    }
                } else if (x0 < x1 && run + units > x0 && run < x1) {
                    const int m0 = max(0, mine[7] - index), m1 = items_before(k, run, x1), slot0 = index - mine[7] + rounds;
                    const int m2 = min(m1, kBatch - slot0);
#pragma unroll 1
                    for (int m = m0; m < m2; ++m) put_item(slot0 + m, k, run, m, x0, x1, rounds, slot0 + m == rounds);
                    if (m2 > m0) atomicMax(const_cast<int*>(mine) + 5, slot0 + m2);
                    if (m1 > m2 && m2 >= m0 && slot0 + m0 <= kBatch) {  // the list is full: the next batch starts here
                        mine[2] = c;
                        mine[3] = m2;
                        mine[4] = run;
                        mine[6] = 1;
                    }
                }
                run += units;
                index += k.items;
            }
            if (pass == 2) break;
            if (pass == 1) {
                __syncthreads();
                continue;
            }
            int iu = sum, ic = count;
#pragma unroll 1
            for (int level = 0; level < 2; ++level) {  // within the warp, then over the warps' sums
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const int yu = __shfl_up_sync(kFull, iu, o), yc = __shfl_up_sync(kFull, ic, o);
                    if (lane >= o) {
                        iu = add_units(iu, yu);
                        ic = add_units(ic, yc);
                    }
                }
                if (level == 1) break;
                before = iu - sum;
                items_at = ic - count;
                if (lane == 31) {
                    part[warp] = iu;
                    part[32 + warp] = ic;
                }
                tc_fence_before();
                __syncthreads();
                tc_fence_after();
                iu = lane < kNT / 32 ? part[lane] : 0;
                ic = lane < kNT / 32 ? part[32 + lane] : 0;
            }
            int T = __shfl_sync(kFull, iu, 31);
            const int bu = __shfl_sync(kFull, iu, max(0, warp - 1));
            const int bc = __shfl_sync(kFull, ic, max(0, warp - 1)), M = __shfl_sync(kFull, ic, 31);
            if (warp) {
                before += bu;
                items_at += bc;
            }
            int share = 0x7fffffff;
            if (T > kMostUnits) {  // nothing is done
                T = 0;
                if (cta == 0 && tid == 0) raise_error(a.err, PKV_DEVERR_BAD_LENGTH);
            } else {
                share = max(kMinShare, (ceil_div(T, ncta) + 1) & ~1);
            }
            if (!f.prefix && M >= 2 * ncta && T / M >= kRoundUnits) rounds = min(kRounds, M / ncta - 1);
            if (tid == 0) {
                mine[5] = mine[12] = rounds;
                mine[6] = 0;
                f.cuts[cta] = make_int4(0, 0, 0, 0);
                if (cta == ncta - 1) *f.share = rounds ? 0 : share;
            }
            if (rounds == 0) {
                x0 = static_cast<int>(min(static_cast<int64_t>(cta) * share, static_cast<int64_t>(T)));
                x1 = static_cast<int>(min(static_cast<int64_t>(x0) + share, static_cast<int64_t>(T)));
                if (tid == 0) {
                    mine[0] = x0;
                    mine[1] = x1;
                }
                continue;
            }
            // Rounds: where the rest begins, then what each CTA still takes of it
            const int rest = rounds * ncta;  // the first item that is in no round
            int u = before, n = items_at;
#pragma unroll 1
            for (int c = c_lo; c < c_hi; ++c) {
                if (per > 1) k = load_chunk(c, false);
                first_unit[c] = u;
                first_item[c] = n;
                if (n <= rest && rest < n + k.items) mine[10] = u + (rest - n) * k.ku;
                u += k.items * k.ku;
                n += k.items;
            }
            if (tid == 0) {
                first_unit[n_chunks] = T;
                first_item[n_chunks] = M;
            }
            __syncthreads();
            auto chunk_of = [&](int item) {
                int lo = 0, hi = n_chunks - 1;
#pragma unroll 1
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (first_item[mid] <= item) lo = mid;
                    else hi = mid - 1;
                }
                return lo;
            };
            const int origin = mine[10];
            int part_c = 0;  // of the rest, for CTA tid
            if (tid < ncta) {
                int load = 0;
#pragma unroll 1
                for (int r = 0; r < rounds; ++r) {
                    const int c = chunk_of(r * ncta + tid);
                    load += (first_unit[c + 1] - first_unit[c]) / (first_item[c + 1] - first_item[c]);
                }
                part_c = max(0, share - load);
            }
            if (tid < rounds) {
                const int item = tid * ncta + cta, c = chunk_of(item), m = item - first_item[c];
                const Chunk w = load_chunk(c, false);
                const int U = first_unit[c] + m * w.ku;
                put_item(tid, w, first_unit[c], m, U, U + w.ku, rounds, false);
            }
            int upto = part_c;
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, upto, o);
                if (lane >= o) upto += y;
            }
            if (lane == 31) part[warp] = upto;
            __syncthreads();
            for (int w = 0; w < warp; ++w) upto += part[w];
            if (tid < ncta) {
                const int x = min(upto - part_c, T - origin), y = min(upto, T - origin);
                if (tid == cta) {
                    mine[0] = x;
                    mine[1] = y;
                }
                if (cta == ncta - 1) f.points[tid] = x;
                if (cta == ncta - 1 && tid == ncta - 1) f.points[ncta] = T - origin;
            }
            __syncthreads();
            before -= origin;
            x0 = mine[0];
            x1 = mine[1];
        }
    }
    const uint32_t tmem = *tmem_slot;

    // The next batch of this CTA's items, by one warp: 32 chunks at a time, a lane each.
    auto list_items = [&]() {
        const int x1 = mine[1];
        int c0 = mine[2], k0 = mine[3], U = mine[4], n = 0, more = 0;
        __syncwarp();
#pragma unroll 1
        while (c0 < n_chunks && U < x1) {
            const int c = c0 + lane;
            Chunk k = {};
            if (c < n_chunks) k = load_chunk(c, false);
            const int units = k.items * k.ku;
            int iu = units;
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, iu, o);
                if (lane >= o) iu += y;
            }
            const int start = U + iu - units, k_lo = lane == 0 ? k0 : 0, cnt = max(0, items_before(k, start, x1) - k_lo);
            int ic = cnt;
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(kFull, ic, o);
                if (lane >= o) ic += y;
            }
            const int pos = n + ic - cnt, fits = min(cnt, max(0, kBatch - pos)), total = __shfl_sync(kFull, ic, 31);
#pragma unroll 1
            for (int i = 0; i < fits; ++i) put_item(pos + i, k, start, k_lo + i, mine[0], x1, mine[12], false);
            if (n + total > kBatch) {  // the first lane whose items do not all fit is where the next batch starts
                const unsigned over = __ballot_sync(kFull, pos + cnt > kBatch);
                if (lane == __ffs(over) - 1) {
                    mine[2] = c;
                    mine[3] = k_lo + fits;
                    mine[4] = start;
                }
                n = kBatch;
                more = 1;
                break;
            }
            n += total;
            U += __shfl_sync(kFull, iu, 31);
            c0 += 32;
            k0 = 0;
        }
        if (lane == 0) {
            mine[5] = n;
            mine[6] = more;
        }
        __syncwarp();
    };
    // Every role runs its body once per batch of listed items.
    auto batches = [&](auto lister, auto&& body) {
        __syncthreads();  // the first batch is listed
#pragma unroll 1
        while (true) {
            const int more = mine[6];
            body(mine[5]);
            if (!more) break;
            __syncthreads();
            if constexpr (decltype(lister)::value) {
                if (warp == 9) list_items();
            }
            __syncthreads();
        }
    };

    // ---- what the joining needs to know of each sequence (from the last CTA down, the first have work in any case), or the
    // rows without keys: each chunk of them by all CTAs.  (One CTA per chunk took 170 us for 1249 tokens of 32 heads.)
    auto zero_rows = [&](int c, size_t first, size_t stride) {
        const Chunk k = load_chunk(c, false);
        uint4* o = reinterpret_cast<uint4*>(a.out) + static_cast<size_t>(k.q0) * a.Hq * 16;
#pragma unroll 1
        for (size_t i = first; i < static_cast<size_t>(k.tokens) * a.Hq * 16; i += stride) o[i] = make_uint4(0u, 0u, 0u, 0u);
    };
    const int n_empty = mine[11];
    if (f.prefix) {
#pragma unroll 1
        for (int s = ncta - 1 - cta; s < n_chunks; s += ncta) {
            const Chunk k = load_chunk(s, false);
            for (int i = tid; i < k.tokens; i += kNT)
                f.seq_plan[k.q0 + i] = make_int4(first_unit[s] + (i >> cta_shift) * a.Hkv * k.ku + item_units(k.w), k.ku, (i & (cta_q - 1)) << g_shift,
                                                  k.ku - item_units(k.w));
        }
    } else if (n_empty <= kEmpty) {
#pragma unroll 1
        for (int e = 0; e < n_empty; ++e) zero_rows(empty[e], static_cast<size_t>(cta) * kNT + tid, static_cast<size_t>(ncta) * kNT);
    } else {
#pragma unroll 1
        for (int s = cta; s < n_chunks; s += ncta)
            if (load_chunk(s, false).keys == 0) zero_rows(s, tid, kNT);
    }

    // the preparing kernel has completed; only then may the next one start, which uses what it cleared
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    bool ok = true;  // this role has seen no timeout
    auto give_up = [&]() {
        ok = false;
        *abort_flag = 1;
    };
    // Group t's key tiles of item i: every one of an item of two query tiles, else every second one (the owner, i & 1,
    // starts with the first).
    auto first_tile = [&](int t, int i, bool pair) { return pair ? 0 : (t ^ i) & 1; };
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PL::kRegsOther));
        if (warp == 8 || warp == 10) {
            // ------------------------------------------------ producers: K tiles (warp 8), V tiles (warp 10)
            const bool is_v = warp == 10;
            const CUtensorMap* map = is_v ? &vmap : &kmap;
            const int full = NARROW == 2 ? kFStg + 4 * is_v : is_v ? kFVFull : kFKFull;
            const int empty = NARROW == 2 ? kFStgFree + 4 * is_v : is_v ? kFVEmpty : kFKEmpty;
            constexpr uint32_t kBytes = NARROW == 0 ? 2 * kKvHalf : kStgSlot;
            const uint32_t dst0 =
                sb + (NARROW == 2 ? PL::kOffStg + is_v * PL::kSlots * kStgSlot : is_v ? PL::kOffV : PL::kOffK) + lane * a.S * 128;
            const int bpt = kKeys / a.S;  // blocks per key tile; it divides 32, so a tile's entries come from one batch of 32
            int g = 0;                    // key tiles copied
            batches(std::false_type{}, [&](int n) {
                if (n == 0) return;
                // table entries come 32 at a time, one per lane: the item's current and next 32, and the next item's first
                auto entry = [&](const Item& it, int idx) {
                    return idx < ceil_div(it.keys, a.S) ? __ldg(a.block_table + static_cast<size_t>(it.table) + idx) : -1;
                };
                auto first = [&](const Item& it) { return ((it.j0 * bpt) >> 5) * 32; };
                int e0 = entry(items[0], first(items[0]) + lane), e1 = entry(items[0], first(items[0]) + 32 + lane);
#pragma unroll 1
                for (int i = 0; i < n && ok; ++i) {
                    const Item it = items[i];
                    const int n_table = ceil_div(it.keys, a.S), h = it.head_pair & 0xffff;
                    int base = first(it), cur = e0, nxt = e1;
                    if (i + 1 < n) {
                        const Item nx = items[i + 1];
                        e0 = entry(nx, first(nx) + lane);
                        e1 = entry(nx, first(nx) + 32 + lane);
                    }
#pragma unroll 1
                    for (int j = it.j0; j < it.j0 + it.n; ++j, ++g) {
                        const int idx0 = j * bpt;
                        if (idx0 >= base + 32) {
                            base += 32;
                            cur = nxt;
                            nxt = entry(it, base + 32 + lane);
                        }
                        const int e = __shfl_sync(kFull, cur, (idx0 + lane) & 31);
                        int row = a.NB * a.S;  // beyond the pool: the copy fills zeros
                        if (lane < bpt && idx0 + lane < n_table) {
                            if (e >= 0 && e < a.NB) row = e * a.S;
                            else if (!is_v) raise_error(a.err, PKV_DEVERR_BAD_BLOCK);
                        }
                        const int st = g % kCopies;
                        if (g >= kCopies && !warp_wait(bar + 8 * (empty + st), (g / kCopies - 1) & 1, a.timeout_ns)) {
                            give_up();
                            break;
                        }
                        const uint32_t fb = bar + 8 * (full + st);
                        if (lane == 0) mbar_arrive_expect_tx(fb, kBytes);
                        if (lane < bpt) {
                            tma_load_3d_nohint(dst0 + st * kBytes, map, 0, h, row, fb);
                            if constexpr (NARROW == 0) tma_load_3d_nohint(dst0 + st * kBytes + kKvHalf, map, 64, h, row, fb);
                        }
                    }
                }
            });
            if (lane == 0)  // its own copies have landed before the CTA may finish (bounded)
#pragma unroll 1
                for (int t = max(0, g - kCopies); t < g; ++t)
                    mbar_wait_bounded(bar + 8 * (full + t % kCopies), (t / kCopies) & 1, a.timeout_ns);
        } else if (warp == 9 || warp == 13) {
            // ------------------------------------------------ scores of group t (A: warp 9, B: 13): S of its key tile c into
            // score buffer c & 1, which the P of tile c - 2 was read from.  Both groups' score warps see every K tile land,
            // in order, and free every stage, a tile that is the other group's at once (the P V warps do the same with V):
            // no barrier of the rings can be a phase further than a warp that waits for it thinks.
            const int t = warp == 13;
            const uint64_t q0 = smem_desc_sw128(sb, 16, 1024) + ((2 * t * kQHalf) >> 4);  // Q, K: K-major rows of 128 B
            const uint64_t k0 = smem_desc_sw128(sb, 16, 1024) + (PL::kOffK >> 4);
            const uint32_t tS = tmem + kColS + 128 * t;
            int g = 0, c = 0, q_n = 0;  // key tiles of the CTA, of this group; items of this group
            batches(std::true_type{}, [&](int n) {
#pragma unroll 1
                for (int i = 0; i < n && ok; ++i) {
                    const int end = g + items[i].n;
                    const bool pair = items[i].head_pair >> 16;
                    int x = g + first_tile(t, i, pair);  // this group's next tile
                    if (x < end) {
                        ok = warp_wait(bar + 8 * (kFQ + t), q_n & 1, a.timeout_ns);
                        ++q_n;
                    }
#pragma unroll 1
                    for (; g < end && ok; ++g) {
                        const int st = g % kStages, b = c & 1;
                        ok = warp_wait(bar + 8 * (kFKFull + st), (g / kStages) & 1, a.timeout_ns);
                        if (g != x) {
                            if (ok && lane == 0) mbar_arrive(bar + 8 * (kFKEmpty + st));
                            continue;
                        }
                        if (c >= 2) ok = ok && warp_wait(bar + 8 * (kFPV + 2 * t + b), ((c - 2) >> 1) & 1, a.timeout_ns);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t b0 = k0 + ((st * kStage) >> 4);
                        const uint32_t d = tS + 64 * b;
                        if constexpr (NARROW == 1) {
                            // E4M3: the query rows' hi codes in the slot's first 16 KB, their lo codes in the second
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                tc_mma_f8_warp(d, q0 + 2 * kk, b0 + 2 * kk, kIdescS8, kk > 0);
                                tc_mma_f8_warp(d, q0 + (kQHalf >> 4) + 2 * kk, b0 + 2 * kk, kIdescS8, 1u);
                            }
                        } else {
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                tc_mma_f16_warp(d, q0 + (((kk >> 2) * kQHalf + (kk & 3) * 32) >> 4),
                                                b0 + (((kk >> 2) * kKvHalf + (kk & 3) * 32) >> 4), kIdescS<NARROW>, kk > 0);
                        }
                        tc_commit_warp(bar + 8 * (kFS + 2 * t + b));
                        tc_commit_warp(bar + 8 * (kFKEmpty + st));
                        ++c;
                        x += pair ? 1 : 2;
                    }
                }
            });
        } else if (warp == 11 || warp == 15) {
            // ------------------------------------------------ O += P V of group t (A: warp 11, B: 15)
            const int t = warp == 15;
            const uint64_t v0 = smem_desc_sw128(sb, kKvHalf, 1024) + (PL::kOffV >> 4);  // V: N-major, halves kKvHalf apart
            const uint32_t tS = tmem + kColS + 128 * t, tO = tmem + kColO + 128 * t;
            int g = 0, c = 0, zeroed = 0;
            batches(std::false_type{}, [&](int n) {
#pragma unroll 1
                for (int i = 0; i < n && ok; ++i) {
                    const int end = g + items[i].n, last_keys = items[i].keys - (items[i].j0 + items[i].n - 1) * kKeys;
                    const bool pair = items[i].head_pair >> 16;
                    const int step = pair ? 1 : 2;
                    int x = g + first_tile(t, i, pair);
                    const int x0 = x;
#pragma unroll 1
                    for (; g < end && ok; ++g) {
                        const int st = g % kStages, b = c & 1;
                        ok = warp_wait(bar + 8 * (kFVFull + st), (g / kStages) & 1, a.timeout_ns);
                        if (g != x) {
                            if (ok && lane == 0) mbar_arrive(bar + 8 * (kFVEmpty + st));
                            continue;
                        }
                        if (NARROW != 2 && g == end - 1 && last_keys < kKeys) {
                            // V rows past the last key are not data, and 0 times what they hold may be NaN (an INT8 code is
                            // a number): the softmax group zeroes them, of an item of two query tiles group A
                            if (!pair || t == 0) {
                                if (ok && lane == 0) {
                                    mine[8 + t] = st;
                                    mbar_arrive(bar + 8 * (kFVThere + t));
                                }
                            } else {
                                ok = ok && warp_wait(bar + 8 * kFZero, zeroed & 1, a.timeout_ns);
                                ++zeroed;
                            }
                        }
                        ok = ok && warp_wait(bar + 8 * (kFP + 2 * t + b), (c >> 1) & 1, a.timeout_ns);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t b0 = v0 + ((st * kStage) >> 4);
                        const uint32_t p = tS + 64 * b;
                        const uint32_t acc0 = g > x0;
                        if constexpr (NARROW == 1) {
                            // E4M3: P's hi codes in 16 columns (four per column), its lo codes in the next 16
#pragma unroll
                            for (int kc = 0; kc < kKeys / 32; ++kc) {
                                tc_mma_f8_ts_warp(tO, p + 8 * kc, b0 + ((kc * 4096) >> 4), kIdescPV8, kc > 0 ? 1u : acc0);
                                tc_mma_f8_ts_warp(tO, p + 16 + 8 * kc, b0 + ((kc * 4096) >> 4), kIdescPV8, 1u);
                            }
                        } else {
#pragma unroll
                            for (int kk = 0; kk < kKeys / 16; ++kk)
                                tc_mma_f16_ts_warp(tO, p + 8 * kk, b0 + ((kk * 2048) >> 4), kIdescPV<NARROW>, kk > 0 ? 1u : acc0);
                        }
                        tc_commit_warp(bar + 8 * (kFPV + 2 * t + b));
                        if (x + step >= end) tc_commit_warp(bar + 8 * (kFO + t));
                        tc_commit_warp(bar + 8 * (kFVEmpty + st));
                        ++c;
                        x += step;
                    }
                }
            });
        } else if (NARROW == 2 && warp >= 16) {
            // ------------------------------------------------ INT8: rows 32 half + lane of every K (warps 16, 18) or V tile
            // (17, 19) from its staging slot into the f16 ring, exactly (the scales go to the scores and the output).  With
            // one warp per operand a key tile took 2300 cycles, whatever else was done with it.
            constexpr int kSlots = PL::kSlots ? PL::kSlots : 1;
            const bool is_v = warp & 1;
            const int r = lane + 32 * (warp >= 18), sw = r & 7;
            const int full = is_v ? kFVFull : kFKFull, empty = is_v ? kFVEmpty : kFKEmpty;
            int g = 0;
            batches(std::false_type{}, [&](int n) {
#pragma unroll 1
                for (int i = 0; i < n && ok; ++i) {
                    const int end = g + items[i].n;
#pragma unroll 1
                    for (; g < end && ok; ++g) {
                        const int slot = g % kSlots, st = g % kStages;
                        ok = warp_wait(bar + 8 * (kFStg + 4 * is_v + slot), (g / kSlots) & 1, a.timeout_ns) &&
                             (g < kStages || warp_wait(bar + 8 * (empty + st), (g / kStages - 1) & 1, a.timeout_ns));
                        if (!ok) break;
                        const uint8_t* src = smem + PL::kOffStg + (is_v * PL::kSlots + slot) * kStgSlot + r * 128;
                        uint8_t* dst = smem + (is_v ? PL::kOffV : PL::kOffK) + st * kStage + r * 128;
#pragma unroll 4
                        for (int k = 0; k < 8; ++k) {  // 16 codes: head dims 16 k .. 16 k + 15
                            const uint4 wv = *reinterpret_cast<const uint4*>(src + ((k ^ sw) * 16));
                            const uint32_t ws[4] = {wv.x, wv.y, wv.z, wv.w};
                            uint32_t o[8];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const uint32_t fl = ws[u] ^ 0x80808080u;
                                o[2 * u] = s8x2_to_f16x2(fl, 0);
                                o[2 * u + 1] = s8x2_to_f16x2(fl, 2);
                            }
                            uint8_t* dh = dst + (k >> 2) * kKvHalf;
                            const int lc = 2 * (k & 3);
                            *reinterpret_cast<uint4*>(dh + ((lc ^ sw) * 16)) = make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4*>(dh + (((lc + 1) ^ sw) * 16)) = make_uint4(o[4], o[5], o[6], o[7]);
                        }
                        fence_proxy_async_smem();  // the MMA (async proxy) reads what was written; the next copy overwrites
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(bar + 8 * (full + st));
                            mbar_arrive(bar + 8 * (kFStgFree + 4 * is_v + slot));
                        }
                    }
                }
            });
        } else {
            batches(std::false_type{}, [&](int) {});
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PL::kRegsSoftmax));
        // ------------------------------------------------ softmax groups: warps 0-3 A, 4-7 B; thread r owns query row r
        const int t = warp >> 2, r = tid & 127;
        const uint32_t trow = static_cast<uint32_t>((warp & 3) * 32) << 16;
        uint8_t* q_slot = smem + 2 * t * kQHalf;
        int c = 0, q_sent = 0;                // this group's key tiles; Q copies sent
        int o_mine = 0, o_other = 0;          // items of this group, of the other one
        int joins_mine = 0, joins_other = 0;  // items that this group joined, that the other one did
        int zeroed = 0;                       // key tiles whose V rows past the last key it zeroed
        bool lent = false;                    // the other group still has to read this group's O
        auto next_item = [&](int i, int n) {  // this group's first item from the i-th on
            while (i < n && first_tile(t, i, items[i].head_pair >> 16) >= items[i].n) ++i;
            return i;
        };
        auto copy_q = [&](const Item& it) {   // by the group's first thread
            const int row = it.q_row + ((it.head_pair >> 16) && t ? rows_q : 0);
            const uint32_t qb = bar + 8 * (kFQ + t);
            mbar_arrive_expect_tx(qb, 2 * kQHalf);
            for (int hf = 0; hf < 2; ++hf)
                tma_load_3d_nohint(smem_u32(q_slot) + hf * kQHalf, &qmap, hf * 64, (it.head_pair & 0xffff) * a.G, row, qb);
            ++q_sent;
        };
        batches(std::false_type{}, [&](int n) {
            int i = next_item(0, n), nxt = n;
            o_other += i;  // the items of the other group alone
            if (i < n && ok && r == 0) copy_q(items[i]);
            __syncwarp();
#pragma unroll 1
            for (; i < n && ok; o_other += nxt - i - 1, i = nxt) {
                const Item& it = items[i];
                nxt = next_item(i + 1, n);
                const bool pair = it.head_pair >> 16;
                const int tiles = it.n, owner = i & 1, step = pair ? 1 : 2, j_first = first_tile(t, i, pair);
                const bool split = !pair && tiles > 1;  // both groups, on the same rows
                const int row = (pair && t ? kRows : 0) + r;  // of the item's rows
                const bool valid = row < it.tokens * a.G;
                const bool live = (row & ~31) < it.tokens * a.G;  // some row of this warp is the item's
                const int h = it.head_pair & 0xffff;
                const size_t tok_row = (static_cast<size_t>(it.q_row) + (row >> g_shift)) * a.Hq + (static_cast<size_t>(h) << g_shift) +
                                       (row & (a.G - 1));
                float m_ref = kLowest, l_run = 0.f;
                // what the scores are multiplied by (log2 units)
                float sm_log2 = a.k_head ? a.sm_base * __ldg(a.k_head + h) : a.sm_log2;
                if (NARROW != 0 && valid) {
                    const float s = f.q_scale[tok_row];  // negative: values that the operands cannot carry
                    // (not of a sequence of length 0 in a group with a prefix, whose q nobody need have written)
                    if (s < 0.f && (!f.prefix || f.lens[it.q_row + (row >> g_shift)] > 0)) raise_error(a.err, PKV_DEVERR_Q_RANGE);
                    sm_log2 *= fabsf(s);
                }
                // (a factor below what fp32 holds, of a row of zeros under a small key scale say: as good as none, but the
                // keys past the last are -inf, and -inf times zero is no number)
                if (sm_log2 == 0.f) sm_log2 = 1.17549435e-38f;
                int left = it.keys - (it.j0 + j_first) * kKeys;  // keys from the current tile on
#pragma unroll 1
                for (int j = j_first; j < tiles; j += step, left -= step * kKeys, ++c) {
                    const int b = c & 1;
                    const uint32_t tS = tmem + kColS + 128 * t + 64 * b + trow;
                    if (!warp_wait(bar + 8 * (kFS + 2 * t + b), (c >> 1) & 1, a.timeout_ns)) {
                        give_up();
                        break;
                    }
                    tc_fence_after();
                    if (j + step >= tiles && nxt < n && r == 0) copy_q(items[nxt]);  // nothing reads this item's Q any more
                    __syncwarp();  // TMEM is read by whole warps
                    if (live) {
                        float v[64];
                        tmem_ld64(tS, v);
                        if (left < kKeys) {  // keys past the last: their probabilities come out as 0
#pragma unroll
                            for (int u = 0; u < 64; ++u) v[u] = u < left ? v[u] : -INFINITY;
                        }
                        float mx[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u) mx[u] = fmaxf(v[2 * u], v[2 * u + 1]);
#pragma unroll
                        for (int u = 16; u < 64; u += 2) mx[(u >> 1) & 7] = fmax3(mx[(u >> 1) & 7], v[u], v[u + 1]);
                        const float mt = fmaxf(fmax3(mx[0], mx[1], mx[2]), fmax3(fmax3(mx[3], mx[4], mx[5]), mx[6], mx[7])) *
                                         sm_log2;
                        const bool need = mt > m_ref + 8.f;
                        // O is rescaled (below) only when some row of the warp needs it; rows that do not keep alpha = 1
                        const bool rescale = j > j_first && __any_sync(kFull, need);
                        const float m_new = need ? (NARROW == 1 ? mt - kP8Shift : mt) : m_ref;
                        const float alpha = ex2_approx(m_ref - m_new);
                        m_ref = m_new;
                        const float2 sc2 = make_float2(sm_log2, sm_log2), nm2 = make_float2(-m_ref, -m_ref);
                        float2 ls2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                        uint32_t pk[32];  // bf16 / f16 pairs; FP8: 16 words of four hi codes, then 16 of four lo codes
#pragma unroll
                        for (int u = 0; u < 64; u += 2) {
                            const float2 x = __ffma2_rn(make_float2(v[u], v[u + 1]), sc2, nm2);
                            const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
                            ls2[(u >> 1) & 1] = __fadd2_rn(ls2[(u >> 1) & 1], make_float2(p0, p1));
                            if constexpr (NARROW != 0) pk[u / 2] = f16x2_rn(p0, p1);
                            else pk[u / 2] = bf16x2_rn(p0, p1);
                        }
                        if constexpr (NARROW == 1) {
                            // the f16 probabilities (at most 2^8) split into two E4M3 parts for the 8-bit P V MMAs
                            uint32_t hl[32];
#pragma unroll
                            for (int k = 0; k < 16; ++k) split_e4m3x4(pk[2 * k], pk[2 * k + 1], hl[k], hl[16 + k]);
#pragma unroll
                            for (int k = 0; k < 32; ++k) pk[k] = hl[k];
                        }
                        const float2 lsum = __fadd2_rn(ls2[0], ls2[1]);
                        l_run = l_run * alpha + (lsum.x + lsum.y);
                        tmem_st32u(tS, pk);  // P over the scores just read (this thread's lane only)
                        if (rescale) {
                            // O may be touched only once the previous P V of this group has completed
                            if (!warp_wait(bar + 8 * (kFPV + 2 * t + ((c - 1) & 1)), ((c - 1) >> 1) & 1, a.timeout_ns)) {
                                give_up();
                                break;
                            }
                            tc_fence_after();
                            const uint32_t tO = tmem + kColO + 128 * t + trow;
#pragma unroll 1
                            for (int k = 0; k < 128; k += 32) {
                                float o[32];
                                tmem_ld32(tO + k, o);
#pragma unroll
                                for (int u = 0; u < 32; ++u) o[u] *= alpha;
                                tmem_st32(tO + k, o);
                            }
                        }
                    }
                    // V rows past the last key: zero, once they have landed
                    if (NARROW != 2 && left < kKeys && (t == 0 || !pair)) {
                        if (!warp_wait(bar + 8 * (kFVThere + t), zeroed++ & 1, a.timeout_ns)) {
                            give_up();
                            break;
                        }
                        const int st = mine[8 + t];
                        constexpr int kRowChunks = NARROW == 1 ? 8 : 16;  // 16-byte pieces of a key's row
#pragma unroll 1
                        for (int u = r; u < (kKeys - left) * kRowChunks; u += 128) {
                            const int key = left + u / kRowChunks, k = u % kRowChunks;
                            *reinterpret_cast<uint4*>(smem + PL::kOffV + st * kStage + (k >> 3) * kKvHalf + key * 128 +
                                                      (k & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        if (pair) mbar_arrive(bar + 8 * kFZero);
                    }
                    if (lent) {  // the P V that this P leads to overwrites O: the other group has read it
                        lent = false;
                        if (!warp_wait(bar + 8 * (kFTaken + (t ^ 1)), (joins_other - 1) & 1, a.timeout_ns)) {
                            give_up();
                            break;
                        }
                        tc_fence_after();
                    }
                    tc_fence_before();
                    mbar_arrive(bar + 8 * (kFP + 2 * t + b));
                }
                ++o_mine;
                if (pair || split) ++o_other;
                if (split && t == owner) ++joins_mine;
                if (split && t != owner) ++joins_other;
                if (!ok) break;
                if (split && t != owner) {  // the owner joins: it reads this group's O where it is
                    ml_out[owner * 128 + r] = make_float2(m_ref, l_run);
                    mbar_arrive(bar + 8 * (kFMl + owner));
                    lent = true;
                    continue;
                }
                // ---- the item's last product: out = O / l, or a record of (O, m, l)
                // (the other group's (m, l) first: past them, its last O but one is complete, so that the wait for its last
                // one is not for a phase too far)
                if (!warp_wait(bar + 8 * (kFO + t), (o_mine - 1) & 1, a.timeout_ns) ||
                    (split && (!warp_wait(bar + 8 * (kFMl + t), (joins_mine - 1) & 1, a.timeout_ns) ||
                               !warp_wait(bar + 8 * (kFO + (t ^ 1)), (o_other - 1) & 1, a.timeout_ns)))) {
                    give_up();
                    break;
                }
                tc_fence_after();
                float w_mine = 1.f, w_other = 0.f;
                if (split) {
                    const float2 ml = ml_out[t * 128 + r];
                    const float m = fmaxf(m_ref, ml.x);
                    w_mine = ex2_approx(m_ref - m);
                    w_other = ex2_approx(ml.x - m);
                    m_ref = m;
                    l_run = l_run * w_mine + ml.y * w_other;
                }
                const size_t rec_row = it.rec == 2 ? static_cast<size_t>(f.extra_row) + static_cast<size_t>(cta) * 256 + row : tok_row;
                const bool rec = it.rec != 0;
                const float inv = rec ? 1.f : l_run > 0.f ? (a.v_head ? __ldg(a.v_head + h) : a.out_mul) / l_run : 0.f;
                const uint32_t tO = tmem + kColO + 128 * t + trow, tO2 = tmem + kColO + 128 * (t ^ 1) + trow;
                w_mine *= inv;
                w_other *= inv;
                if (live) {
                    float* rec_o = f.rec_o + rec_row * 128;
                    uint4* out_o = reinterpret_cast<uint4*>(a.out) + tok_row * 16;
#pragma unroll 1
                    for (int k = 0; k < 128; k += 32) {
                        float o[32];
                        tmem_ld32(tO + k, o);
#pragma unroll
                        for (int u = 0; u < 32; ++u) o[u] *= w_mine;
                        if (split) {
                            float o2[32];
                            tmem_ld32(tO2 + k, o2);
#pragma unroll
                            for (int u = 0; u < 32; ++u) o[u] = fmaf(o2[u], w_other, o[u]);
                        }
                        if (valid && rec) {
#pragma unroll
                            for (int u = 0; u < 4; ++u) store_v8(rec_o + k + 8 * u, o + 8 * u);
                        } else if (valid) {
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                out_o[k / 8 + u] = make_uint4(bf16x2_rn(o[8 * u], o[8 * u + 1]), bf16x2_rn(o[8 * u + 2], o[8 * u + 3]),
                                                              bf16x2_rn(o[8 * u + 4], o[8 * u + 5]),
                                                              bf16x2_rn(o[8 * u + 6], o[8 * u + 7]));
                        }
                        __syncwarp();  // TMEM is read by whole warps: the rows that are none wait for the others
                    }
                    if (rec && valid) f.rec_ml[rec_row] = make_float2(m_ref, l_run);
                }
                tc_fence_before();  // the next item's first P V overwrites O, once this group's P of it is there
                if (split) mbar_arrive(bar + 8 * (kFTaken + t));
            }
        });
        // a Q copy that nobody waited for (after a timeout) lands before the CTA finishes
        if (r == 0 && !ok && q_sent > 0) mbar_wait_bounded(bar + 8 * (kFQ + t), (q_sent - 1) & 1, a.timeout_ns);
    }
    if (!ok && lane == 0) *abort_flag = 1;
    // ---- drain: nothing of this CTA may still be in flight when TMEM is freed and the CTA exits
    __syncthreads();
    if (warp >= 8 && warp < 16 && (warp & 1) && *abort_flag) {
        tc_commit_warp(bar + 8 * kFDrain);  // arrives once every MMA this warp issued has completed
        mbar_wait_bounded(bar + 8 * kFDrain, 0, a.timeout_ns);
    }
    if (*abort_flag && tid == 0) raise_error(a.err, PKV_DEVERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 11) tmem_dealloc(tmem, kTmemCols);
}

namespace {

// A row's pieces so far, four head dims per lane
struct Joined {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void add(const FullArgs& f, size_t row, int lane) {
        const float2 ml = f.rec_ml[row];
        const float4 x = reinterpret_cast<const float4*>(f.rec_o + row * 128)[lane];
        const float mn = fmaxf(m, ml.x);
        const float w0 = m == -INFINITY ? 0.f : ex2_approx(m - mn), w1 = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - mn);
        m = mn;
        l = l * w0 + ml.y * w1;
        o = make_float4(o.x * w0 + x.x * w1, o.y * w0 + x.y * w1, o.z * w0 + x.z * w1, o.w * w0 + x.w * w1);
    }
    __device__ __forceinline__ void store(const PrefillArgs& a, size_t row, int h, int lane) const {
        const float inv = l > 0.f ? (a.v_head ? __ldg(a.v_head + h) : a.out_mul) / l : 0.f;
        reinterpret_cast<uint2*>(a.out)[row * 32 + lane] =
            make_uint2(bf16x2_rn(o.x * inv, o.y * inv), bf16x2_rn(o.z * inv, o.w * inv));
    }
};

}  // namespace

// Block (c, part) takes rows [8 part, 8 part + 8) of the item whose second piece starts CTA c's share; one warp per row.
// (With 32 rows per block, four per warp in turn, 24 x 5 tokens over 1150 FP8 states took 38 us instead of 34.7.)
__global__ void __launch_bounds__(256) join_cuts_kernel(const PrefillArgs a, const FullArgs f) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x, ncta = gridDim.x, lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int4 cut = f.cuts[c];
    const int share = *f.share;  // 0: the parts' starts are listed
    const int U0 = cut.z, U1 = cut.w, h = cut.y >> 16;
    if (U1 == 0 || r >= (cut.y & 0xffff) * a.G) return;
    auto start = [&](int k) { return share ? k * share : f.points[k]; };
    // the item's first extra piece does it: the cut before it, if any, falls before the item or in its first units
    int prev = c - 1;
    while (prev > 0 && start(prev) == start(c)) --prev;  // (a part may be empty)
    if (prev >= 0 && start(prev) > U0) return;
    const size_t row = (static_cast<size_t>(cut.x) + r / a.G) * a.Hq + static_cast<size_t>(h) * a.G + r % a.G;
    const size_t extra = static_cast<size_t>(f.extra_row) + r;
    Joined j;
    j.add(f, row, lane);
#pragma unroll 2
    for (int k = c; k < ncta && start(k) < U1; ++k)
        if (share || f.points[k] < f.points[k + 1]) j.add(f, extra + static_cast<size_t>(k) * 256, lane);
    j.store(a, row, h, lane);
}

// Shared prefixes: one warp per (sequence, query head).
__global__ void __launch_bounds__(256) join_rows_kernel(const PrefillArgs a, const FullArgs f) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const size_t row = static_cast<size_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= static_cast<size_t>(f.num_seqs) * a.Hq) return;
    const int s = static_cast<int>(row / a.Hq), hq = static_cast<int>(row % a.Hq), h = hq / a.G, blocks = f.prefix_blocks[s];
    const int4 sp = f.seq_plan[s];
    const int share = *f.share;
    if (blocks <= 0) return;  // the row is written
    const int U0 = sp.x + h * sp.y, c0 = U0 / share, c1 = (U0 + sp.w - 1) / share;
    const size_t extra = static_cast<size_t>(f.extra_row) + sp.z + hq % a.G;
    Joined j;
    j.add(f, row, lane);
    if (f.lens[s] > blocks * a.S) j.add(f, static_cast<size_t>(f.own_row) + row, lane);
#pragma unroll 4
    for (int k = c0 + 1; k <= c1; ++k) j.add(f, extra + static_cast<size_t>(k) * 256, lane);
    j.store(a, row, h, lane);
}

// What precedes the stream: the decode's counters cleared (shared prefixes), and for one-byte caches the queries turned
// into the MMAs' operands, once for all of the items that use them: 256 bytes a row, and what the row's scores are
// multiplied by -- negative if a value cannot be carried.  One warp per row (token, query head), four head dims per lane.
//   FP8: the row is scaled by 2^e, e chosen so that its largest magnitude lies in [128, 256), and split into hi = E4M3(x)
//   and lo = E4M3(x - hi), 128 bytes each; hi + lo is the scaled value exactly for elements within 2^-10 of the row's
//   largest.  INT8: f16, exactly for |q| in [2^-14, 65504].
template <int NARROW>
__global__ void __launch_bounds__(256) full_prepare_kernel(const uint2* __restrict__ q, uint8_t* __restrict__ ops,
                                                           float* __restrict__ scale, int64_t rows, int* __restrict__ counters,
                                                           int64_t n_counters) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256, first = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    for (int64_t i = first; i < n_counters; i += stride) counters[i] = 0;
    if constexpr (NARROW != 0) {
        for (int64_t row = first >> 5; row < rows; row += stride >> 5) {
            const uint2 w = q[row * 32 + lane];
            const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
            uint8_t* out = ops + row * 256;
            if constexpr (NARROW == 1) {
                uint32_t m = max(max((w.x << 17) >> 1, (w.x & 0x7fff0000u)), max((w.y << 17) >> 1, (w.y & 0x7fff0000u)));
                m = __reduce_max_sync(kFull, m);  // |value| bits: ordered like the values
                const int e = min(126, max(-126, 7 - (static_cast<int>(m >> 23) - 127)));
                const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
                const float v0 = a.x * up, v1 = a.y * up, v2 = b.x * up, v3 = b.y * up;
                const uint32_t h01 = f32x2_to_e4m3x2(v0, v1), h23 = f32x2_to_e4m3x2(v2, v3);
                const float2 b01 = f16x2_to_float2(e4m3x2_to_f16x2_u(h01)), b23 = f16x2_to_float2(e4m3x2_to_f16x2_u(h23));
                reinterpret_cast<uint32_t*>(out)[lane] = h01 | (h23 << 16);
                reinterpret_cast<uint32_t*>(out)[32 + lane] =
                    f32x2_to_e4m3x2(v0 - b01.x, v1 - b01.y) | (f32x2_to_e4m3x2(v2 - b23.x, v3 - b23.y) << 16);
                const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                if (lane == 0) scale[row] = m >= 0x7f800000u ? -down : down;  // inf or NaN
            } else {
                const bool fits = fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))) < 65520.f;
                const bool number = a.x == a.x && a.y == a.y && b.x == b.x && b.y == b.y;
                reinterpret_cast<uint2*>(out)[lane] = make_uint2(f16x2_rn(a.x, a.y), f16x2_rn(b.x, b.y));
                const bool good = __all_sync(kFull, fits && number);
                if (lane == 0) scale[row] = good ? 1.f : -1.f;
            }
        }
    }
}

template <int NARROW>
static size_t full_smem() {
    return static_cast<size_t>(FullPlan<NARROW>::kOffMeta) + kFEnd + 1024;
}

size_t paged_full_smem_bytes(int narrow) { return narrow == 2 ? full_smem<2>() : narrow == 1 ? full_smem<1>() : full_smem<0>(); }

cudaError_t launch_full_prepare(const void* q, void* ops, float* scale, int64_t rows, int* counters, int64_t n_counters,
                                int narrow, int sms, cudaStream_t stream) {
    const int64_t work = std::max<int64_t>(narrow ? rows * 32 : 0, n_counters);
    const int grid = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(sms) * 8, (work + 255) / 256));
    const uint2* src = static_cast<const uint2*>(q);
    uint8_t* dst = static_cast<uint8_t*>(ops);
    if (narrow == 1) full_prepare_kernel<1><<<grid, 256, 0, stream>>>(src, dst, scale, rows, counters, n_counters);
    else if (narrow == 2) full_prepare_kernel<2><<<grid, 256, 0, stream>>>(src, dst, scale, rows, counters, n_counters);
    else full_prepare_kernel<0><<<grid, 256, 0, stream>>>(src, dst, scale, rows, counters, n_counters);
    return cudaGetLastError();
}

template <int NARROW>
static cudaError_t launch_full(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                               const PrefillArgs& a, const FullArgs& f, int grid, bool prepared, cudaStream_t stream) {
    const size_t smem = full_smem<NARROW>();
    auto kern = paged_full_kernel<NARROW>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(FullPlan<NARROW>::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = prepared ? 1 : 0;  // beside the preparing kernel; not beside what the caller's stream had before
    return cudaLaunchKernelEx(&cfg, kern, qmap, kmap, vmap, a, f);
}

cudaError_t launch_paged_full(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                              const PrefillArgs& a, const FullArgs& f, int narrow, int grid, bool prepared,
                              cudaStream_t stream) {
    switch (narrow) {
        case 0: return launch_full<0>(qmap, kmap, vmap, a, f, grid, prepared, stream);
        case 1: return launch_full<1>(qmap, kmap, vmap, a, f, grid, prepared, stream);
        case 2: return launch_full<2>(qmap, kmap, vmap, a, f, grid, prepared, stream);
        default: return cudaErrorInvalidValue;
    }
}

// Launched beside the kernel before it: its blocks wait for it where they start.
template <class Kernel>
static cudaError_t launch_beside(Kernel kern, dim3 grid, const PrefillArgs& a, const FullArgs& f, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, f);
}

cudaError_t launch_join_cuts(const PrefillArgs& a, const FullArgs& f, int grid, cudaStream_t stream) {
    return launch_beside(join_cuts_kernel, dim3(grid, 32), a, f, stream);
}

cudaError_t launch_join_rows(const PrefillArgs& a, const FullArgs& f, cudaStream_t stream) {
    const size_t rows = static_cast<size_t>(f.num_seqs) * a.Hq;
    return launch_beside(join_rows_kernel, dim3(static_cast<unsigned>((rows + 7) / 8)), a, f, stream);
}

}  // namespace pkv
