// full_tile.cu -- attention of many query rows over a paged K/V range without a mask: cross attention to an encoder's
// states (pkv_paged_cross_attention) and the shared prefixes of a decode batch (pkv_paged_attention_decode_prefix).
//
// A chunk is a run of query tokens that attend to the same keys: a sequence's tokens and its encoder states, or a group
// of sequences (one token each) and their common prefix.  For KV head h its rows are (token, query head of h's group),
// stacked in query tiles of 128; an item is one or two query tiles of one KV head against all of the chunk's keys, which
// it reads once: S = Q K^T, P = 2^(S - m) with the running maximum m, O += P V per tile of 64 keys.
//
// Work split: the items' key tiles are laid end to end and cut into equal shares, one per CTA (SM).  An item that is cut
// leaves a partial (O, m, l) record for each of its pieces; they join as
//   M = max m_i,  l = sum 2^(m_i - M) l_i,  O = sum 2^(m_i - M) O_i / l
// in full_combine_kernel (cross attention) or at the end of the suffix decode (decode_mma.cuh).
//
// A CTA runs its share as one stream: TMEM, barriers and the K/V rings live through all of its items, and the copies of
// the next item's keys run while the current one ends.  Two softmax groups (A, B: one thread per query row, 128 rows, a
// Q slot, two score buffers and an output accumulator in TMEM each) work side by side: on an item's two query tiles, or,
// where items have one tile, on items in turn, so that one item's first products run while the last one is written out.
//   * warps 0-3 and 4-7: the softmax groups.  A group's first thread also copies its next item's Q, once the scores of
//     the current item's last key tile are there (nothing reads the old Q any more);
//   * warps 8 and 10 copy the K and V tiles (TMA, one block of the block table per copy, one lane per block);
//   * warps 9 and 11 issue the MMAs (tcgen05): scores and P V;
//   * INT8 caches: warps 12-15 widen the codes to f16, two warps per operand, half of the rows each.
// Hand-offs are mbarriers; every wait is bounded.  On a timeout a role records the error and does nothing more, the CTA
// drains its own MMAs and copies (bounded) and frees TMEM.
#include "full_tile.cuh"
#include "prefill_tile.cuh"

namespace pkv {

namespace {

// Fewest key tiles in a share: a piece costs a record and its joining whatever its length.
constexpr int kMinShare = 2;
constexpr int kBatch = 64;  // items that a CTA lists at a time

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
    static constexpr int kThreads = NARROW == 2 ? 512 : 384;
    // registers per thread after the split (the launch gives 128 of 512 threads or 168 of 384)
    static constexpr int kRegsSoftmax = NARROW == 2 ? 184 : 208, kRegsOther = NARROW == 2 ? 72 : 88;
};

// mbarriers
constexpr int kFKFull = 0, kFKEmpty = 8, kFVFull = 16, kFVEmpty = 24;  // + stage
constexpr int kFS = 32, kFP = 36, kFPV = 40;        // + 2 * group + buffer: scores written, P written, P V done
constexpr int kFQ = 44, kFQConv = 46, kFO = 48;     // + group: Q landed, Q converted, O complete
constexpr int kFDrain = 50;
constexpr int kFStg = 51, kFStgFree = 59;           // + 4 * (V ? 1 : 0) + slot
constexpr int kFBars = 67;
constexpr int kFTmem = 8 * kFBars, kFAbort = kFTmem + 4, kFPart = kFAbort + 4;  // byte offsets
constexpr int kFMine = kFPart + 64;                 // this CTA's x0, x1, first item, items
constexpr int kFItems = 704;
constexpr int kFPre = kFItems + 32 * kBatch;        // key tiles and items before each chunk, [kMaxSeqs + 1] each
constexpr int kFEnd = kFPre + 8 * (kMaxSeqs + 1);
static_assert(kFMine + 16 <= kFItems, "meta slots overlap");

// One CTA's part of an item
struct Item {
    int q_row, tokens;  // the item's first row of q, its query tokens
    int keys, table;    // keys of the chunk, its block table row
    int j0, n;          // first key tile, key tiles
    int head_groups;    // KV head, softmax groups (bit mask) << 16
    int rec;            // 0: the result goes to out; 1: a record at the rows of (token, query head); 2: at the CTA's own rows
};
static_assert(sizeof(Item) == 32, "item size");

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ void store_v8(float* p, const float* v) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
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
    Item* items = reinterpret_cast<Item*>(meta + kFItems);
    int* pre_w = reinterpret_cast<int*>(meta + kFPre);  // key tiles before chunk s
    int* pre_i = pre_w + kMaxSeqs + 1;                  // items before chunk s
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x, ncta = gridDim.x;
    const int rows_q = kRows / a.G, cta_q = 2 * rows_q;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (tid == 0) {
        for (int i = 0; i < kFBars; ++i) {
            int count = 1;
            if (i >= kFP && i < kFP + 4) count = 128;
            if (i >= kFQConv && i < kFQConv + 2) count = 4;
            if (i == kFDrain) count = 2;
            if (NARROW == 2 && (i < kFKEmpty || (i >= kFVFull && i < kFVEmpty) || i >= kFStgFree)) count = 2;
            mbar_init(bar + 8 * i, count);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }

    // ---- the plan.  Chunk s: query tokens [q0, q1), keys; nothing to do for a malformed chunk.
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
    {
        // key tiles and items per chunk, then their exclusive prefix: each thread takes a contiguous run of chunks
        const int per = ceil_div(a.nseq, kNT);
        const int c_lo = min(tid * per, a.nseq), c_hi = min(c_lo + per, a.nseq);
        int sw = 0, si = 0;
        for (int c = c_lo; c < c_hi; ++c) {
            int q0, q1, kv;
            chunk(c, q0, q1, kv, cta == 0);
            const int n = kv > 0 ? ceil_div(q1 - q0, cta_q) * a.Hkv : 0, w = n * ceil_div(max(kv, 0), kKeys);
            pre_w[c + 1] = w;
            pre_i[c + 1] = n;
            sw += w;
            si += n;
        }
        int iw = sw, ii = si;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int yw = __shfl_up_sync(kFull, iw, o), yi = __shfl_up_sync(kFull, ii, o);
            if (lane >= o) {
                iw += yw;
                ii += yi;
            }
        }
        __shared__ int part_i[16];
        if (lane == 31) {
            part[warp] = iw;
            part_i[warp] = ii;
        }
        __syncthreads();
        int rw = iw - sw, ri = ii - si;
        for (int w = 0; w < warp; ++w) {
            rw += part[w];
            ri += part_i[w];
        }
        for (int c = c_lo; c < c_hi; ++c) {
            pre_w[c + 1] = rw += pre_w[c + 1];
            pre_i[c + 1] = ri += pre_i[c + 1];
        }
        if (tid == 0) pre_w[0] = pre_i[0] = 0;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    // what the roles need of the plan stays in shared memory: their registers are for the tiles
    volatile int* mine = reinterpret_cast<volatile int*>(meta + kFMine);
    const uint32_t tmem = *tmem_slot;
    const int T = pre_w[a.nseq];
    const int share = max(kMinShare, ceil_div(T, ncta));
    auto find = [&](const int* p, int x) {  // the chunk that holds x
        int lo = 0, hi = a.nseq - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p[mid] <= x) lo = mid; else hi = mid - 1;
        }
        return lo;
    };
    if (tid == 0) {
        const int x0 = static_cast<int>(min(static_cast<int64_t>(cta) * share, static_cast<int64_t>(T)));
        const int x1 = static_cast<int>(min(static_cast<int64_t>(x0) + share, static_cast<int64_t>(T)));
        auto item_at = [&](int x) {
            const int c = find(pre_w, x);
            return pre_i[c] + (x - pre_w[c]) / ceil_div(a.kv_lens[c], kKeys);
        };
        mine[0] = x0;
        mine[1] = x1;
        mine[2] = x0 < x1 ? item_at(x0) : 0;  // this CTA's items, the first and the last perhaps in part
        mine[3] = x0 < x1 ? item_at(x1 - 1) - mine[2] + 1 : 0;
        if (x0 >= x1) f.cuts[cta] = make_int4(0, 0, 0, 0);
    }
    __syncthreads();
    auto list_item = [&](int i, int index) {
        const int c = find(pre_i, index);
        int q0, q1, kv;
        chunk(c, q0, q1, kv, false);
        const int kt = ceil_div(kv, kKeys), k = index - pre_i[c], h = k % a.Hkv, t0 = (k / a.Hkv) * cta_q;
        const int U0 = pre_w[c] + k * kt, U1 = U0 + kt, xs = max(U0, mine[0]), xe = min(U1, mine[1]);
        Item it;
        it.q_row = q0 + t0;
        it.tokens = min(cta_q, q1 - q0 - t0);
        it.keys = kv;
        it.table = f.prefix ? q0 : c;
        it.j0 = xs - U0;
        it.n = xe - xs;
        it.head_groups = h | ((it.tokens > rows_q ? 3 : 1 << (i & 1)) << 16);
        it.rec = !(f.prefix || it.n < kt) ? 0 : xs == U0 ? 1 : 2;
        items[i] = it;
        if (index == mine[2])
            f.cuts[cta] = xs == U0 ? make_int4(0, 0, 0, 0) : make_int4(it.q_row, it.tokens | (h << 16), U0, U1);
    };
    // Every role runs its body once per batch of listed items.
    auto batches = [&](auto&& body) {
        for (int base = 0; base < mine[3]; base += kBatch) {
            const int n = min(kBatch, mine[3] - base);
            __syncthreads();
            if (tid < n) list_item(tid, mine[2] + base + tid);
            __syncthreads();
            body(n);
        }
    };

    // ---- what the joining of the pieces needs to know, and the rows without keys
    if (cta == ncta - 1 && tid == 0) *f.share = share;
    if (f.prefix) {
        for (int g = ncta - 1 - cta; g < a.nseq; g += ncta) {  // from the last CTA down: the first have work in any case
            int q0, q1, kv;
            chunk(g, q0, q1, kv, false);
            const int kt = kv > 0 ? ceil_div(kv, kKeys) : 0;
            for (int i = tid; i < q1 - q0; i += kNT)
                f.seq_plan[q0 + i] = make_int4(pre_w[g] + (i / cta_q) * a.Hkv * kt, kt, (i % cta_q) * a.G, 0);
        }
    } else {
        for (int s = ncta - 1 - cta; s < a.nseq; s += ncta) {
            if (a.kv_lens[s] != 0) continue;
            int q0, q1, kv;
            chunk(s, q0, q1, kv, false);
            uint4* o = reinterpret_cast<uint4*>(a.out) + static_cast<size_t>(q0) * a.Hq * 16;
            for (size_t i = tid; i < static_cast<size_t>(q1 - q0) * a.Hq * 16; i += kNT) o[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    }

    bool ok = true;  // this role has seen no timeout
    auto give_up = [&]() {
        ok = false;
        *abort_flag = 1;
    };
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PL::kRegsOther));
        if (warp == 8 || warp == 10) {
            // ------------------------------------------------ producers: K tiles (warp 8), V tiles (warp 10)
            const bool is_v = warp == 10;
            const CUtensorMap* map = is_v ? &vmap : &kmap;
            if (lane == 0) prefetch_tensormap(map);
            const int full = NARROW == 2 ? kFStg + 4 * is_v : is_v ? kFVFull : kFKFull;
            const int empty = NARROW == 2 ? kFStgFree + 4 * is_v : is_v ? kFVEmpty : kFKEmpty;
            constexpr uint32_t kBytes = NARROW == 0 ? 2 * kKvHalf : kStgSlot;
            const uint32_t dst0 = sb + (NARROW == 2 ? PL::kOffStg + is_v * PL::kSlots * kStgSlot : is_v ? PL::kOffV : PL::kOffK);
            const int bpt = kKeys / a.S;  // blocks per key tile; it divides 32, so a tile's entries come from one batch of 32
            int g = 0;                    // key tiles copied
            batches([&](int n) {
                // table entries come 32 at a time, one per lane: the item's current and next 32, and the next item's first
                auto entry = [&](const Item& it, int idx) {
                    return idx < ceil_div(it.keys, a.S) ? __ldg(a.block_table + static_cast<size_t>(it.table) * a.MB + idx) : -1;
                };
                auto first = [&](const Item& it) { return ((it.j0 * bpt) >> 5) * 32; };
                int e0 = entry(items[0], first(items[0]) + lane), e1 = entry(items[0], first(items[0]) + 32 + lane);
                for (int i = 0; i < n && ok; ++i) {
                    const Item it = items[i];
                    const int n_table = ceil_div(it.keys, a.S), h = it.head_groups & 0xffff;
                    int base = first(it), cur = e0, nxt = e1;
                    if (i + 1 < n) {
                        const Item nx = items[i + 1];
                        e0 = entry(nx, first(nx) + lane);
                        e1 = entry(nx, first(nx) + 32 + lane);
                    }
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
                        if ((g >= kCopies && !__all_sync(kFull, mbar_spin_bounded(bar + 8 * (empty + st), (g / kCopies - 1) & 1,
                                                                                a.timeout_ns))) ||
                            __any_sync(kFull, *abort_flag != 0)) {
                            give_up();
                            break;
                        }
                        const uint32_t fb = bar + 8 * (full + st);
                        if (lane == 0) mbar_arrive_expect_tx(fb, kBytes);
                        __syncwarp();
                        if (lane < bpt) {
                            const uint32_t dst = dst0 + st * kBytes + lane * a.S * 128;
                            tma_load_3d_nohint(dst, map, 0, h, row, fb);
                            if constexpr (NARROW == 0) tma_load_3d_nohint(dst + kKvHalf, map, 64, h, row, fb);
                        }
                    }
                }
            });
            if (lane == 0)  // its own copies have landed before the CTA may finish (bounded)
                for (int t = max(0, g - kCopies); t < g; ++t)
                    mbar_wait_bounded(bar + 8 * (full + t % kCopies), (t / kCopies) & 1, a.timeout_ns);
        } else if (warp == 9) {
            // ------------------------------------------------ scores: S of group t's key tile c into buffer c & 1, which the
            // P of tile c - 2 was read from
            const uint64_t d_kmaj = smem_desc_sw128(sb, 16, 1024);  // Q and K: K-major rows of 128 B
            int g = 0, c0 = 0, c1 = 0, q0 = 0, q1 = 0;  // key tiles of the CTA, of each group; items of each group
            batches([&](int n) {
                for (int i = 0; i < n && ok; ++i) {
                    const int tiles = items[i].n, groups = items[i].head_groups >> 16;
                    for (int j = 0; j < tiles && ok; ++j, ++g) {
                        const int st = g % kStages;
                        const uint32_t kb = bar + 8 * (kFKFull + st), kph = (g / kStages) & 1;
    #pragma unroll 1
                        for (int t = groups == 2; t < (groups == 1 ? 1 : 2); ++t) {
                            const int c = t ? c1 : c0, b = c & 1;
                            if (j == 0)
                                ok = __all_sync(kFull, mbar_spin_bounded(bar + 8 * ((NARROW ? kFQConv : kFQ) + t), (t ? q1 : q0) & 1,
                                                                         a.timeout_ns));
                            if (ok)
                                ok = c < 2 ? __all_sync(kFull, mbar_spin_bounded(kb, kph, a.timeout_ns))
                                           : __all_sync(kFull, mbar_spin2_bounded(bar + 8 * (kFPV + 2 * t + b), ((c - 2) >> 1) & 1,
                                                                                  kb, kph, a.timeout_ns));
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t a0 = d_kmaj + ((2 * t * kQHalf) >> 4);
                            const uint64_t b0 = d_kmaj + ((PL::kOffK + st * kStage) >> 4);
                            const uint32_t d = tmem + kColS + 128 * t + 64 * b;
                            if constexpr (NARROW == 1) {
                                // E4M3: the query rows' hi codes in the slot's first 16 KB, their lo codes in the second
    #pragma unroll
                                for (int kk = 0; kk < 4; ++kk) {
                                    tc_mma_f8_warp(d, a0 + 2 * kk, b0 + 2 * kk, kIdescS8, kk > 0);
                                    tc_mma_f8_warp(d, a0 + (kQHalf >> 4) + 2 * kk, b0 + 2 * kk, kIdescS8, 1u);
                                }
                            } else {
    #pragma unroll
                                for (int kk = 0; kk < 8; ++kk)
                                    tc_mma_f16_warp(d, a0 + (((kk >> 2) * kQHalf + (kk & 3) * 32) >> 4),
                                                    b0 + (((kk >> 2) * kKvHalf + (kk & 3) * 32) >> 4), kIdescS<NARROW>, kk > 0);
                            }
                            tc_commit_warp(bar + 8 * (kFS + 2 * t + b));
                            if (t) ++c1; else ++c0;
                        }
                        if (ok) tc_commit_warp(bar + 8 * (kFKEmpty + st));
                    }
                    q0 += groups & 1;
                    q1 += groups >> 1;
                }
            });
        } else if (warp == 11) {
            // ------------------------------------------------ O += P V once group t's softmax of its tile c is done
            const uint64_t d_v = smem_desc_sw128(sb, kKvHalf, 1024);  // V: N-major, d-halves kKvHalf apart
            int g = 0, c0 = 0, c1 = 0;
            batches([&](int n) {
                for (int i = 0; i < n && ok; ++i) {
                    const int tiles = items[i].n, groups = items[i].head_groups >> 16;
                    for (int j = 0; j < tiles && ok; ++j, ++g) {
                        const int st = g % kStages;
                        const uint32_t vb = bar + 8 * (kFVFull + st), vph = (g / kStages) & 1;
    #pragma unroll 1
                        for (int t = groups == 2; t < (groups == 1 ? 1 : 2); ++t) {
                            const int c = t ? c1 : c0, b = c & 1;
                            ok = __all_sync(kFull, mbar_spin2_bounded(bar + 8 * (kFP + 2 * t + b), (c >> 1) & 1, vb, vph,
                                                                      a.timeout_ns));
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t b0 = d_v + ((PL::kOffV + st * kStage) >> 4);
                            const uint32_t d = tmem + kColO + 128 * t, p = tmem + kColS + 128 * t + 64 * b;
                            const uint32_t acc0 = j > 0;
                            if constexpr (NARROW == 1) {
                                // E4M3: P's hi codes in 16 columns (four per column), its lo codes in the next 16
    #pragma unroll
                                for (int kc = 0; kc < kKeys / 32; ++kc) {
                                    tc_mma_f8_ts_warp(d, p + 8 * kc, b0 + ((kc * 4096) >> 4), kIdescPV8, kc > 0 ? 1u : acc0);
                                    tc_mma_f8_ts_warp(d, p + 16 + 8 * kc, b0 + ((kc * 4096) >> 4), kIdescPV8, 1u);
                                }
                            } else {
    #pragma unroll
                                for (int kk = 0; kk < kKeys / 16; ++kk)
                                    tc_mma_f16_ts_warp(d, p + 8 * kk, b0 + ((kk * 2048) >> 4), kIdescPV<NARROW>,
                                                       kk > 0 ? 1u : acc0);
                            }
                            tc_commit_warp(bar + 8 * (kFPV + 2 * t + b));
                            if (j == tiles - 1) tc_commit_warp(bar + 8 * (kFO + t));
                            if (t) ++c1; else ++c0;
                        }
                        if (ok) tc_commit_warp(bar + 8 * (kFVEmpty + st));
                    }
                }
            });
        } else if (NARROW == 2 && warp >= 12) {
            // ------------------------------------------------ INT8: rows 32 half + lane of every K (warps 12, 14) or V tile
            // (13, 15) from its staging slot into the f16 ring, exactly (the scales go to the scores and the output)
            const bool is_v = warp & 1;
            const int r = lane + 32 * ((warp - 12) >> 1), sw = r & 7;
            const int full = is_v ? kFVFull : kFKFull, empty = is_v ? kFVEmpty : kFKEmpty;
            int g = 0;
            batches([&](int n) {
                for (int i = 0; i < n && ok; ++i) {
                    const int tiles = items[i].n;
                    for (int j = 0; j < tiles; ++j, ++g) {
                        const int slot = g % (PL::kSlots ? PL::kSlots : 1), st = g % kStages;
                        if (!__all_sync(kFull, mbar_spin_bounded(bar + 8 * (kFStg + 4 * is_v + slot),
                                                                 (g / (PL::kSlots ? PL::kSlots : 1)) & 1, a.timeout_ns)) ||
                            (g >= kStages && !__all_sync(kFull, mbar_spin_bounded(bar + 8 * (empty + st), (g / kStages - 1) & 1,
                                                                                  a.timeout_ns)))) {
                            give_up();
                            break;
                        }
                        const uint8_t* src = smem + PL::kOffStg + (is_v * PL::kSlots + slot) * kStgSlot + r * 128;
                        uint8_t* dst = smem + (is_v ? PL::kOffV : PL::kOffK) + st * kStage + r * 128;
    #pragma unroll
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
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PL::kRegsSoftmax));
        // ------------------------------------------------ softmax groups: warps 0-3 A, 4-7 B; thread r owns query row r
        const int t = warp >> 2, r = tid & 127;
        const uint32_t trow = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tO = tmem + kColO + 128 * t + trow;
        uint8_t* q_slot = smem + 2 * t * kQHalf;
        int c = 0, q_n = 0, q_sent = 0;  // key tiles, items, Q copies of this group
        int g = 0;                       // key tiles of the CTA before the current item
        auto copy_q = [&](int i, int n) {  // by the group's first thread: Q of its first item from the i-th on
            while (i < n && !(items[i].head_groups >> (16 + t) & 1)) ++i;
            if (i == n) return;
            const Item it = items[i];
            const int first = it.q_row + (it.head_groups >> 16 == 3 ? t * rows_q : 0);
            const uint32_t qb = bar + 8 * (kFQ + t);
            mbar_arrive_expect_tx(qb, 2 * kQHalf);
            for (int hf = 0; hf < 2; ++hf)
                tma_load_3d_nohint(smem_u32(q_slot) + hf * kQHalf, &qmap, hf * 64, (it.head_groups & 0xffff) * a.G, first, qb);
            ++q_sent;
        };
        batches([&](int n) {
            if (r == 0 && ok) copy_q(0, n);
            for (int i = 0; i < n && ok; ++i) {
                const Item& it = items[i];
                if (!(it.head_groups >> (16 + t) & 1)) {
                    g += it.n;
                    continue;
                }
                const bool pair = it.head_groups >> 16 == 3;
                const int row = (pair ? t * kRows : 0) + r;  // of the item's rows
                const bool valid = row < it.tokens * a.G;
                float m_ref = -INFINITY, l_run = 0.f;
                float sm_log2 = a.k_head ? a.sm_base * __ldg(a.k_head + (it.head_groups & 0xffff)) : a.sm_log2;
                if constexpr (NARROW != 0) {
                    if (!__all_sync(kFull, mbar_spin_bounded(bar + 8 * (kFQ + t), q_n & 1, a.timeout_ns))) {
                        give_up();
                        break;
                    }
                }
                if constexpr (NARROW == 1) {
                    // This thread's query row (bf16: dims 0-63 in the slot's first 16 KB, 64-127 in the second) is scaled
                    // by 2^e, e chosen so that its largest magnitude lies in [128, 256), and split into hi = E4M3(x) and
                    // lo = E4M3(x - hi), written over the row (hi codes in the first 16 KB, lo codes in the second);
                    // hi + lo is the scaled value exactly for elements within 2^-10 of the row's largest.  The scores
                    // are multiplied back by 2^-e.
                    uint8_t* qt = q_slot + r * 128;
                    const int sw = r & 7;
                    auto dims8 = [&](int hf, int k) -> uint4 {  // bf16 dims 64 hf + 8 k .. + 7
                        return *reinterpret_cast<const uint4*>(qt + hf * kQHalf + ((k ^ sw) << 4));
                    };
                    auto amax4 = [](uint32_t m, const uint4& x) {  // |value| bits: ordered like the values
                        const uint32_t ws[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u) m = max(m, max((ws[u] << 17) >> 1, ((ws[u] >> 16) & 0x7fffu) << 16));
                        return m;
                    };
                    uint4 w1[8];  // dims 64..127, kept: the lo codes of dims 0..63 are written over them
                    uint32_t amax_bits = 0;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        w1[k] = dims8(1, k);
                        amax_bits = amax4(amax4(amax_bits, w1[k]), dims8(0, k));
                    }
                    if (amax_bits >= 0x7f800000u && valid) raise_error(a.err, PKV_DEVERR_Q_RANGE);  // inf or NaN
                    const int ex = static_cast<int>(amax_bits >> 23) - 127;  // floor(log2(max |x|))
                    const int e = min(126, max(-126, 7 - ex));
                    const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
                    sm_log2 *= __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {  // output chunk k: head dims 16 k .. 16 k + 15
                        const uint4 s0 = k < 4 ? dims8(0, 2 * k) : w1[2 * k - 8];
                        const uint4 s1 = k < 4 ? dims8(0, 2 * k + 1) : w1[2 * k - 7];
                        uint32_t hw[4], lw[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {  // dims 16 k + 4 u .. + 3
                            const uint4 src = (u >> 1) ? s1 : s0;
                            const uint32_t x01 = (u & 1) ? src.z : src.x, x23 = (u & 1) ? src.w : src.y;
                            const float2 f01 = bf16x2_to_float2(x01), f23 = bf16x2_to_float2(x23);
                            const float v0 = f01.x * up, v1 = f01.y * up, v2 = f23.x * up, v3 = f23.y * up;
                            const uint32_t h01 = f32x2_to_e4m3x2(v0, v1), h23 = f32x2_to_e4m3x2(v2, v3);
                            const float2 b01 = f16x2_to_float2(e4m3x2_to_f16x2_u(h01));
                            const float2 b23 = f16x2_to_float2(e4m3x2_to_f16x2_u(h23));
                            hw[u] = h01 | (h23 << 16);
                            lw[u] = f32x2_to_e4m3x2(v0 - b01.x, v1 - b01.y) | (f32x2_to_e4m3x2(v2 - b23.x, v3 - b23.y) << 16);
                        }
                        *reinterpret_cast<uint4*>(qt + ((k ^ sw) << 4)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
                        *reinterpret_cast<uint4*>(qt + kQHalf + ((k ^ sw) << 4)) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
                    }
                }
                if constexpr (NARROW == 2) {
                    // f16 MMAs: this thread's row converted in place, exactly for |q| in [2^-14, 65504]
                    bool in_range = true;
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        uint4* p = reinterpret_cast<uint4*>(q_slot + (k >> 3) * kQHalf + r * 128 + (((k & 7) ^ (r & 7)) << 4));
                        const uint4 w = *p;
                        uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float2 x = bf16x2_to_float2(ws[u]);
                            in_range = in_range && fabsf(x.x) < 65520.f && fabsf(x.y) < 65520.f;
                            ws[u] = f16x2_rn(x.x, x.y);
                        }
                        *p = make_uint4(ws[0], ws[1], ws[2], ws[3]);
                    }
                    if (!in_range && valid) raise_error(a.err, PKV_DEVERR_Q_RANGE);
                }
                if constexpr (NARROW != 0) {
                    fence_proxy_async_smem();  // the S MMAs (async proxy) read what was written
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar + 8 * (kFQConv + t));
                }

                bool s_ready = false;  // the next tile's scores were seen complete ahead of time
                const int tiles = it.n;
                int left = it.keys - it.j0 * kKeys;  // keys from the current tile on
                for (int j = 0; j < tiles; ++j, ++c, left -= kKeys) {
                    const int b = c & 1;
                    const uint32_t tS = tmem + kColS + 128 * t + 64 * b + trow;
                    if (!__all_sync(kFull, s_ready) &&
                        !__all_sync(kFull, mbar_spin_bounded(bar + 8 * (kFS + 2 * t + b), (c >> 1) & 1, a.timeout_ns))) {
                        give_up();
                        break;
                    }
                    tc_fence_after();
                    if (j == tiles - 1 && r == 0) copy_q(i + 1, n);  // every product with this item's Q has completed
                    float v[64];
                    tmem_ld64(tS, v);
                    // test the next tile's scores now; the answer is used only when that tile starts
                    s_ready = j + 1 < tiles && mbar_test(bar + 8 * (kFS + 2 * t + (b ^ 1)), ((c + 1) >> 1) & 1);
                    const bool masked = left < kKeys;
                    float mx[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) mx[u] = -INFINITY;
                    if (!masked) {
#pragma unroll
                        for (int u = 0; u < 64; u += 2) mx[(u >> 1) & 7] = fmax3(mx[(u >> 1) & 7], v[u], v[u + 1]);
                    } else {
#pragma unroll
                        for (int u = 0; u < 64; ++u) mx[u & 7] = fmaxf(mx[u & 7], u < left ? v[u] : -INFINITY);
                    }
                    const float mraw = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                             fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
                    const float mt = mraw * sm_log2;
                    const bool need = mt > m_ref + 8.f;
                    // O is rescaled (below) only when some row of the warp needs it; rows that do not keep alpha = 1
                    const bool rescale = j > 0 && __any_sync(kFull, need);
                    const float m_new = need ? (NARROW == 1 ? mt - kP8Shift : mt) : m_ref;
                    const float alpha = ex2_approx(m_ref - m_new);
                    m_ref = m_new;
                    const float2 sc2 = make_float2(sm_log2, sm_log2), nm2 = make_float2(-m_ref, -m_ref);
                    float2 ls2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    uint32_t pk[32];  // bf16 / f16 pairs; FP8: 16 words of four hi codes, then 16 of four lo codes
                    auto exp_pack = [&](auto with_mask) {
#pragma unroll
                        for (int u = 0; u < 64; u += 2) {
                            const float2 x = __ffma2_rn(make_float2(v[u], v[u + 1]), sc2, nm2);
                            float p0 = ex2_approx(x.x);
                            float p1 = ex2_approx(x.y);
                            if constexpr (decltype(with_mask)::value) {
                                p0 = u < left ? p0 : 0.f;
                                p1 = u + 1 < left ? p1 : 0.f;
                            }
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
                    };
                    if (masked) exp_pack(std::true_type{});
                    else exp_pack(std::false_type{});
                    const float2 lsum = __fadd2_rn(ls2[0], ls2[1]);
                    l_run = l_run * alpha + (lsum.x + lsum.y);
                    tmem_st32u(tS, pk);  // P over the scores just read (this thread's lane only)
                    if (rescale) {
                        // O may be touched only once the previous P V of this group has completed
                        if (!__all_sync(kFull, mbar_wait_bounded(bar + 8 * (kFPV + 2 * t + ((c - 1) & 1)), ((c - 1) >> 1) & 1,
                                                                 a.timeout_ns))) {
                            give_up();
                            break;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float o[64];
                            tmem_ld64(tO + 64 * k, o);
#pragma unroll
                            for (int u = 0; u < 64; ++u) o[u] *= alpha;
                            tmem_st64(tO + 64 * k, o);
                        }
                    }
                    // keys past the last: their V rows are not data, make them zero once they have landed (the item's
                    // first group does it: its P V is issued first)
                    if (masked && (t == 0 || !pair)) {
                        const int st = (g + j) % kStages;
                        if (!__all_sync(kFull, mbar_wait_bounded(bar + 8 * (kFVFull + st), ((g + j) / kStages) & 1,
                                                                 a.timeout_ns))) {
                            give_up();
                            break;
                        }
                        constexpr int kRowChunks = NARROW == 1 ? 8 : 16;  // 16-byte pieces of a key's row
                        for (int u = r; u < (kKeys - left) * kRowChunks; u += 128) {
                            const int key = left + u / kRowChunks, k = u % kRowChunks;
                            *reinterpret_cast<uint4*>(smem + PL::kOffV + st * kStage + (k >> 3) * kKvHalf + key * 128 +
                                                      (k & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                    }
                    tc_fence_before();
                    mbar_arrive(bar + 8 * (kFP + 2 * t + b));
                }
                g += it.n;
                if (!ok) break;
                // ---- the item's last product: out = O / l, or a record of (O, m, l)
                if (!__all_sync(kFull, mbar_wait_bounded(bar + 8 * (kFO + t), q_n & 1, a.timeout_ns))) {
                    give_up();
                    break;
                }
                ++q_n;
                tc_fence_after();
                const int h = it.head_groups & 0xffff;
                const size_t tok_row = (static_cast<size_t>(it.q_row) + row / a.G) * a.Hq + static_cast<size_t>(h) * a.G + row % a.G;
                if (it.rec != 0) {
                    const size_t rec = it.rec == 1 ? tok_row : static_cast<size_t>(f.extra_row) + static_cast<size_t>(cta) * 256 + row;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float o[64];
                        tmem_ld64(tO + 64 * k, o);
                        if (valid) {
#pragma unroll
                            for (int u = 0; u < 8; ++u) store_v8(f.rec_o + rec * 128 + 64 * k + 8 * u, o + 8 * u);
                        }
                    }
                    if (valid) f.rec_ml[rec] = make_float2(m_ref, l_run);
                } else {
                    const float inv = l_run > 0.f ? (a.v_head ? __ldg(a.v_head + h) : a.out_mul) / l_run : 0.f;
                    uint4* orow = reinterpret_cast<uint4*>(a.out) + tok_row * 16;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float o[64];
                        tmem_ld64(tO + 64 * k, o);
                        if (valid) {
#pragma unroll
                            for (int u = 0; u < 8; ++u)
                                orow[8 * k + u] = make_uint4(bf16x2_rn(o[8 * u] * inv, o[8 * u + 1] * inv),
                                                             bf16x2_rn(o[8 * u + 2] * inv, o[8 * u + 3] * inv),
                                                             bf16x2_rn(o[8 * u + 4] * inv, o[8 * u + 5] * inv),
                                                             bf16x2_rn(o[8 * u + 6] * inv, o[8 * u + 7] * inv));
                        }
                    }
                }
                tc_fence_before();  // the next item's first P V overwrites O, once this group's P of it is there
            }
        });
        // a Q copy that nobody waited for (after a timeout) lands before the CTA finishes
        if (r == 0 && !ok && q_sent > 0) mbar_wait_bounded(bar + 8 * (kFQ + t), (q_sent - 1) & 1, a.timeout_ns);
    }
    if (!ok && lane == 0) *abort_flag = 1;

    // ---- drain: nothing of this CTA may still be in flight when TMEM is freed and the CTA exits
    __syncthreads();
    if ((warp == 9 || warp == 11) && *abort_flag) {
        tc_commit_warp(bar + 8 * kFDrain);  // arrives once every MMA this warp issued has completed
        mbar_wait_bounded(bar + 8 * kFDrain, 0, a.timeout_ns);
    }
    if (*abort_flag && tid == 0) raise_error(a.err, PKV_DEVERR_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, kTmemCols);
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
static size_t full_smem() {
    return static_cast<size_t>(FullPlan<NARROW>::kOffMeta) + kFEnd + 1024;
}

size_t paged_full_smem_bytes(int narrow) { return narrow == 2 ? full_smem<2>() : narrow == 1 ? full_smem<1>() : full_smem<0>(); }

template <int NARROW>
static cudaError_t launch_full(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                               const PrefillArgs& a, const FullArgs& f, int grid, cudaStream_t stream) {
    const size_t smem = full_smem<NARROW>();
    auto kern = paged_full_kernel<NARROW>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    kern<<<grid, FullPlan<NARROW>::kThreads, smem, stream>>>(qmap, kmap, vmap, a, f);
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
