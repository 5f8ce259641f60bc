// attn_paged.cu -- attention of a chunk of new tokens over the paged KV rows
// on the 5th-generation tensor cores (BF16 in, fp32 accumulate): MQA in the MLA
// layout (up to 128 heads share one KV row of 512 latent + 64 rope columns, V is
// the latent part), dense causal or over each query's selected positions.
//
// Split.  O (128 rows x 512 fp32) fills a whole SM's tensor memory, so an item's
// output columns are halved between two CTAs.  Each computes all of
// S = Q K^T (128 x 576 by 576 x 64 a tile) and its 128 x 256 half of O += P V.
// Nothing is exchanged: the CTAs are independent.  The price is computing S
// twice, 1344 tensor cycles a tile; halving the contraction between the CTAs of a
// cluster (as attn_tc.cu does) costs an exchange of partial scores and
// probabilities through distributed shared memory, and measured 2590 us here
// (two chunks of 531 and 586 tokens behind 4200 keys each, 128 heads) against 1830
// us: 0.45 of the burst matrix rate, 2700 cycles a tile.  The clock is part of that:
// in a run of calls the power cap holds 1.55 to 1.6 GHz, ten calls after a pause take
// 1585 us (a selected chunk 1100 and 940).  The times beside the choices below are
// short runs of graph replays, 1700 us for this case.
//
// Work items.  An item is a group of query rows and a part of their keys.  A
// selection's item is one query; a dense item is up to 128 / heads consecutive
// tokens of a sequence, so that a rank that holds few heads still fills the 128
// rows of the MMA (row r: token r / heads, head r % heads; each row masks its
// own causal limit).  With fewer items than SM pairs the keys of an item are
// split into parts, which leave normalised fp32 rows and their log-sum-exp in
// the workspace for attn_paged_combine_kernel to join.  The grid is persistent:
// CTA c takes units c, c + grid, ... (unit = item and half).
//
// Pipeline of a 64-key tile g.  A tile's nine 64-column blocks are held in two
// parts: the four that are also V (three stages), and the five that only S reads
// (one stage in two groups, each refilled as soon as its MMAs are done).  The MMA
// thread issues
//     S over group 0 | S over group 1 and the V blocks | PV of g - 1
// so that the softmax of g - 1 runs under S(g), S(g + 1) finds its accumulator read
// while PV(g - 1) runs, and every load has 1300 cycles or more.
//
// Measured on this layout (one SM, cycles): tcgen05.mma M 128, K 16 with A in
// tensor memory: 32 at N 64, issued under elect.sync (45 under lane == 0);
// with A in shared memory 48 (its reads of A and B at 128 bytes a cycle); N 256:
// 128.  So S is 24 x 32 + 12 x 48 = 1344 and PV 512.  Rows gathered by 16-byte
// cp.async reach 70 bytes a cycle (1040 a tile), gather4 TMA 8 to 22.
//
// Tensor memory: O [0, 256), S [256, 320), Q [320, 512) (six of its nine
// 64-column blocks; the other three are read from shared memory).
// Warps: 0-7 softmax (two threads a row, 32 keys each), 8-11 Q loads and the
// epilogue (thread <-> row), 12-18 producers, 19 MMA.
#include <type_traits>

#include "rows.cuh"

namespace dsa {

constexpr int PA_N = 64;                    // keys per tile
constexpr uint32_t PA_BLK = PA_N * 128;     // one 64-column block of a tile
constexpr uint32_t PA_VST = 4 * PA_BLK;     // the blocks that are also V
constexpr uint32_t PA_QBLK = 128 * 128;     // one 64-column block of Q
constexpr int PA_NST = 3;                   // stages of the V blocks
constexpr int PA_THREADS = 640;
constexpr int PA_EPI0 = 8, PA_PROD0 = 12, PA_PRODUCERS = 7, PA_MMA = 19;
constexpr int PA_SCAN_ROUNDS = 2048 / 32 / 4;  // index words per epilogue warp
constexpr int PA_GRPS = (16 + PA_PRODUCERS - 1) / PA_PRODUCERS;                // groups of 4 keys per producer warp
constexpr uint32_t PA_TM_O = 0, PA_TM_S = 256, PA_TM_Q = 320;

// One work item's rows and its part of their keys.
struct PaItem {
    int64_t t0;        // first query token
    int64_t pos0;      // its position
    int64_t seqlen_k;
    int ntok;          // query tokens (0: an empty item)
    int b;
    int lo, count;     // dense: first key position and keys of the part; selected: slots
    bool ok;
};

struct PaLayout {
    static constexpr uint32_t OFF_K = 0;
    static constexpr uint32_t OFF_V = OFF_K + 5 * PA_BLK;
    static constexpr uint32_t OFF_Q = OFF_V + PA_NST * PA_VST;   // three blocks of Q
    static constexpr uint32_t OFF_P = OFF_Q + 3 * PA_QBLK;       // probabilities, no-swizzle K-major
    static constexpr uint32_t OFF_EPI = OFF_P + 128 * PA_N * 2;  // per epilogue warp 32 rows x 128 bytes
    static constexpr uint32_t OFF_ML = OFF_EPI + 4 * 4096;       // [2] maxima [128], sums [2][128]
    static constexpr uint32_t OFF_XM = OFF_ML + 2 * 1536;        // [2][2][128] the key halves' maxima of a tile
    static constexpr uint32_t OFF_VM = OFF_XM + 2 * 1024;        // [2][64] validity bits of 2048 slots
    static constexpr uint32_t OFF_ITEM = OFF_VM + 512;           // [2] PaItem
    static constexpr uint32_t OFF_INFO = OFF_ITEM + 128;         // [2][8] per epilogue warp: last used slot, (dense) pages missing
    static constexpr uint32_t OFF_BAR = OFF_INFO + 64;
    static constexpr uint32_t SMEM = OFF_BAR + 256;
};
static_assert(2 * sizeof(PaItem) <= 128, "item ring");
static_assert(PaLayout::SMEM <= 232448, "shared memory budget");

struct PaBars {
    uint64_t kfull, kfree[2];                // the two groups of the blocks that only S reads
    uint64_t vfull[PA_NST], vfree[PA_NST];   // (vfull: of the second group too)
    uint64_t s_full, s_free;    // S complete / read by the softmax warps
    uint64_t p_full, p_free;    // P written (and O rescaled) / its PV complete
    uint64_t q_full, q_free;    // Q in place / its last S complete
    uint64_t o_full, o_free;    // O complete / read by the epilogue
    uint64_t xm_full[4];        // a tile's maxima of both key halves, per lane quadrant
    uint64_t ml_full[2];        // an item's maxima and sums, per ring slot
    uint64_t info_full[2], info_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(PaBars) <= 256, "barrier block");

DSA_DEV uint32_t pa_swz(int row, int chunk) { return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4)); }

// One lane of a converged warp.  Issuing tcgen05.mma under it, and not under
// lane == 0, keeps the descriptors in uniform registers (32 against 45 cycles an
// MMA of N 64).
DSA_DEV bool elect_one() {
    uint32_t p;
    asm volatile("{ .reg .pred P; elect.sync _|P, 0xffffffff; selp.u32 %0, 1, 0, P; }" : "=r"(p));
    return p != 0;
}

// mbar_wait with the bounded loop out of line, for the thread that issues the MMAs:
// its code between two batches is what the tensor core waits for (dense chunks 1915
// us inlined, 1770 so; the other warps' waits are better inlined).
__device__ __noinline__ bool pa_wait_long(uint32_t bar, uint32_t parity, volatile int* abort, StatusHdr* st, int where) {
    return mbar_wait(bar, parity, abort, st, where);
}
DSA_DEV bool pa_wait_one(uint32_t bar, uint32_t parity, volatile int* abort, StatusHdr* st, int where) {
    return mbar_test(bar, parity) || pa_wait_long(bar, parity, abort, st, where);
}
// 16 bytes global -> shared; n = 0: zeros, the source is not read
DSA_DEV void cp_async16_n(uint32_t dst, const void* src, uint32_t n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"((uint64_t)src), "r"(n) : "memory");
}

DSA_DEV uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// First item slot of sequence b's groups: groups of R tokens never cross a
// sequence; ceil(l / R) of them fit between floor(cu[b] / R) + b and the next.
DSA_DEV int64_t pa_first_group(int64_t cu, int b, int R) { return R == 1 ? cu : cu / R + b; }

template <bool DENSE>
DSA_DEV PaItem pa_item(const PagedAttnArgs& a, int64_t grp, int part, int sel_part) {
    PaItem it = {};
    int b;
    if (!DENSE || a.group == 1) {
        const RowInfo ri = row_info_guess(a.sv, grp, a.total_q);
        it.t0 = grp;
        it.b = ri.b;
        it.pos0 = ri.pos;
        it.seqlen_k = ri.seqlen_k;
        it.ok = ri.ok;
        it.ntok = ri.ok ? 1 : 0;  // rows without a valid position are left as they were
    } else {
        int lo = 0, hi = a.sv.batch - 1;
        while (lo < hi) {  // largest b whose first group is not past grp
            const int mid = (lo + hi + 1) >> 1;
            if (pa_first_group(__ldg(a.sv.cu_q + mid), mid, a.group) <= grp) lo = mid;
            else hi = mid - 1;
        }
        b = lo;
        const int64_t q0 = __ldg(a.sv.cu_q + b), lq = __ldg(a.sv.cu_q + b + 1) - q0;
        const int64_t lk = __ldg(a.sv.cu_k + b + 1) - __ldg(a.sv.cu_k + b);
        const int64_t i0 = (grp - pa_first_group(q0, b, a.group)) * a.group;
        it.b = b;
        it.t0 = q0 + i0;
        it.seqlen_k = lk;
        it.pos0 = lk - lq + i0;
        it.ntok = i0 < lq ? (int)min((int64_t)a.group, lq - i0) : 0;
        it.ok = it.ntok == 0 || (it.pos0 >= 0 && q0 >= 0 && it.t0 + it.ntok <= a.total_q);
        if (!it.ok) it.ntok = 0;
    }
    if (!it.ok || it.ntok == 0) return it;
    if (DENSE) {
        const int64_t n = it.pos0 + it.ntok;  // keys of the last row
        const int64_t per = ((n + PA_N - 1) / PA_N + a.splits - 1) / a.splits * PA_N;
        const int64_t lo = part * per;
        it.lo = (int)min(lo, n);
        it.count = (int)(min(n, lo + per) - it.lo);
    } else {
        it.lo = min(part * sel_part, a.k_sel);
        it.count = min(a.k_sel, it.lo + sel_part) - it.lo;
    }
    return it;
}

template <bool DENSE>
__global__ void __launch_bounds__(PA_THREADS, 1) attn_paged_kernel(const __grid_constant__ PagedAttnArgs a) {
    using Lay = PaLayout;
    extern __shared__ __align__(1024) uint8_t smem[];
    PaBars* bars = (PaBars*)(smem + Lay::OFF_BAR);
    uint32_t* vmask = (uint32_t*)(smem + Lay::OFF_VM);
    PaItem* items = (PaItem*)(smem + Lay::OFF_ITEM);  // [2]
    int* pmax = (int*)(smem + Lay::OFF_INFO);         // [2][8]
    if (smem_u32(smem) & 1023) {                      // the layout needs a 1024-byte aligned base
        if (threadIdx.x == 0) report(a.st, DSA_ERR_UNSUPPORTED, -3);
        return;
    }
    // (broadcasts tell the compiler that a value, and with it a branch or a loop, is
    // the same in all lanes: only then do the MMA operands live in uniform registers)
    const int warp = __shfl_sync(0xffffffffu, (int)warp_id(), 0), lane = (int)lane_id();
    next_grid();
    StatusHdr* st = a.st;
    volatile int* abort = &bars->abort;

    // this CTA's units: blockIdx.x + i * gridDim.x (an even grid: always the same half)
    const int half = (int)(blockIdx.x & 1);
    const int64_t item0 = blockIdx.x >> 1, step = gridDim.x >> 1, n_items = a.groups * a.splits;
    const int64_t nq = item0 < n_items ? (n_items - item0 + step - 1) / step : 0;
    // slots of a selection's part
    const int sel_part = DENSE ? 0 : ((a.k_sel + PA_N - 1) / PA_N + a.splits - 1) / a.splits * PA_N;
    // 64-column blocks of the row: V's four, and the other five (the first three of
    // these have their Q in shared memory)
    auto vblk = [&](int i) { return 4 * half + i; };
    auto kblk = [&](int i) { return i == 4 ? 8 : 4 * (half ^ 1) + i; };

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bars->kfull), PA_PRODUCERS * 32);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&bars->kfree[i]), 1);
        for (int i = 0; i < PA_NST; ++i) {
            mbar_init(smem_u32(&bars->vfull[i]), PA_PRODUCERS * 32);
            mbar_init(smem_u32(&bars->vfree[i]), 1);
        }
        mbar_init(smem_u32(&bars->s_full), 1);
        mbar_init(smem_u32(&bars->s_free), 8);
        mbar_init(smem_u32(&bars->p_full), 8);
        mbar_init(smem_u32(&bars->p_free), 1);
        mbar_init(smem_u32(&bars->q_full), 8);
        mbar_init(smem_u32(&bars->q_free), 1);
        mbar_init(smem_u32(&bars->o_full), 1);
        mbar_init(smem_u32(&bars->o_free), 4);
        for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&bars->xm_full[i]), 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars->ml_full[i]), 8);
            mbar_init(smem_u32(&bars->info_full[i]), 4);
            mbar_init(smem_u32(&bars->info_empty[i]), 9 + PA_PRODUCERS);  // 8 softmax warps, the MMA warp, the producers
        }
        mbar_init(smem_u32(&bars->drain), 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == PA_MMA) tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const uint32_t s_k = smem_u32(smem + Lay::OFF_K), s_v = smem_u32(smem + Lay::OFF_V);
    // tiles of the item in ring slot qi & 1 (its info has arrived)
    auto tiles_of = [&](int64_t qi) {
        int mx = -1;
#pragma unroll
        for (int w = 0; w < 4; ++w) mx = max(mx, pmax[(qi & 1) * 8 + w]);
        return __shfl_sync(0xffffffffu, (mx + PA_N) / PA_N, 0);
    };
    auto info_wait = [&](int64_t qi, int where) {
        return wait_warp(smem_u32(&bars->info_full[qi & 1]), (uint32_t)((qi >> 1) & 1), abort, st, where);
    };
    auto info_done = [&](int64_t qi) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->info_empty[qi & 1]));
    };

    // Sets the values that are not finite to zero in the V rows row0 + i, i in `keys`, of
    // the stage at sv (S of the tile is complete, its PV not issued).  Warps may do this
    // together: they write the same zeros.
    auto clear_not_finite = [&](uint32_t sv, int row0, uint32_t keys) {
        for (; keys; keys &= keys - 1) {
            const int row = row0 + __ffs((int)keys) - 1;
            const uint32_t at = sv + (lane >> 3) * PA_BLK + pa_swz(row, lane & 7);  // 4 blocks x 8 chunks
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t v;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at + 4 * i) : "memory");
                uint32_t w = v;
                if ((v & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
                if ((v & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
                if (w != v) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 4 * i), "r"(w) : "memory");
            }
        }
    };

    // Q of an item: three blocks into shared memory, six through registers and
    // this warp's staging tile (a row a lane) into tensor memory.  Rows past the
    // item are zero.  Loads take 4 rows x 128 bytes an instruction: a row a lane
    // costs 32 cache lines each (9200 cycles an item, now about 2500).
    // wait: until the last S of the item before has completed
    // part: of two warps that share the rows, the first or the second half of the
    // blocks; 2: all.
    auto load_q = [&](const PaItem& it, int quad, uint8_t* stg, int part, auto wait) -> bool {
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const int sub = lane >> 3, chunk = lane & 7;
        int64_t off[8];  // rows 4 j + sub of this warp
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = quad * 32 + 4 * j + sub, tk = r / a.heads;
            off[j] = tk < it.ntok ? (it.t0 + tk) * a.q_stride_tok + (int64_t)(r - tk * a.heads) * a.q_stride_head + chunk * 8
                                  : -1;
        }
        const __nv_bfloat16* q = (const __nv_bfloat16*)a.q;
        uint4 x[8];
        auto fetch = [&](int blk) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = off[j] >= 0 ? __ldg((const uint4*)(q + off[j] + blk * 64)) : make_uint4(0u, 0u, 0u, 0u);
        };
        auto blk_of = [&](int i) { return i < 2 ? kblk(3 + i) : vblk(i - 2); };  // tensor-memory blocks in their order
        const int i0 = part == 1 ? 3 : 0, i1 = part == 0 ? 3 : 6;
        fetch(blk_of(i0));
        if (!wait()) return false;
        tc_fence_after();
        const uint32_t sq = smem_u32(smem + Lay::OFF_Q);
#pragma unroll 1
        for (int i = part == 1 ? 2 : 0; i < (part == 0 ? 2 : 3); ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                cp_async16_n(sq + i * PA_QBLK + pa_swz(quad * 32 + 4 * j + sub, chunk),
                             q + (off[j] >= 0 ? off[j] + kblk(i) * 64 : 0), off[j] >= 0 ? 16u : 0u);
#pragma unroll 1
        for (int i = i0; i < i1; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) *(uint4*)(stg + pa_swz(4 * j + sub, chunk)) = x[j];
            __syncwarp();
            if (i + 1 < i1) fetch(blk_of(i + 1));
            uint32_t r[32];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint4 v = *(const uint4*)(stg + pa_swz(lane, c));
                r[4 * c] = v.x, r[4 * c + 1] = v.y, r[4 * c + 2] = v.z, r[4 * c + 3] = v.w;
            }
            tmem_st32(tmem + lane_off + PA_TM_Q + i * 32, r);
            __syncwarp();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        tmem_wait_st();
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        return true;
    };

    if (warp >= PA_PROD0 && warp < PA_MMA) {
        // ================= gather producers =================
        const int pw = warp - PA_PROD0;
        // 16 groups of 4 keys per tile; warp w takes groups w, w + 7, w + 14
        const int sub = lane >> 3, chunk = lane & 7;
        const int ngrp = (16 - pw + PA_PRODUCERS - 1) / PA_PRODUCERS;
        uint32_t g = 0;  // tile of the CTA's whole sequence
        bool ok = true;
        const __nv_bfloat16* pool = (const __nv_bfloat16*)a.k + chunk * 8;
        // the first item's first two tiles into L2, before its info is there
        if (nq > 0) {
            const int64_t grp = item0 / a.splits;
            const PaItem it = pa_item<DENSE>(a, grp, (int)(item0 - grp * a.splits), sel_part);
            for (int key = 4 * pw + sub; key < min(2 * PA_N, it.count); key += 4 * PA_PRODUCERS) {
                const int32_t v = DENSE ? it.lo + key : __ldg(a.idx + it.t0 * a.ld_idx + it.lo + key);
                if (v < 0 || v >= it.seqlen_k) continue;
                const PageRef pr = page_of(a.pv, it.b, v);
                if (pr.page < 0) continue;
                const __nv_bfloat16* row = (const __nv_bfloat16*)a.k + pr.page * a.k_page_stride + (int64_t)pr.slot * a.k_stride;
                prefetch_l2(row + chunk * 64);
                if (chunk == 0) prefetch_l2(row + 512);
            }
        }
        for (int64_t qi = 0; ok && qi < nq; ++qi) {
            if (!info_wait(qi, 0x2103)) break;
            const PaItem it = items[qi & 1];
            const int n_tiles = tiles_of(qi);
            info_done(qi);
            const int32_t* irow = DENSE ? nullptr : a.idx + it.t0 * a.ld_idx + it.lo;
            const int count = it.count;  // keys (dense) or slots of this item's part
            // ---- the item's tiles.  A row's place takes two dependent loads (its
            // position, its page): positions are read two tiles ahead and pages one,
            // so that neither is waited for. ----
            auto position = [&](int j, int gi) -> int32_t {
                const int sj = j * PA_N + 4 * (pw + PA_PRODUCERS * gi) + sub;
                if (gi >= ngrp || sj >= count) return -1;
                return DENSE ? it.lo + sj : __ldg(irow + sj);
            };
            const int32_t* table = a.pv.table + it.b * a.pv.ld_table;
            int32_t np[PA_GRPS] = {}, ps[PA_GRPS], pg[PA_GRPS];  // positions of tile j + 1; slots and pages of tile j
            auto look_up = [&](int gi) {
                int32_t v = np[gi];
                if (!DENSE && v >= it.seqlen_k) v = -1;
                uint32_t p, o;
                page_split(a.pv, (uint32_t)v, p, o);
                ps[gi] = (int32_t)o;
                pg[gi] = v >= 0 && (int64_t)p < a.pv.ld_table ? __ldg(table + p) : -1;
            };
            if (n_tiles > 0) {
#pragma unroll
                for (int gi = 0; gi < PA_GRPS; ++gi) {
                    np[gi] = position(0, gi);
                    look_up(gi);
                    np[gi] = position(1, gi);
                }
            }
            for (int j = 0; j < n_tiles; ++j, ++g) {
                const uint32_t s = g % PA_NST;
                const __nv_bfloat16* src[PA_GRPS];
                uint32_t n[PA_GRPS];
#pragma unroll
                for (int gi = 0; gi < PA_GRPS; ++gi) {
                    // a slot that holds no row is filled with zeros, so that a masked
                    // probability of zero never meets a stray NaN or infinity
                    const bool have = (uint32_t)pg[gi] < (uint32_t)a.pv.num_pages;
                    if (DENSE && !have && gi < ngrp && j * PA_N + 4 * (pw + PA_PRODUCERS * gi) + sub < count)
                        report(st, DSA_ERR_INDEX, it.t0);
                    src[gi] = have ? pool + (int64_t)pg[gi] * a.k_page_stride + (int64_t)ps[gi] * a.k_stride : pool;
                    n[gi] = have ? 16u : 0u;
                    look_up(gi);
                    np[gi] = position(j + 2, gi);
                }
                bool got = true;
                auto copy = [&](uint32_t base, int i0, int i1, bool v) {  // blocks [i0, i1) of this warp's rows
#pragma unroll
                    for (int gi = 0; gi < PA_GRPS; ++gi) {
                        if (gi >= ngrp) break;
                        const uint32_t dst = base + pa_swz(4 * (pw + PA_PRODUCERS * gi) + sub, chunk);
#pragma unroll
                        for (int i = i0; i < i1; ++i)
                            cp_async16_n(dst + i * PA_BLK, src[gi] + (v ? vblk(i) : kblk(i)) * 64, n[gi]);
                    }
                };
                // (the V blocks first: their buffers are free long before the others')
                got = wait_warp(smem_u32(&bars->vfree[s]), ((g / PA_NST) & 1) ^ 1, abort, st, 0x2104);
                if (got) {
                    copy(s_v + s * PA_VST, 0, 4, true);
                    got = wait_warp(smem_u32(&bars->kfree[0]), (g & 1) ^ 1, abort, st, 0x2101);
                }
                if (got) {
                    copy(s_k, 0, 3, false);
                    cp_async_arrive(smem_u32(&bars->kfull));
                    got = wait_warp(smem_u32(&bars->kfree[1]), (g & 1) ^ 1, abort, st, 0x2105);
                }
                if (!got) { ok = false; break; }
                copy(s_k, 3, 5, false);
                cp_async_arrive(smem_u32(&bars->vfull[s]));
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == PA_MMA) {
        // ================= MMA issuer =================
        // One thread waits and issues, tile after tile: it runs only a few MMAs ahead of
        // the tensor core, so every wait between its batches idles it, and a wait by the
        // whole warp costs 115 cycles even for a barrier that is long complete, by one
        // thread 56.  For the same reason its code is short (the V stage is an offset:
        // 1710 us against 1770 with a copy for each stage).  The tensor memory is all
        // this CTA's, so it begins at column 0.
        constexpr uint32_t idesc_s = idesc_make(1, 1, false, 128, PA_N);
        constexpr uint32_t idesc_pv = idesc_make(1, 1, true, 128, 256);
        const uint32_t base = smem_u32(smem);
        auto issue_sk = [&](auto grp_c) {  // S over group 0 (Q in shared memory) or 1 (in tensor memory)
            constexpr int grp = decltype(grp_c)::value;
#pragma unroll
            for (int i = grp ? 3 : 0; i < (grp ? 5 : 3); ++i)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t kd = sdesc_sw128(base + Lay::OFF_K + i * PA_BLK + ks * 32, 16, 1024);
                    if (grp == 0)
                        mma_bf16_ss(PA_TM_S, sdesc_sw128(base + Lay::OFF_Q + i * PA_QBLK + ks * 32, 16, 1024), kd, idesc_s,
                                    (i | ks) ? 1u : 0u);
                    else
                        mma_bf16_ts(PA_TM_S, PA_TM_Q + (i - 3) * 32 + ks * 8, kd, idesc_s, 1u);
                }
            mma_commit(smem_u32(&bars->kfree[grp]));
        };
        auto issue_sv = [&](uint32_t s, bool last) {
            const uint32_t vst = Lay::OFF_V + s * PA_VST;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_bf16_ts(PA_TM_S, PA_TM_Q + (2 + i) * 32 + ks * 8,
                                sdesc_sw128(base + vst + i * PA_BLK + ks * 32, 16, 1024), idesc_s, 1u);
            mma_commit(smem_u32(&bars->s_full));
            if (last) mma_commit(smem_u32(&bars->q_free));
        };
        auto issue_pv = [&](uint32_t s, bool first, bool last) {
            const uint32_t vst = Lay::OFF_V + s * PA_VST;
#pragma unroll
            for (int ks = 0; ks < PA_N / 16; ++ks)
                mma_bf16_ss(PA_TM_O, sdesc_noswz(base + Lay::OFF_P + ks * 4096, 2048, 128),
                            sdesc_sw128(base + vst + ks * 2048, PA_BLK, 1024), idesc_pv, (!first || ks > 0) ? 1u : 0u);
            mma_commit(smem_u32(&bars->vfree[s]));
            mma_commit(smem_u32(&bars->p_free));
            if (last) mma_commit(smem_u32(&bars->o_full));
        };
        using C0 = std::integral_constant<int, 0>;
        using C1 = std::integral_constant<int, 1>;
        uint32_t g = 0, e = 0;  // tiles and items (with tiles) begun
        auto wait = [&](uint64_t* bar, uint32_t parity, int where) {
            return pa_wait_one(smem_u32(bar), parity, abort, st, where);
        };
        // the tiles of an item
        auto run = [&](int n_tiles) -> bool {
            // PV of tile p; a first tile overwrites O, which the epilogue of the item
            // before has read
            auto pv = [&](uint32_t p, bool first, bool last) -> bool {
                if (!wait(&bars->p_full, p & 1, 0x2201)) return false;
                if (first && e > 0 && !wait(&bars->o_free, (e - 1) & 1, 0x2202)) return false;
                tc_fence_after();
                const uint32_t s = p % PA_NST;
                issue_pv(s, first, last);
                return true;
            };
            if (!wait(&bars->q_full, e & 1, 0x2204)) return false;
            for (int u = 0; u < n_tiles; ++u, ++g) {
                const uint32_t s = g % PA_NST;
                if (!wait(&bars->s_free, (g & 1) ^ 1, 0x2206) || !wait(&bars->kfull, g & 1, 0x2205)) return false;
                fence_proxy_async();  // the rows arrived by cp.async (P's writers fence their own)
                tc_fence_after();
                issue_sk(C0());
                if (!wait(&bars->vfull[s], (g / PA_NST) & 1, 0x2207)) return false;
                fence_proxy_async();
                issue_sk(C1());
                const bool last = u + 1 == n_tiles;
                issue_sv(s, last);
                if (u > 0 && !pv(g - 1, u == 1, false)) return false;
            }
            return pv(g - 1, n_tiles == 1, true);  // before anything of the next item is waited for
        };
        for (int64_t qi = 0; qi < nq; ++qi) {
            if (!info_wait(qi, 0x2203)) break;
            const int n_tiles = tiles_of(qi);
            info_done(qi);
            if (n_tiles == 0) continue;
            bool ok = true;
            const uint32_t g0 = g;
            if (elect_one()) ok = run(n_tiles);
            __syncwarp();
            if (!__all_sync(0xffffffffu, ok)) break;
            g = g0 + n_tiles;
            ++e;
        }
        if (*abort) {
            if (elect_one()) {
                mma_commit(smem_u32(&bars->drain));
                mbar_wait(smem_u32(&bars->drain), 0, nullptr, st, 0x2208, 1ll << 28);
            }
            __syncwarp();
        }
    } else if (warp < PA_EPI0) {
        // ================= softmax: two threads per row, 32 keys of a tile each =================
        const int quad = warp & 3, kh = warp >> 2, h = quad * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const float scale_log2 = a.scale * 1.4426950408889634f;
        const bool zero = scale_log2 == 0.f;
        const int tok_off = h / a.heads;  // this row's token of the item
        uint8_t* prow = smem + Lay::OFF_P + kh * 4 * 2048 + h * 16;
        float* xm = (float*)(smem + Lay::OFF_XM);
        uint32_t g = 0, e = 0;
        bool ok = true;
        // the first item's Q, half of its blocks a warp, while the epilogue warps read
        // its selection (staged in P's buffer and theirs; not used if the item turns out
        // empty)
        if (nq > 0) {
            const int64_t grp = item0 / a.splits;
            load_q(pa_item<DENSE>(a, grp, (int)(item0 - grp * a.splits), sel_part), quad,
                   smem + (kh == 0 ? Lay::OFF_P : Lay::OFF_EPI) + quad * 4096, kh, [] { return true; });
            if (!info_wait(0, 0x2301)) ok = false;
            else if (tiles_of(0) > 0 && lane == 0) mbar_arrive(smem_u32(&bars->q_full));
            __syncwarp();
        }
        for (int64_t qi = 0; ok && qi < nq; ++qi) {
            if (!info_wait(qi, 0x2301)) break;
            const int n_tiles = tiles_of(qi);
            // keys of the part that this row may see (dense), from this half's first
            int lim = 0;
            bool holes = false;
            if constexpr (DENSE) {
                const PaItem& it = items[qi & 1];
                lim = (int)min((int64_t)it.count, max((int64_t)0, it.pos0 + tok_off + 1 - it.lo)) - 32 * kh;
#pragma unroll
                for (int w = 0; w < 4; ++w) holes = holes || pmax[(qi & 1) * 8 + 4 + w] != 0;
                holes = __shfl_sync(0xffffffffu, holes, 0);
            }
            const uint32_t* vm = vmask + (qi & 1) * 64 + kh;
            float m_used = -INFINITY, l = 0.f;
            for (int u = 0; u < n_tiles; ++u, ++g) {
                uint32_t msk = DENSE ? low_bits(lim - u * PA_N) : vm[2 * u];  // keys that this row sees
                if (DENSE && holes) {  // and that have a page (lane i looks for key i)
                    const PaItem& it = items[qi & 1];
                    const int key = u * PA_N + 32 * kh + lane;
                    msk &= __ballot_sync(0xffffffffu, key < it.count && page_of(a.pv, it.b, it.lo + key).page >= 0);
                }
                if (!wait_warp(smem_u32(&bars->s_full), g & 1, abort, st, 0x2302)) { ok = false; break; }
                tc_fence_after();
                uint32_t x[32];
                tmem_ld32(tmem + lane_off + PA_TM_S + 32 * kh, x);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->s_free));
                if (__any_sync(0xffffffffu, msk != 0xffffffffu)) {
                    // A later token of the group may hold a NaN or an infinity, and 0 times
                    // that is NaN.  V is the row's leading columns, so its score is then
                    // not finite for any query: such masked keys' V values are set to
                    // zero.  A row that sees the key has a NaN for its probability, or a
                    // score of -inf and no weight on it.
                    if constexpr (DENSE) {
                        uint32_t odd = 0;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if ((x[i] & 0x7f800000u) == 0x7f800000u) odd |= 1u << i;
                        odd = __reduce_or_sync(0xffffffffu, odd & ~msk);
                        if (odd) {
                            // (long complete: S was computed from it)
                            if (!wait_warp(smem_u32(&bars->vfull[g % PA_NST]), (g / PA_NST) & 1, abort, st, 0x2305)) {
                                ok = false;
                                break;
                            }
                            clear_not_finite(s_v + g % PA_NST * PA_VST, 32 * kh, odd);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!((msk >> i) & 1u)) x[i] = 0xff800000u;  // -inf
                }
                float mt[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 32; ++i) mt[i & 3] = fmaxf(mt[i & 3], __uint_as_float(x[i]));
                float mx = fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3]));
                {  // with the other half's
                    float* slot = xm + (g & 1) * 256;
                    slot[kh * 128 + h] = mx;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars->xm_full[quad]));
                    if (!wait_warp(smem_u32(&bars->xm_full[quad]), g & 1, abort, st, 0x2303)) { ok = false; break; }
                    mx = fmaxf(mx, slot[(kh ^ 1) * 128 + h]);
                }
                // (no key seen: -inf, also where scale is 0)
                const float ms = mx == -INFINITY ? -INFINITY : mx * scale_log2;
                // the running maximum moves only when it grows by more than 2^8
                float alpha = 1.f;
                if (ms > m_used + 8.0f) {
                    alpha = m_used == -INFINITY ? 0.f : ex2(m_used - ms);
                    l *= alpha;
                    m_used = ms;
                }
                // the probabilities; rounding them to bf16 for the MMA is half a step
                // (2^-8) of each, their sum is kept unrounded in fp32.  A masked key is
                // -inf here, unless scale is 0 (-inf * 0): its probability is set apart.
                const float sub = m_used == -INFINITY ? 0.f : m_used;
                float rs[4] = {0.f, 0.f, 0.f, 0.f};
                uint32_t w[16];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int i = 8 * c + 2 * q;
                        float p0 = ex2(fmaf(__uint_as_float(x[i]), scale_log2, -sub));
                        float p1 = ex2(fmaf(__uint_as_float(x[i + 1]), scale_log2, -sub));
                        if (zero) {
                            p0 = ((msk >> i) & 1u) ? p0 : 0.f;
                            p1 = ((msk >> (i + 1)) & 1u) ? p1 : 0.f;
                        }
                        rs[q & 1] += p0;
                        rs[2 + (q & 1)] += p1;
                        w[4 * c + q] = pack_bf16(p0, p1);
                    }
                }
                l += (rs[0] + rs[1]) + (rs[2] + rs[3]);
                // P may be written, and O rescaled, once PV(g - 1) is complete
                if (!wait_warp(smem_u32(&bars->p_free), (g & 1) ^ 1, abort, st, 0x2304)) { ok = false; break; }
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *(uint4*)(prow + c * 2048) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                if (u > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {  // each half takes 128 of the columns
                    tc_fence_after();
                    for (int c = 0; c < 4; ++c) {
                        uint32_t r[32];
                        const uint32_t ta = tmem + lane_off + PA_TM_O + kh * 128 + c * 32;
                        tmem_ld32(ta, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
                        tmem_st32(ta, r);
                    }
                    tmem_wait_st();
                }
                fence_proxy_async();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->p_full));
            }
            if (!ok) break;
            info_done(qi);
            if (n_tiles == 0) continue;
            float* ml = (float*)(smem + Lay::OFF_ML) + (e & 1) * 384;
            if (kh == 0) ml[h] = m_used;
            ml[128 + kh * 128 + h] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->ml_full[e & 1]));
            ++e;
        }
    } else {
        // ================= Q loads and the epilogue: one thread per row =================
        const int quad = warp - PA_EPI0, h = quad * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const int tok_off = h / a.heads, head = h - tok_off * a.heads;
        const int dv0 = 256 * half;
        uint8_t* stg = smem + Lay::OFF_EPI + quad * 4096;
        // base 2; -inf: nothing attended
        auto write_lse = [&](const PaItem& it, int64_t item, float v) {
            if (half != 0) return;
            if (a.splits > 1) a.part_lse[item * 128 + h] = v;
            else if (a.lse && tok_off < it.ntok) a.lse[(it.t0 + tok_off) * a.heads + head] = v * 0.69314718055994531f;
        };
        // The item's rows of the output.  One part: O / l in bf16 and the lse.
        // Several: normalised fp32 partials and their base-2 lse, per item.
        // Rows leave through this warp's staging tile, so that a store covers
        // 64-byte pieces of 8 rows.
        auto epilogue = [&](const PaItem& it, int64_t item, uint32_t e) -> bool {
            // (a barrier for each slot of the ring: item e + 1 may finish its softmax before
            // this warp looks, item e + 2 not before this epilogue has read O)
            if (!wait_warp(smem_u32(&bars->ml_full[e & 1]), (e >> 1) & 1, abort, st, 0x2401)) return false;
            const float* ml = (const float*)(smem + Lay::OFF_ML) + (e & 1) * 384;
            const float m_used = ml[h], l = ml[128 + h] + ml[256 + h];
            const float inv = l != 0.f ? 1.0f / l : 0.f;  // a NaN sum stays a NaN row
            if (!wait_warp(smem_u32(&bars->o_full), e & 1, abort, st, 0x2402)) return false;
            tc_fence_after();
            const int64_t mine = tok_off < it.ntok
                                     ? (it.t0 + tok_off) * a.out_stride_tok + (int64_t)head * a.out_stride_head + dv0
                                     : -1;
            int64_t off[4];  // output rows 8 i + lane / 4 of this warp (-1: not a row of the item)
#pragma unroll
            for (int i = 0; i < 4; ++i) off[i] = __shfl_sync(0xffffffffu, mine, 8 * i + (lane >> 2));
            __nv_bfloat16* out = (__nv_bfloat16*)a.out;
            float* part = a.part_o + (item * 128 + quad * 32) * 512 + dv0;
            const int k4 = lane & 3;
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {  // 32 columns at a time
                uint32_t r[32];
                tmem_ld32(tmem + lane_off + PA_TM_O + c * 32, r);
                tmem_wait_ld();
                if (c == 7) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars->o_free));  // O may be overwritten now
                }
                if (a.splits > 1) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {  // 16 columns at a time
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t* x = &r[16 * q + 4 * k];
                            *(float4*)(stg + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) =
                                make_float4(__uint_as_float(x[0]) * inv, __uint_as_float(x[1]) * inv,
                                            __uint_as_float(x[2]) * inv, __uint_as_float(x[3]) * inv);
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = 8 * i + (lane >> 2);
                            *(float4*)(part + (int64_t)row * 512 + c * 32 + q * 16 + k4 * 4) =
                                *(const float4*)(stg + row * 64 + ((k4 ^ ((row >> 1) & 3)) << 4));
                        }
                        __syncwarp();
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t w[4];
#pragma unroll
                        for (int p = 0; p < 4; ++p)
                            w[p] = pack_bf16(__uint_as_float(r[8 * k + 2 * p]) * inv, __uint_as_float(r[8 * k + 2 * p + 1]) * inv);
                        *(uint4*)(stg + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = 8 * i + (lane >> 2);
                        const uint4 v = *(const uint4*)(stg + row * 64 + ((k4 ^ ((row >> 1) & 3)) << 4));
                        if (off[i] >= 0) *(uint4*)(out + off[i] + c * 32 + k4 * 8) = v;
                    }
                    __syncwarp();
                }
            }
            // (__log2f: 2^-22 absolute for l near 1, 2 ulp elsewhere; a score is off by more)
            write_lse(it, item, l != 0.f ? m_used + __log2f(l) : -INFINITY);
            return true;
        };

        // Item qi's rows, and for a selection the validity bits of its slots and the
        // last used one, one item ahead of the other warps.
        auto publish = [&](int64_t qi) -> bool {
            const uint32_t slot = (uint32_t)(qi & 1);
            const int64_t item = item0 + qi * step, grp = item / a.splits;
            const PaItem it = pa_item<DENSE>(a, grp, (int)(item - grp * a.splits), sel_part);
            // Q rows into L2 (their loads begin when the item before has issued its last S)
            if (tok_off < it.ntok) {
                const char* qr = (const char*)((const __nv_bfloat16*)a.q + (it.t0 + tok_off) * a.q_stride_tok +
                                               (int64_t)head * a.q_stride_head);
                for (int kb = 0; kb < 9; ++kb) prefetch_l2(qr + kb * 128);
            }
            if (!wait_warp(smem_u32(&bars->info_empty[slot]), (uint32_t)((qi >> 1) & 1) ^ 1u, abort, st, 0x2102)) return false;
            int m = -1, holes = 0;
            if constexpr (DENSE) {
                m = it.count - 1;
                // a part with positions that have no page: the softmax looks for them
                // (nothing in its tiles otherwise)
                if (it.count > 0) {
                    uint32_t p0, p1, o;
                    page_split(a.pv, (uint32_t)it.lo, p0, o);
                    page_split(a.pv, (uint32_t)(it.lo + it.count - 1), p1, o);
                    const int32_t* table = a.pv.table + it.b * a.pv.ld_table;
#pragma unroll 4
                    for (uint32_t p = p0 + quad * 32 + lane; p <= p1; p += 128)
                        holes |= (int64_t)p >= a.pv.ld_table || (uint32_t)__ldg(table + p) >= (uint32_t)a.pv.num_pages;
                    holes = __any_sync(0xffffffffu, holes);
                }
            } else {
                const int32_t* irow = a.idx + it.t0 * a.ld_idx + it.lo;
                int32_t v[PA_SCAN_ROUNDS];
#pragma unroll
                for (int r = 0; r < PA_SCAN_ROUNDS; ++r) {
                    const int j = (quad + 4 * r) * 32 + lane;
                    v[r] = j < it.count ? __ldg(irow + j) : -1;
                }
#pragma unroll
                for (int r = 0; r < PA_SCAN_ROUNDS; ++r) {
                    const int w = quad + 4 * r;  // 32-slot word of the part
                    bool val = v[r] >= 0;
                    if (val) m = w * 32 + lane;
                    if (val && (v[r] >= it.seqlen_k || page_of(a.pv, it.b, v[r]).page < 0)) {
                        report(st, DSA_ERR_INDEX, it.t0);
                        val = false;
                    }
                    const uint32_t bits = __ballot_sync(0xffffffffu, val);
                    if (lane == 0) vmask[slot * 64 + w] = bits;
                }
                for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            }
            if (lane == 0) {
                if (quad == 0) {
                    items[slot] = it;
                    if (!it.ok && half == 0) report(st, DSA_ERR_INDEX, it.t0);
                }
                pmax[slot * 8 + quad] = m;
                if (DENSE) pmax[slot * 8 + 4 + quad] = holes;
                mbar_arrive(smem_u32(&bars->info_full[slot]));
            }
            __syncwarp();
            return true;
        };
        uint32_t e = 0;     // items with tiles begun
        bool ok = nq == 0 || publish(0), pend = false;  // the (e - 1)-th item's epilogue is still to be done
        int64_t item_pend = 0;
        PaItem it_pend = {};
        for (int64_t qi = 0; ok && qi < nq; ++qi) {
            const int64_t item = item0 + qi * step;
            if (!info_wait(qi, 0x2403)) { ok = false; break; }
            const PaItem it = items[qi & 1];
            const int n_tiles = tiles_of(qi);
            if (n_tiles > 0 && qi > 0) {  // (the first item's Q: the softmax warps)
                // (an empty first item: its Q, unused, must have landed; later items' info
                // was published after that)
                auto wait = [&]() {
                    if (e > 0) return wait_warp(smem_u32(&bars->q_free), (e - 1) & 1, abort, st, 0x2404);
                    return qi > 1 || wait_warp(smem_u32(&bars->info_empty[0]), 0, abort, st, 0x2405);
                };
                if (!load_q(it, quad, stg, 2, wait)) { ok = false; break; }
                if (lane < 2) mbar_arrive(smem_u32(&bars->q_full));  // (for two warps of the first)
            }
            // ---- the previous item's epilogue (this item's first S overlaps it) ----
            if (pend && !epilogue(it_pend, item_pend, e - 1)) { ok = false; break; }
            pend = false;
            if (n_tiles == 0) {  // nothing to attend to: zero rows, lse -inf (a part: its lse alone)
                write_lse(it, item, -INFINITY);
                if (a.splits == 1 && tok_off < it.ntok) {
                    uint4* dst = (uint4*)((__nv_bfloat16*)a.out + (it.t0 + tok_off) * a.out_stride_tok +
                                          (int64_t)head * a.out_stride_head + dv0);
#pragma unroll 4
                    for (int i = 0; i < 32; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
                }
            } else {
                pend = true;
                it_pend = it;
                item_pend = item;
                ++e;
            }
            if (qi + 1 < nq && !publish(qi + 1)) { ok = false; break; }
        }
        if (ok && pend) epilogue(it_pend, item_pend, e - 1);
        // (groups are cut from the sequences: a token of none falls in no group)
        if (DENSE && a.group > 1 && blockIdx.x == 0 && threadIdx.x == 32 * PA_EPI0)
            report_no_sequence(a.sv, 0, a.total_q, st);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == PA_MMA) tmem_dealloc(tmem, 512);
}

// Joins the parts of every item's rows: weights 2^(lse_p - max), one block a
// row (token and head).  Bound by reading the partial rows, which are in L2.
__global__ void __launch_bounds__(128) attn_paged_combine_kernel(const PagedAttnArgs a, int dense) {
    const int64_t grp = blockIdx.x / (unsigned)(a.group * a.heads);
    const int row = (int)(blockIdx.x - grp * (a.group * a.heads));
    PaItem it = dense ? pa_item<true>(a, grp, 0, 0) : pa_item<false>(a, grp, 0, a.k_sel);
    const int tok = row / a.heads, head = row - tok * a.heads;
    const int64_t t = it.t0 + tok;
    const float* pl = a.part_lse + grp * a.splits * 128 + row;
    grid_wait();
    if (tok >= it.ntok) return;
    // lane p of every warp holds the weights of parts p and p + 32
    const int lane = (int)lane_id();
    float m = -INFINITY, z[2], w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        z[i] = lane + 32 * i < a.splits ? pl[(lane + 32 * i) * 128] : -INFINITY;
        m = fmaxf(m, z[i]);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
#pragma unroll
    for (int i = 0; i < 2; ++i) w[i] = z[i] == -INFINITY ? 0.f : ex2(z[i] - m);  // NaN stays NaN
    const float* po = a.part_o + (grp * a.splits * 128 + row) * 512 + threadIdx.x * 4;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int p = 0; p < a.splits; ++p) {
        const float wp = __shfl_sync(0xffffffffu, p < 32 ? w[0] : w[1], p & 31);
        if (wp == 0.f) continue;  // an empty part: its rows were not written
        const float4 v = *(const float4*)(po + (int64_t)p * 128 * 512);
        l += wp;
        o.x = fmaf(wp, v.x, o.x), o.y = fmaf(wp, v.y, o.y), o.z = fmaf(wp, v.z, o.z), o.w = fmaf(wp, v.w, o.w);
    }
    const float inv = l != 0.f ? 1.0f / l : 0.f;
    *(uint2*)((__nv_bfloat16*)a.out + t * a.out_stride_tok + (int64_t)head * a.out_stride_head + threadIdx.x * 4) =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (a.lse && threadIdx.x == 0)
        a.lse[t * a.heads + head] = l != 0.f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}

template <bool DENSE>
static bool pa_launch(const PagedAttnArgs& a, cudaStream_t s) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return false;
    if (cudaFuncSetAttribute((const void*)attn_paged_kernel<DENSE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             PaLayout::SMEM) != cudaSuccess)
        return false;
    const int64_t units = 2 * a.groups * a.splits, most = sms & ~1;
    attn_paged_kernel<DENSE><<<(unsigned)(units < most ? units : most), PA_THREADS, PaLayout::SMEM, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return false;
    if (a.splits == 1) return true;
    return launch_after(attn_paged_combine_kernel, dim3((unsigned)(a.groups * a.group * a.heads)), dim3(128), s, a,
                        DENSE ? 1 : 0);
}

bool launch_paged_attn_tc(const PagedAttnArgs& a, cudaStream_t s) {
    if (a.groups <= 0) return true;
    return a.idx ? pa_launch<false>(a, s) : pa_launch<true>(a, s);
}

}  // namespace dsa
