// attn_paged.cu -- attention of a chunk of new tokens over the paged KV rows
// on the 5th-generation tensor cores (BF16 in, fp32 accumulate): MQA in the MLA
// layout (up to 128 heads share one KV row of 512 latent + 64 rope columns, V is
// the latent part), dense causal or over each query's selected positions.
//
// The tile pipeline is that of attn_tc.cu (a CTA pair splits the contraction
// and the output columns, exchanging partial scores and probabilities); what
// differs:
//   * Work items.  An item is a group of query rows and a part of their keys.  A
//     selection's item is one query; a dense item is up to 128 / heads
//     consecutive tokens of a sequence, so that a rank that holds few heads
//     still fills the 128 rows of the MMA (row r: token r / heads, head
//     r % heads; each row masks its own causal limit).
//   * Parts.  With fewer items than CTA pairs the keys of an item are split;
//     the parts leave normalised fp32 rows and their log-sum-exp in the
//     workspace and attn_paged_combine_kernel joins them.
//   * Rows through the page table, looked up one tile ahead.  Slots that hold no row
//     are filled with zeros, so a masked probability never meets a stray NaN.
//   * The running maximum is a true one where it moves (see stage B), so scores
//     whose two partial sums are large and of opposite sign lose nothing.
#include "attn_pair.cuh"
#include "rows.cuh"

namespace dsa {

constexpr int PA_NST = 3, PA_NPB = 3;  // K/V stages and P tiles, as the packed kernel

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

struct PaLayout : AtLayout<PA_NST, false, PA_NPB, 1> {
    using Base = AtLayout<PA_NST, false, PA_NPB, 1>;
    static_assert(Base::EPI_STAGE && Base::EPI_COLS == 32, "the epilogue stages 32 columns of 32 rows");
    static constexpr uint32_t OFF_ITEM = Base::SMEM;        // [2] PaItem
    static constexpr uint32_t OFF_TMX = OFF_ITEM + 128;     // [2][128] the peer's true maxima
    static constexpr uint32_t SMEM = OFF_TMX + 1024;
};
static_assert(2 * sizeof(PaItem) <= 128, "item ring");
static_assert(PaLayout::SMEM <= 232448, "shared memory budget");

struct PaBars : AtBars {
    uint64_t tm_full[8];  // [quadrant][2]: the peer's true maxima (bytes)
};
static_assert(sizeof(PaBars) <= 512, "barrier block");

// 16 bytes global -> shared, or zeros (the source is then not read)
DSA_DEV void cp_async16_zfill(uint32_t dst, const void* src, bool have) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"((uint64_t)src), "r"(have ? 16 : 0)
                 : "memory");
}

DSA_DEV uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

DSA_DEV int32_t page_slot(const PageView& pv, int32_t s) {
    return pv.shift >= 0 ? s & (pv.page_size - 1) : (int32_t)((uint32_t)s % (uint32_t)pv.page_size);
}

// First item slot of sequence b's groups: groups of R tokens never cross a
// sequence; ceil(l / R) of them fit between floor(cu[b] / R) + b and the next.
DSA_DEV int64_t pa_first_group(int64_t cu, int b, int R) { return R == 1 ? cu : cu / R + b; }

template <bool DENSE>
DSA_DEV PaItem pa_item(const PagedAttnArgs& a, int64_t grp, int part, int sel_part) {
    PaItem it = {};
    int b;
    if (!DENSE || a.group == 1) {
        const RowInfo ri = row_info(a.sv, grp);
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
        const int64_t per = ((n + AT_N - 1) / AT_N + a.splits - 1) / a.splits * AT_N;
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
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(AT_THREADS, 1)
    attn_paged_kernel(const __grid_constant__ PagedAttnArgs a) {
    static_assert(AT_SOFT0 % 4 == 0 && AT_PRODUCERS < AT_SOFT0, "warp roles");
    constexpr int NST = PA_NST, NPB = PA_NPB;
    using Lay = PaLayout;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    PaBars* bars = (PaBars*)(smem + Lay::OFF_BAR);
    uint32_t* vmask = (uint32_t*)(smem + Lay::OFF_VM);
    int* pmax = (int*)(smem + Lay::OFF_INFO);  // [2][8]
    int* ntab = pmax + 16;                      // [AT_NTAB]
    PaItem* items = (PaItem*)(smem + Lay::OFF_ITEM);  // [2]
    if ((uintptr_t)smem != (uintptr_t)smem_raw) {  // the layout needs a 1024-byte aligned base
        if (threadIdx.x == 0) report(a.st, DSA_ERR_UNSUPPORTED, -3);
        return;
    }
    const uint32_t warp = warp_id(), lane = lane_id();
    const uint32_t rank = cluster_ctarank(), peer = rank ^ 1u;
    StatusHdr* st = a.st;
    volatile int* abort = &bars->abort;

    // work items of this pair: pair + i * npairs
    const int64_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1, n_items = a.groups * a.splits;
    const int64_t nq = pair < n_items ? (n_items - pair + npairs - 1) / npairs : 0;
    const float scale_log2 = a.scale * 1.4426950408889634f;
    // tiles of a selection's part (dense: from the item's own length)
    const int sel_part = DENSE ? 0 : ((a.k_sel + AT_N - 1) / AT_N + a.splits - 1) / a.splits * AT_N;
    const int nb = rank ? 5 : 4;      // 64-column blocks of K held here
    const int col0 = rank ? 256 : 0;  // first K column
    const int dv0 = rank ? 256 : 0;   // first output column

    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(smem_u32(&bars->full[i]), AT_PRODUCERS * 32);
            mbar_init(smem_u32(&bars->empty[i]), 1);
        }
        mbar_init(smem_u32(&bars->s_full), 2);   // one commit per issuer
        mbar_init(smem_u32(&bars->s_empty), 8);  // 4 A + 4 B warps read every S tile
        mbar_init(smem_u32(&bars->s_go), 1);
        mbar_init(smem_u32(&bars->drain2), 1);
        for (int i = 0; i < 3; ++i) {
            mbar_init(smem_u32(&bars->p_full[i]), 4);   // (only NPB of them are used)
            mbar_init(smem_u32(&bars->p_free[i]), 2);
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(smem_u32(&bars->tm_full[i]), 1);
            mbar_arrive_expect_tx(smem_u32(&bars->tm_full[i]), 128);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars->sx_full[i]), 1);
            mbar_init(smem_u32(&bars->sx_free[i]), 4);
            mbar_init(smem_u32(&bars->info_full[i]), AT_PRODUCERS);
            mbar_init(smem_u32(&bars->info_empty[i]), 9);
        }
        mbar_init(smem_u32(&bars->q_full), 4);
        mbar_init(smem_u32(&bars->o_full), 1);
        mbar_init(smem_u32(&bars->o_free), 8);
        mbar_init(smem_u32(&bars->lx_full), 1);
        mbar_init(smem_u32(&bars->lx_loc), 4);
        mbar_init(smem_u32(&bars->drain), 1);
        // byte counts of the first phase of every peer-filled barrier; each
        // later phase is armed once the one before it has completed
        for (int i = 0; i < NPB; ++i) mbar_expect_tx(smem_u32(&bars->p_full[i]), AT_PX_BYTES);
        mbar_arrive_expect_tx(smem_u32(&bars->sx_full[0]), AT_SX_BYTES);
        mbar_arrive_expect_tx(smem_u32(&bars->lx_full), AT_LX_BYTES);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == AT_MMA_WARP) tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tc_fence_before();
    cluster_sync();  // barriers of both CTAs initialised and armed
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    const uint32_t s_stage0 = smem_u32(smem);
    const uint32_t s_p0 = smem_u32(smem + Lay::OFF_P);
    const uint32_t s_qr = smem_u32(smem + Lay::OFF_QR);
    // Half hf of the S tile of stage s: K-blocks 2hf, 2hf+1 (Q from TMEM) and, on
    // rank 1, K-steps 2hf, 2hf+1 of the rope block (Q from shared memory), into
    // accumulator hf.  Issued by one thread.
    auto s_half = [&](int hf, uint32_t s) {
        constexpr uint32_t idesc_s = idesc_make(1, 1, false, 128, AT_N);
        const uint32_t kst = s_stage0 + s * Lay::STAGE;
        const uint32_t d = tmem + TM_S + 64 * hf;
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
            const int kb = 2 * hf + k2;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_bf16_ts(d, tmem + TM_Q + kb * 32 + ks * 8, sdesc_sw128(kst + kb * AT_BLK + ks * 32, 16, 1024), idesc_s,
                            (k2 | ks) ? 1u : 0u);
        }
        if (nb == 5)
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
                const int ks = 2 * hf + k2;
                mma_bf16_ss(d, sdesc_sw128(s_qr + ks * 32, 16, 1024), sdesc_sw128(kst + 4 * AT_BLK + ks * 32, 16, 1024),
                            idesc_s, 1u);
            }
    };
    if (warp < AT_PRODUCERS) {
        // ================= gather producers (6 warps) =================
        if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(AT_REGS_WG0));
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(AT_REGS_WG1));
        // 16 groups of 4 keys per tile; warp w takes groups w, w+7, w+14
        const int sub = (int)(lane >> 3), chunk = (int)(lane & 7);
        const int ngrp = (16 - (int)warp + AT_PRODUCERS - 1) / AT_PRODUCERS;
        uint32_t g = 0;  // tile of the pair's whole sequence
        bool ok = true;
        const __nv_bfloat16* pool = (const __nv_bfloat16*)a.k + col0 + chunk * 8;
        for (int64_t qi = 0; ok && qi < nq; ++qi) {
            const uint32_t slot = (uint32_t)(qi & 1);
            const int64_t item = pair + qi * npairs, grp = item / a.splits;
            const PaItem it = pa_item<DENSE>(a, grp, (int)(item - grp * a.splits), sel_part);
            const int32_t* irow = DENSE ? nullptr : a.idx + it.t0 * a.ld_idx + it.lo;
            const int count = it.count;  // keys (dense) or slots of this item's part
            // ---- item info: rows, and for a selection the validity bits of its
            // slots and the last used one ----
            if (!wait_warp(smem_u32(&bars->info_empty[slot]), (uint32_t)((qi >> 1) & 1) ^ 1u, abort, st, 0x2102)) {
                ok = false;
                break;
            }
            int m = -1;
            if constexpr (DENSE) {
                m = count - 1;
            } else {
                int32_t v[AT_SCAN_ROUNDS];
#pragma unroll
                for (int r = 0; r < AT_SCAN_ROUNDS; ++r) {
                    const int j = ((int)warp + AT_PRODUCERS * r) * 32 + (int)lane;
                    v[r] = j < count ? __ldg(irow + j) : -1;
                }
#pragma unroll
                for (int r = 0; r < AT_SCAN_ROUNDS; ++r) {
                    const int w = (int)warp + AT_PRODUCERS * r;  // 32-slot word of the part
                    bool val = v[r] >= 0;
                    if (val && v[r] >= it.seqlen_k) {
                        report(st, DSA_ERR_INDEX, it.t0);
                        val = false;
                    }
                    if (val) {
                        m = w * 32 + (int)lane;
                        if (page_of(a.pv, it.b, v[r]).page < 0) {
                            report(st, DSA_ERR_INDEX, it.t0);
                            val = false;
                        }
                    }
                    const uint32_t bits = __ballot_sync(0xffffffffu, val);
                    if (lane == 0 && w < 64) vmask[slot * 64 + w] = bits;
                }
                for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            }
            if (lane == 0) {
                if (warp == 0) {
                    items[slot] = it;
                    if (!it.ok && rank == 0) report(st, DSA_ERR_INDEX, it.t0);
                }
                pmax[slot * 8 + warp] = m;
                mbar_arrive(smem_u32(&bars->info_full[slot]));
            }
            if (!wait_warp(smem_u32(&bars->info_full[slot]), (uint32_t)((qi >> 1) & 1), abort, st, 0x2103)) {
                ok = false;
                break;
            }
            int mx = -1;
#pragma unroll
            for (int w = 0; w < AT_PRODUCERS; ++w) mx = max(mx, pmax[slot * 8 + w]);
            const int n_tiles = (mx + AT_N) / AT_N;
            // ---- pull the next item's Q rows (and its index row) into L2 while this
            // item's tiles run ----
            if (qi + 1 < nq) {
                const int64_t gn = (item + npairs) / a.splits;
                const PaItem nx = pa_item<DENSE>(a, gn, 0, sel_part);
                if (!DENSE && warp == 0) {
                    const char* ir = (const char*)(a.idx + nx.t0 * a.ld_idx);
                    if (nx.ok)
                        for (int off = (int)lane * 128; off < a.k_sel * 4; off += 32 * 128) prefetch_l2(ir + off);
                } else if (warp >= 1 && warp <= 4) {
                    const int row = (int)(warp - 1) * 32 + (int)lane;
                    const int tk = row / a.heads;
                    if (tk < nx.ntok) {
                        const char* qr = (const char*)((const __nv_bfloat16*)a.q + (nx.t0 + tk) * a.q_stride_tok +
                                                       (int64_t)(row - tk * a.heads) * a.q_stride_head + col0);
                        for (int kb = 0; kb < nb; ++kb) prefetch_l2(qr + kb * 128);
                    }
                }
            }
            // ---- the item's tiles: position and page of this lane's rows, one tile ahead ----
            int32_t nv[3] = {-1, -1, -1}, np[3] = {-1, -1, -1};
            auto look_up = [&](int j) {
#pragma unroll
                for (int gi = 0; gi < 3; ++gi) {
                    const int sj = j * AT_N + 4 * ((int)warp + AT_PRODUCERS * gi) + sub;
                    nv[gi] = -1;
                    if (gi < ngrp && sj < count) nv[gi] = DENSE ? it.lo + sj : __ldg(irow + sj);
                    if (!DENSE && nv[gi] >= it.seqlen_k) nv[gi] = -1;
                }
#pragma unroll
                for (int gi = 0; gi < 3; ++gi) np[gi] = nv[gi] >= 0 ? (int32_t)page_of(a.pv, it.b, nv[gi]).page : -1;
            };
            if (n_tiles > 0) look_up(0);
            for (int j = 0; j < n_tiles; ++j, ++g) {
                const uint32_t s = g % NST;
                int32_t cv[3], cp[3];
#pragma unroll
                for (int gi = 0; gi < 3; ++gi) cv[gi] = nv[gi], cp[gi] = np[gi];
                if (j + 1 < n_tiles) look_up(j + 1);
                if (!wait_warp(smem_u32(&bars->empty[s]), ((g / NST) & 1) ^ 1, abort, st, 0x2101)) {
                    ok = false;
                    break;
                }
                const uint32_t kst = s_stage0 + s * Lay::STAGE;
#pragma unroll
                for (int gi = 0; gi < 3; ++gi) {
                    if (gi >= ngrp) break;
                    // a slot that holds no row is filled with zeros, so that a masked
                    // probability of zero never meets a stray NaN or infinity
                    const bool have = cp[gi] >= 0;
                    if (DENSE && cv[gi] >= 0 && !have) report(st, DSA_ERR_INDEX, it.t0);
                    const int32_t in = have ? page_slot(a.pv, cv[gi]) : 0;
                    const int key = 4 * ((int)warp + AT_PRODUCERS * gi) + sub;  // key of the tile
                    const __nv_bfloat16* src = have ? pool + (int64_t)cp[gi] * a.k_page_stride + (int64_t)in * a.k_stride : pool;
                    const uint32_t dst = kst + swz(key, chunk);
                    for (int kb = 0; kb < nb; ++kb) cp_async16_zfill(dst + kb * AT_BLK, have ? src + kb * 64 : src, have);
                }
                cp_async_arrive(smem_u32(&bars->full[s]));
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == AT_MMA_WARP) {
        // ================= MMA issuer =================
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(AT_REGS_WG1));
        constexpr uint32_t idesc_pv = idesc_make(1, 1, true, 128, 256);
        // Two cursors over the pair's tile sequence.  S cursor: query qs (ns
        // tiles once its info is read, else -1), tile js, sequence tile gs,
        // nqs queries with tiles begun.  PV cursor: query-with-tiles nqu, tile
        // ju, sequence tile gu; tile counts of begun queries are kept in ntab.
        int64_t qs = 0;
        int js = 0, ns = -1, ju = 0;
        uint32_t gs = 0, nqs = 0, gu = 0, nqu = 0;
        bool ok = true;
        long long idle0 = clock64();
        while (ok && (qs < nq || nqu < nqs)) {
            bool done = false;
            // ---- PV cursor (S(gu) issued, so its query has begun) ----
            if (gu < gs) {
                const int nu = ntab[nqu % AT_NTAB];
                const uint32_t b = gu % NPB;
                bool rdy = mbar_probe(smem_u32(&bars->p_full[b]), (gu / NPB) & 1);
                if (ju == 0 && nqu > 0) rdy = rdy && mbar_probe(smem_u32(&bars->o_free), (nqu - 1) & 1);
                if (__all_sync(0xffffffffu, rdy)) {
                    tc_fence_after();
                    if (lane == 0) {
                        mbar_expect_tx(smem_u32(&bars->p_full[b]), AT_PX_BYTES);  // its next phase
                        const uint32_t vb = s_stage0 + (gu % NST) * Lay::STAGE;
                        const uint32_t pb = s_p0 + b * AT_TILE128;
#pragma unroll
                        for (int ks = 0; ks < AT_N / 16; ++ks)
                            mma_bf16_ss(tmem + TM_O, sdesc_noswz(pb + ks * 4096, 2048, 128),
                                        sdesc_sw128(vb + ks * 2048, AT_BLK, 1024), idesc_pv, (ju > 0 || ks > 0) ? 1u : 0u);
                        mma_commit(smem_u32(&bars->empty[gu % NST]));
                        mma_commit_mc(smem_u32(&bars->p_free[b]), (uint16_t)3);
                        if (ju + 1 == nu) mma_commit(smem_u32(&bars->o_full));
                    }
                    __syncwarp();
                    ++gu;
                    if (++ju == nu) {
                        ju = 0;
                        ++nqu;
                    }
                    done = true;
                }
            }
            // ---- S cursor ----
            if (!done && qs < nq) {
                if (ns < 0) {
                    const uint32_t slot = (uint32_t)(qs & 1);
                    if (__all_sync(0xffffffffu, mbar_probe(smem_u32(&bars->info_full[slot]), (uint32_t)((qs >> 1) & 1)))) {
                        int mx = -1;
#pragma unroll
                        for (int w = 0; w < AT_PRODUCERS; ++w) mx = max(mx, pmax[slot * 8 + w]);
                        ns = (mx + AT_N) / AT_N;
                        if (lane == 0) {
                            if (ns > 0) ntab[nqs % AT_NTAB] = ns;
                            mbar_arrive(smem_u32(&bars->info_empty[slot]));
                        }
                        __syncwarp();
                        if (ns == 0) {
                            ns = -1;
                            ++qs;
                        }
                        done = true;
                    }
                } else {
                    const uint32_t s = gs % NST;
                    bool rdy = mbar_probe(smem_u32(&bars->full[s]), (gs / NST) & 1) &&
                               mbar_probe(smem_u32(&bars->s_empty), (gs & 1) ^ 1);
                    if (js == 0) rdy = rdy && mbar_probe(smem_u32(&bars->q_full), nqs & 1);
                    if (__all_sync(0xffffffffu, rdy)) {
                        fence_proxy_async();
                        tc_fence_after();
                        if (lane == 0) {
                            // first half of S: blocks 0, 1 (+ rope K-steps 0, 1); the
                            // second issuer adds blocks 2, 3 (+ rope 2, 3) into its own
                            // accumulator
                            bars->go[gs & 1] = (int)s;
                            mbar_arrive(smem_u32(&bars->s_go));
                            s_half(0, s);
                            mma_commit(smem_u32(&bars->s_full));
                        }
                        __syncwarp();
                        ++gs;
                        if (++js == ns) {
                            js = 0;
                            ns = -1;
                            ++qs;
                            ++nqs;
                        }
                        done = true;
                    }
                }
            }
            if (done) {
                idle0 = clock64();
            } else {
                const long long el = clock64() - idle0;
                bool give_up = *abort != 0;
                if (!give_up && el > (1ll << 20) && *(volatile int*)&st->code == DSA_ERR_TIMEOUT) give_up = true;
                if (!give_up && el > kWaitBudget) {
                    report(st, DSA_ERR_TIMEOUT, 0x2203);
                    give_up = true;
                }
                if (__any_sync(0xffffffffu, give_up)) {
                    *abort = 1;
                    ok = false;
                }
            }
        }
        if (ok && lane == 0) {  // no more S tiles
            bars->go[gs & 1] = -1;
            mbar_arrive(smem_u32(&bars->s_go));
        }
        if (*abort && lane == 0) {
            mma_commit(smem_u32(&bars->drain));
            mbar_wait(smem_u32(&bars->drain), 0, nullptr, st, 0x2205, 1ll << 28);
        }
    } else if (warp == AT_MMA2_WARP) {
        // ================= second S issuer =================
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(AT_REGS_WG1));
        for (uint32_t g = 0;; ++g) {
            if (!wait_warp(smem_u32(&bars->s_go), g & 1, abort, st, 0x2401)) break;
            const int s = *(volatile int*)&bars->go[g & 1];
            if (s < 0) break;
            fence_proxy_async();
            tc_fence_after();
            if (lane == 0) {
                s_half(1, (uint32_t)s);
                mma_commit(smem_u32(&bars->s_full));
            }
            __syncwarp();
        }
        if (*abort && lane == 0) {
            mma_commit(smem_u32(&bars->drain2));
            mbar_wait(smem_u32(&bars->drain2), 0, nullptr, st, 0x2405, 1ll << 28);
        }
    } else {
        // ================= softmax / exchange / epilogue (8 warps) =================
        // Stage-specialised: warps 8..11 ("A", one per TMEM lane quadrant) read
        // each S tile, form the row's partial maximum and send the peer's 32
        // partial columns; warps 12..15 ("B") read their own 32 columns of the
        // same tile, combine them with the peer's partials, form the
        // probabilities and write P.  Both groups run every tile concurrently.
        // Per query: load Q (after the previous query's last S), finish the
        // previous query (row sums, O / l), then the tiles.
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(AT_REGS_SOFT));
        const uint32_t quad = warp & 3;
        const bool is_b = warp >= AT_SOFT0 + 4;
        const int h = (int)(quad * 32 + lane);
        const uint32_t lane_off = (quad * 32) << 16;
        const int kh = (int)rank;  // this CTA's key half of every tile
        uint8_t* sx = smem + Lay::OFF_SX;
        const int tok_off = h / a.heads, head = h - tok_off * a.heads;  // this row's token of the item, and head
        const float* pmx = (const float*)(smem + Lay::OFF_PM);
        float* tmx = (float*)(smem + Lay::OFF_TMX);  // [2][128] the peer's true maxima
        const uint32_t peer_tmx = mapa(smem_u32(tmx), peer);
        const uint32_t peer_tm_full0 = mapa(smem_u32(&bars->tm_full[0]), peer);
        uint32_t n_tm = 0;  // exchanges of true maxima so far
        float* lx = (float*)(smem + Lay::OFF_LX);
        const float* lxr = (const float*)(smem + Lay::OFF_LXR);
        const uint32_t peer_sx = mapa(smem_u32(sx), peer);
        const uint32_t peer_pm = mapa(smem_u32(smem + Lay::OFF_PM), peer);
        const uint32_t peer_lxr = mapa(smem_u32(smem + Lay::OFF_LXR), peer);
        const uint32_t peer_p = mapa(s_p0, peer);
        const uint32_t peer_sx_full0 = mapa(smem_u32(&bars->sx_full[0]), peer);
        const uint32_t peer_sx_free0 = mapa(smem_u32(&bars->sx_free[0]), peer);
        const uint32_t peer_p_full0 = mapa(smem_u32(&bars->p_full[0]), peer);
        const uint32_t peer_lx_full = mapa(smem_u32(&bars->lx_full), peer);
        const uint32_t my_sx_full0 = smem_u32(&bars->sx_full[0]), my_sx_free0 = smem_u32(&bars->sx_free[0]);
        const uint32_t my_p_full0 = smem_u32(&bars->p_full[0]), my_p_free0 = smem_u32(&bars->p_free[0]);
        const bool arm_thread = threadIdx.x == (AT_SOFT0 + 4) * 32;
        const int ocol = is_b ? 0 : 128;  // this warp's 128 of the CTA's 256 output columns

        // The item's rows of the output.  One part: O / l in bf16 and the lse.
        // Several: normalised fp32 partials and their base-2 lse, per item.
        // Rows leave through this warp's staging tile, so that a store covers
        // 64-byte pieces of 8 rows.
        uint8_t* stg = smem + Lay::OFF_EPI + (warp - AT_SOFT0) * Lay::EPI_WARP_BYTES;
        auto write_lse = [&](const PaItem& it, int64_t item, float v) {  // base 2; -inf: nothing attended
            if (rank != 0 || !is_b) return;
            if (a.splits > 1) a.part_lse[item * 128 + h] = v;
            else if (a.lse && tok_off < it.ntok) a.lse[(it.t0 + tok_off) * a.heads + head] = v * 0.69314718055994531f;
        };
        // element offsets in the output of the rows 8 i + lane / 4 of this warp
        // (-1: not a row of the item)
        auto out_rows = [&](const PaItem& it, int64_t (&off)[4]) {
            const int64_t mine = tok_off < it.ntok
                                     ? (it.t0 + tok_off) * a.out_stride_tok + (int64_t)head * a.out_stride_head + dv0 + ocol
                                     : -1;
#pragma unroll
            for (int i = 0; i < 4; ++i) off[i] = __shfl_sync(0xffffffffu, mine, 8 * i + (int)(lane >> 2));
        };
        auto epilogue = [&](const PaItem& it, int64_t item, uint32_t e, float m_used, float l) -> bool {
            float l_tot = 0.f;
            if (is_b) {
                // the peer's buffer is free: it read its previous sums before its
                // A warps sent the partials of this item's tiles
                st_async_b32(peer_lxr + h * 4, __float_as_uint(l), peer_lx_full);
                if (!wait_warp(smem_u32(&bars->lx_full), e & 1, abort, st, 0x2308)) return false;
                l_tot = l + lxr[h];
                if (arm_thread) mbar_arrive_expect_tx(smem_u32(&bars->lx_full), AT_LX_BYTES);  // its next phase
                lx[h] = l_tot;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->lx_loc));
            } else {
                if (!wait_warp(smem_u32(&bars->lx_loc), e & 1, abort, st, 0x2306)) return false;
                l_tot = lx[h];
            }
            if (!wait_warp(smem_u32(&bars->o_full), e & 1, abort, st, 0x2309)) return false;
            tc_fence_after();
            const float inv = l_tot != 0.f ? 1.0f / l_tot : 0.f;  // a NaN sum stays a NaN row
            uint32_t r[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tmem + lane_off + TM_O + ocol + c * 32, r[c]);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->o_free));  // O may be overwritten now
            write_lse(it, item, l_tot != 0.f ? m_used + __log2f(l_tot) : -INFINITY);
            if (a.splits > 1) {
                float* base = a.part_o + (item * 128 + quad * 32) * 512 + dv0 + ocol;
#pragma unroll
                for (int qc = 0; qc < 8; ++qc) {  // 16 columns at a time
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t* x = &r[qc >> 1][16 * (qc & 1) + 4 * k];
                        *(float4*)(stg + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) =
                            make_float4(__uint_as_float(x[0]) * inv, __uint_as_float(x[1]) * inv,
                                        __uint_as_float(x[2]) * inv, __uint_as_float(x[3]) * inv);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = 8 * i + (int)(lane >> 2), k = (int)(lane & 3);
                        *(float4*)(base + (int64_t)row * 512 + qc * 16 + k * 4) =
                            *(const float4*)(stg + row * 64 + ((k ^ ((row >> 1) & 3)) << 4));
                    }
                    __syncwarp();
                }
                return true;
            }
            int64_t off[4];
            out_rows(it, off);
            __nv_bfloat16* out = (__nv_bfloat16*)a.out;
#pragma unroll
            for (int qc = 0; qc < 4; ++qc) {  // 32 columns at a time
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t w[4];
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        w[p] = pack_bf16(__uint_as_float(r[qc][8 * k + 2 * p]) * inv,
                                         __uint_as_float(r[qc][8 * k + 2 * p + 1]) * inv);
                    *(uint4*)(stg + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 8 * i + (int)(lane >> 2), k = (int)(lane & 3);
                    const uint4 v = *(const uint4*)(stg + row * 64 + ((k ^ ((row >> 1) & 3)) << 4));
                    if (off[i] >= 0) *(uint4*)(out + off[i] + qc * 32 + k * 8) = v;
                }
                __syncwarp();
            }
            return true;
        };

        uint32_t g = 0;    // tile of the pair's whole sequence
        uint32_t nqt = 0;  // items with tiles begun
        bool ok = true;
        bool pend = false;  // an item's epilogue is still to be done
        int64_t item_pend = 0;
        PaItem it_pend = {};
        float m_pend = -INFINITY, l_pend = 0.f;
        for (int64_t qi = 0; ok && qi < nq; ++qi) {
            const int64_t item = pair + qi * npairs;
            const uint32_t slot = (uint32_t)(qi & 1);
            if (!wait_warp(smem_u32(&bars->info_full[slot]), (uint32_t)((qi >> 1) & 1), abort, st, 0x2310)) {
                ok = false;
                break;
            }
            const PaItem it = items[slot];
            int mx = -1;
#pragma unroll
            for (int w = 0; w < AT_PRODUCERS; ++w) mx = max(mx, pmax[slot * 8 + w]);
            const int n_tiles = (mx + AT_N) / AT_N;
            if (n_tiles == 0) {  // nothing to attend to: zero rows, lse -inf (a part: its lse alone)
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->info_empty[slot]));
                write_lse(it, item, -INFINITY);
                if (a.splits == 1 && tok_off < it.ntok) {
                    uint4* dst = (uint4*)((__nv_bfloat16*)a.out + (it.t0 + tok_off) * a.out_stride_tok +
                                          (int64_t)head * a.out_stride_head + dv0 + ocol);
#pragma unroll
                    for (int i = 0; i < 16; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
                }
                continue;
            }
            // ---- Q of this item -> TMEM (A operand of S = Q K^T), by the A warps,
            // which finish an item's tiles first; every S of the earlier items has
            // completed (this warp saw its s_full).  Rows past the item are zero. ----
            if (!is_b) {
                const bool row_ok = tok_off < it.ntok;
                const __nv_bfloat16* qrow = (const __nv_bfloat16*)a.q +
                                            (row_ok ? (it.t0 + tok_off) * a.q_stride_tok + (int64_t)head * a.q_stride_head : 0) +
                                            col0;
                uint4 qreg[5][8];
#pragma unroll
                for (int kb = 0; kb < 5; ++kb) {
                    if (kb < nb) {
                        const uint4* src = (const uint4*)(qrow + kb * 64);
#pragma unroll
                        for (int j = 0; j < 8; ++j) qreg[kb][j] = row_ok ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
                    }
                }
#pragma unroll
                for (int kb = 0; kb < 5; ++kb) {
                    if (kb >= nb) continue;
                    uint32_t r[32];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        r[4 * j] = qreg[kb][j].x;
                        r[4 * j + 1] = qreg[kb][j].y;
                        r[4 * j + 2] = qreg[kb][j].z;
                        r[4 * j + 3] = qreg[kb][j].w;
                    }
                    if (kb < 4) {
                        tmem_st32(tmem + lane_off + TM_Q + kb * 32, r);
                    } else {
                        uint8_t* qr = smem + Lay::OFF_QR;
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            *(uint4*)(qr + swz(h, c)) = make_uint4(r[4 * c], r[4 * c + 1], r[4 * c + 2], r[4 * c + 3]);
                    }
                }
                tmem_wait_st();
                fence_proxy_async();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->q_full));
            }
            // ---- the previous item's epilogue (this item's first S overlap it) ----
            if (pend) {
                if (!epilogue(it_pend, item_pend, nqt - 1, m_pend, l_pend)) {
                    ok = false;
                    break;
                }
                pend = false;
            }
            // keys of the part that this row may see (dense)
            const int lim = DENSE ? (int)min((int64_t)it.count, max((int64_t)0, it.pos0 + tok_off + 1 - it.lo)) : 0;
            float m_used = -INFINITY, l = 0.f;
            for (int u = 0; ok && u < n_tiles; ++u, ++g) {
                constexpr uint32_t xb = 0;
                const uint32_t xph = g & 1;  // phase of the partial-score buffer
                uint32_t mlo, mhi;           // keys of the tile that this row sees
                if constexpr (DENSE) {
                    const int n = min(max(lim - u * AT_N, 0), AT_N);
                    mlo = low_bits(n);
                    mhi = low_bits(n - 32);
                } else {
                    mlo = vmask[slot * 64 + 2 * u];
                    mhi = vmask[slot * 64 + 2 * u + 1];
                }
                if (!wait_warp(smem_u32(&bars->s_full), g & 1, abort, st, 0x2301)) { ok = false; break; }
                tc_fence_after();
                // this CTA's partial S = accumulator 0 + accumulator 1, both key
                // halves read in one TMEM round trip; stage A sends the peer's
                // half on before it forms the partial maximum
                const uint32_t ta = tmem + lane_off + TM_S;
                const int ph_ = kh ^ 1, oh = kh;  // key halves: the peer's, this CTA's
                uint32_t rp[32], ro[32], xo[32];
                {
                    uint32_t x[32];
                    tmem_ld32(ta + 32 * ph_, rp);
                    tmem_ld32(ta + 64 + 32 * ph_, x);
                    tmem_ld32(ta + 32 * oh, ro);
                    tmem_ld32(ta + 64 + 32 * oh, xo);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) rp[i] = __float_as_uint(__uint_as_float(rp[i]) + __uint_as_float(x[i]));
                }
                if (!is_b) {
                    // ---- stage A: send the peer's 32 partial columns, then the partial max ----
                    if (!wait_warp(my_sx_free0 + 8 * xb, xph ^ 1, abort, st, 0x2302)) { ok = false; break; }
                    const uint32_t dst = peer_sx + xb * AT_TILE128;
                    const uint32_t bar = peer_sx_full0 + 8 * xb;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        st_async_v4(dst + chunk_off(h, c), rp[4 * c], rp[4 * c + 1], rp[4 * c + 2], rp[4 * c + 3], bar);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) ro[i] = __float_as_uint(__uint_as_float(ro[i]) + __uint_as_float(xo[i]));
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->s_empty));
                const uint32_t mo = kh ? mhi : mlo, mp = kh ? mlo : mhi;  // valid slots of the own / peer half
                float pm = -INFINITY;  // partial maximum of this CTA's row over the tile's valid keys
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    if ((mo >> i) & 1u) pm = fmaxf(pm, __uint_as_float(ro[i]));
                    if ((mp >> i) & 1u) pm = fmaxf(pm, __uint_as_float(rp[i]));
                }
                if (!is_b) {
                    st_async_b32(peer_pm + xb * 512 + h * 4, __float_as_uint(pm), peer_sx_full0 + 8 * xb);
                    continue;
                }
                // ---- stage B: combine, probabilities, both copies of P ----
                const uint32_t msk = mo;
                if (!wait_warp(my_sx_full0 + 8 * xb, xph, abort, st, 0x2303)) { ok = false; break; }
                if (arm_thread) mbar_arrive_expect_tx(my_sx_full0 + 8 * xb, AT_SX_BYTES);  // its next phase
                float s32[32];
                {
                    const uint8_t* rowp = sx + xb * AT_TILE128;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float4 v = *(const float4*)(rowp + chunk_off(h, c));
                        const float pv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s32[4 * c + e] = __uint_as_float(ro[4 * c + e]) + pv[e];
                    }
                }
                const float pm_peer = pmx[xb * 128 + h];
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(peer_sx_free0 + 8 * xb);
                // The sum of the two partial maxima bounds every score of the row, and
                // both CTAs form it alike.  While it stays within 2^8 of the running
                // maximum, that maximum serves.  Where it does not, the warps of these
                // heads in both CTAs exchange the true maxima of their keys: the bound
                // alone may lie so far above the scores that all of exp underflows.
                const float mb = (pm == -INFINITY || pm_peer == -INFINITY) ? -INFINITY : (pm + pm_peer) * scale_log2;
                float alpha = 1.f;
                if (__any_sync(0xffffffffu, !(mb <= m_used + 8.0f))) {
                    float tm = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if ((msk >> i) & 1u) tm = fmaxf(tm, s32[i]);
                    const uint32_t tb = n_tm & 1;
                    st_async_b32(peer_tmx + tb * 512 + h * 4, __float_as_uint(tm), peer_tm_full0 + 8 * (quad * 2 + tb));
                    const uint32_t bar = smem_u32(&bars->tm_full[quad * 2 + tb]);
                    if (!wait_warp(bar, (n_tm >> 1) & 1, abort, st, 0x2307)) { ok = false; break; }
                    const float mt = fmaxf(tm, tmx[tb * 128 + h]) * scale_log2;
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(bar, 128);  // its next phase
                    ++n_tm;
                    if (mt > m_used + 8.0f) {
                        alpha = m_used == -INFINITY ? 0.f : ex2(m_used - mt);
                        l *= alpha;
                        m_used = mt;
                    }
                }
                uint32_t pw[16];
                {
                    // (scores of -inf alone: probabilities of 0, not of exp2(-inf + inf))
                    const float m_sub = m_used == -INFINITY ? 0.f : m_used;
                    float rs0 = 0.f, rs1 = 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float p0 = ((msk >> (2 * i)) & 1u) ? ex2(fmaf(s32[2 * i], scale_log2, -m_sub)) : 0.f;
                        const float p1 = ((msk >> (2 * i + 1)) & 1u) ? ex2(fmaf(s32[2 * i + 1], scale_log2, -m_sub)) : 0.f;
                        rs0 += p0;
                        rs1 += p1;
                        pw[i] = pack_bf16(p0, p1);
                    }
                    l += rs0 + rs1;
                }
                // P tile pb is free once PV(g - NPB) is done in both CTAs
                const uint32_t pb = g % NPB;
                if (!wait_warp(my_p_free0 + 8 * pb, ((g / NPB) & 1) ^ 1, abort, st, 0x2304)) { ok = false; break; }
                {
                    uint8_t* prow = smem + Lay::OFF_P + pb * AT_TILE128;
                    const uint32_t pdst = peer_p + pb * AT_TILE128;
                    const uint32_t bar = peer_p_full0 + 8 * pb;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int c = 4 * kh + q;
                        *(uint4*)(prow + chunk_off(h, c)) = make_uint4(pw[4 * q], pw[4 * q + 1], pw[4 * q + 2], pw[4 * q + 3]);
                        st_async_v4(pdst + chunk_off(h, c), pw[4 * q], pw[4 * q + 1], pw[4 * q + 2], pw[4 * q + 3], bar);
                    }
                }
                if (u > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    // O may be rescaled only between PV(g-1) and PV(g)
                    const uint32_t w = g - 1;
                    if (!wait_warp(my_p_free0 + 8 * (w % NPB), (w / NPB) & 1, abort, st, 0x2305)) { ok = false; break; }
                    tc_fence_after();
                    for (int c = 0; c < 8; ++c) {
                        uint32_t r[32];
                        const uint32_t ta = tmem + lane_off + TM_O + c * 32;
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
                if (lane == 0) mbar_arrive(my_p_full0 + 8 * pb);
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->info_empty[slot]));
            pend = true;
            it_pend = it;
            item_pend = item;
            m_pend = m_used;
            l_pend = l;
            ++nqt;
        }
        if (ok && pend) ok = epilogue(it_pend, item_pend, nqt - 1, m_pend, l_pend);
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();  // no DSMEM traffic may target a CTA that has exited
    tc_fence_after();
    if (warp == AT_MMA_WARP) tmem_dealloc(tmem, 512);
}

// Joins the parts of every item's rows: weights 2^(lse_p - max), one block a
// row (token and head).  Bound by reading the partial rows, which are in L2.
__global__ void __launch_bounds__(128) attn_paged_combine_kernel(const PagedAttnArgs a, int dense) {
    const int64_t grp = blockIdx.x / (unsigned)(a.group * a.heads);
    const int row = (int)(blockIdx.x - grp * (a.group * a.heads));
    PaItem it = dense ? pa_item<true>(a, grp, 0, 0) : pa_item<false>(a, grp, 0, a.k_sel);
    const int tok = row / a.heads, head = row - tok * a.heads;
    if (tok >= it.ntok) return;
    const int64_t t = it.t0 + tok;
    const float* pl = a.part_lse + grp * a.splits * 128 + row;
    float m = -INFINITY;
    for (int p = 0; p < a.splits; ++p) m = fmaxf(m, __ldg(pl + p * 128));
    const float* po = a.part_o + (grp * a.splits * 128 + row) * 512 + threadIdx.x * 4;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    for (int p = 0; p < a.splits; ++p) {
        const float z = __ldg(pl + p * 128);
        if (z == -INFINITY) continue;  // an empty part: its rows were not written
        const float w = ex2(z - m);    // NaN stays NaN
        const float4 v = __ldg((const float4*)(po + (int64_t)p * 128 * 512));
        l += w;
        o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y), o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
    }
    const float inv = l != 0.f ? 1.0f / l : 0.f;
    *(uint2*)((__nv_bfloat16*)a.out + t * a.out_stride_tok + (int64_t)head * a.out_stride_head + threadIdx.x * 4) =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (a.lse && threadIdx.x == 0)
        a.lse[t * a.heads + head] = l != 0.f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// CTA pairs that can be resident at once (the persistent grid).
template <bool DENSE>
static int pa_pairs_resident() {
    static int cached = 0;
    if (cached > 0) return cached;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * 1024, 1, 1);
    cfg.blockDim = dim3(AT_THREADS, 1, 1);
    cfg.dynamicSmemBytes = PaLayout::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, (const void*)attn_paged_kernel<DENSE>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;
    }
    if (n > 0) cached = n;
    return n;
}

template <bool DENSE>
static bool pa_launch(const PagedAttnArgs& a, cudaStream_t s) {
    const void* fn = (const void*)attn_paged_kernel<DENSE>;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, PaLayout::SMEM) != cudaSuccess) return false;
    // the setmaxnreg split must fit the registers the block is launched with
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, fn) != cudaSuccess || (int64_t)fa.numRegs * AT_THREADS < (int64_t)AT_REGS_SPLIT)
        return false;
    const int pairs = pa_pairs_resident<DENSE>();
    if (pairs <= 0) return false;
    const int64_t items = a.groups * a.splits;
    const int64_t grid = items < pairs ? items : pairs;
    attn_paged_kernel<DENSE><<<(unsigned)(2 * grid), AT_THREADS, PaLayout::SMEM, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return false;
    if (a.splits > 1) {
        const int64_t rows = a.groups * a.group * a.heads;
        attn_paged_combine_kernel<<<(unsigned)rows, 128, 0, s>>>(a, DENSE ? 1 : 0);
    }
    return cudaGetLastError() == cudaSuccess;
}

bool launch_paged_attn_tc(const PagedAttnArgs& a, cudaStream_t s) {
    if (a.groups <= 0) return true;
    return a.idx ? pa_launch<false>(a, s) : pa_launch<true>(a, s);
}

}  // namespace dsa
