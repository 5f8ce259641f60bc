// paged_scores.cu -- lightning-indexer scores of folded queries over the paged
// indexer keys.
//
// I[t, s] = ReLU((u_t . k_s) * s_k[s] * s_row[t]) for s <= pos_t, over keys found
// through the page table.
//
// FP8: keys are the M side of the MMA (128 keys a tile, one TMEM lane each) and
// up to 16 queries (paged_scores_few_kernel: decode) or 128 (paged_scores_kernel:
// chunks) of a sequence the N side: every key row is read once per 128 queries, and
// a warp's stores are 32 consecutive scores of one query.  Bound by HBM: a decode
// reads 132 bytes a key, a chunk writes 4 bytes a (query, key) pair; the MMA of a
// tile (M 128, N 16 or 128, K 128) takes less time than either.
// The key rows arrive by 16-byte cp.async, 4 rows x 128 bytes an instruction,
// because pages may start at any row of a tile and have any size; a warp looks
// up its 32 keys' pages with one load and shuffles the rows' places around.
// Keys that the page table does not hold get -inf and are reported.
//
// Few queries: a CTA's start (tensor memory, barriers, the first dependent loads)
// costs about 5 us, and sequences differ in length, so the grid holds as many CTAs
// as are resident and each takes an equal stretch of all sequences' key tiles,
// found by a scan over the lengths.  The queries travel with every tile (128 bytes
// beside 16 KB for a decode), so a stretch may cross sequences at any tile.  A CTA
// per 28 tiles of one sequence measured 87 us (64 caches of 16K to 64K keys, graph
// replays, as all times beside choices here), this form 66 us; a call among others
// takes 70 us, 0.77 of the copy bandwidth.
#include "rows.cuh"

namespace dsa {

constexpr int PS_KEYS = 128;  // keys per tile
// Key stages: three measured 65 us against 66 (the decode above) and 33.1 against 32.7
// (1000 queries on 32000 keys); more would take a CTA from the SM.
constexpr int PS_NST = 4;
constexpr int PS_PROD = 4;    // producer warps
constexpr uint32_t PS_STAGE = PS_KEYS * 128;

template <int NQ>
struct PsSmem {
    static constexpr uint32_t OFF_B = PS_NST * PS_STAGE;  // queries, 128-byte swizzled rows
    static constexpr uint32_t OFF_SROW = OFF_B + NQ * 128;
    static constexpr uint32_t OFF_BAR = OFF_SROW + NQ * 4;
    static constexpr uint32_t SMEM = OFF_BAR + 256 + 1024;  // + alignment
    static constexpr uint32_t TMEM_COLS = 2 * NQ < 32 ? 32 : 2 * NQ;
    // Warps: the epilogue's (one per TMEM lane quadrant and 64 queries), producers, MMA
    static constexpr int EPI = NQ / 16;
    static constexpr int HALF = NQ / (EPI / 4);  // queries of an epilogue warp
    static constexpr int MMA_WARP = EPI + PS_PROD;
    static constexpr int THREADS = 32 * (MMA_WARP + 1);
};
struct PsBars {
    uint64_t full[PS_NST], empty[PS_NST];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

DSA_DEV float ps_relu(float x) {  // as the packed scores: -0 and below to +0, NaN to +inf
    int b = __float_as_int(x);
    b = max(b, 0);
    b = min(b, 0x7F800000);
    return __int_as_float(b);
}

template <int NQ>
__global__ void __launch_bounds__(PsSmem<NQ>::THREADS) paged_scores_kernel(const PagedScoresArgs a) {
    using Lay = PsSmem<NQ>;
    extern __shared__ uint8_t ps_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)ps_raw + 1023) & ~(uintptr_t)1023);
    PsBars* bars = (PsBars*)(smem + Lay::OFF_BAR);
    float* srow = (float*)(smem + Lay::OFF_SROW);
    constexpr int PS_EPI = Lay::EPI, PS_MMA_WARP = Lay::MMA_WARP, PS_THREADS = Lay::THREADS;
    const int warp = (int)warp_id(), lane = (int)lane_id();
    volatile int* abort = &bars->abort;
    StatusHdr* st = a.st;
    if (blockIdx.x == 0 && threadIdx.x == 0) report_no_sequence(a.sv, a.row_begin, a.row_begin + a.row_count, st);

    // this CTA: queries [t_first, t_first + nrows) of sequence b, key tiles [t_lo, t_hi)
    const int64_t nblk = (a.max_seqlen_q + NQ - 1) / NQ;
    const int64_t tiles = (a.cols + PS_KEYS - 1) / PS_KEYS;
    const int64_t nsplit = (tiles + a.tiles_per_cta - 1) / a.tiles_per_cta;
    const int64_t u = blockIdx.x / nsplit, split = blockIdx.x - u * nsplit;
    const int b = (int)(u / nblk);
    const int64_t q0 = __ldg(a.sv.cu_q + b), q1 = __ldg(a.sv.cu_q + b + 1);
    const int64_t lk = __ldg(a.sv.cu_k + b + 1) - __ldg(a.sv.cu_k + b), lq = q1 - q0;
    const int64_t i0 = (u - b * nblk) * NQ;
    if (i0 >= lq) return;
    const int64_t t_first = q0 + i0;
    const int nrows = (int)min((int64_t)NQ, min(lq - i0, a.total_q - t_first));
    const int64_t pos_first = lk - lq + i0;  // position of block row 0
    if (t_first < 0 || pos_first < 0) {      // the batch's description is inconsistent
        if (threadIdx.x == 0) report(st, DSA_ERR_INDEX, t_first);
        if (t_first < 0) return;
    }
    // rows of the block that are asked for (and have a position)
    const int r_lo = (int)max(max((int64_t)0, -pos_first), a.row_begin - t_first);
    const int r_hi = (int)min((int64_t)nrows, a.row_begin + a.row_count - t_first);
    if (r_lo >= r_hi) return;
    const int64_t pos_last = pos_first + r_hi - 1;           // of the last row asked for
    const int64_t t_lo = split * a.tiles_per_cta;
    const int64_t t_hi = min(tiles, t_lo + a.tiles_per_cta);
    const int64_t t_act = max(t_lo, min(t_hi, pos_last / PS_KEYS + 1));  // tiles with keys some row sees
    if (t_act == t_lo && !a.fill) return;

    const uint32_t s_a = smem_u32(smem), s_b = smem_u32(smem + Lay::OFF_B);
    if (threadIdx.x == 0) {
        for (int i = 0; i < PS_NST; ++i) {
            mbar_init(smem_u32(&bars->full[i]), PS_PROD * 32);
            mbar_init(smem_u32(&bars->empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars->acc_full[i]), 1);
            mbar_init(smem_u32(&bars->acc_empty[i]), PS_EPI);
        }
        mbar_init(smem_u32(&bars->drain), 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == PS_MMA_WARP) {
        tmem_alloc(smem_u32(&bars->tmem_base), Lay::TMEM_COLS);
        tmem_relinquish();  // several CTAs share an SM
    }
    // the queries, 16 bytes a thread; rows past the block are zero
    for (int i = threadIdx.x; i < NQ * 8; i += PS_THREADS) {
        const int r = i >> 3, c = i & 7;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (r < nrows) v = __ldg((const uint4*)((const uint8_t*)a.u + (t_first + r) * 128 + c * 16));
        *(uint4*)(smem + Lay::OFF_B + r * 128 + ((c ^ (r & 7)) << 4)) = v;
    }
    for (int i = threadIdx.x; i < NQ; i += PS_THREADS) srow[i] = i < nrows ? __ldg(a.s_row + t_first + i) : 0.f;
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    if (warp >= PS_EPI && warp < PS_MMA_WARP) {
        // ================= producers =================
        const int pw = warp - PS_EPI, sub = lane >> 3, chunk = lane & 7;
        const uint8_t* pool = (const uint8_t*)a.k;
        auto place = [&](int64_t tile) -> int64_t {  // byte offset of this lane's key, -1: not loaded
            const int64_t s = tile * PS_KEYS + pw * 32 + lane;
            if (tile >= t_act || s > pos_last) return -1;
            const PageRef pr = page_of(a.pv, b, s);
            return pr.page < 0 ? -1 : pr.page * a.k_page_stride + (int64_t)pr.slot * 128;
        };
        int64_t nxt = place(t_lo);
        uint32_t g = 0;
        for (int64_t tile = t_lo; tile < t_act; ++tile, ++g) {
            const int64_t cur = nxt;
            nxt = place(tile + 1);
            const uint32_t s = g % PS_NST;
            if (!wait_warp(smem_u32(&bars->empty[s]), ((g / PS_NST) & 1) ^ 1, abort, st, 0x4101)) break;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int key = i * 4 + sub;
                const int64_t off = __shfl_sync(0xffffffffu, cur, key);
                const int r = pw * 32 + key;
                if (off >= 0) cp_async16(s_a + s * PS_STAGE + r * 128 + ((chunk ^ (r & 7)) << 4), pool + off + chunk * 16);
            }
            cp_async_arrive(smem_u32(&bars->full[s]));
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == PS_MMA_WARP) {
        // ================= MMA issuer =================
        constexpr uint32_t idesc = idesc_make(0, 0, false, PS_KEYS, NQ);
        uint32_t g = 0;
        for (int64_t tile = t_lo; tile < t_act; ++tile, ++g) {
            const uint32_t s = g % PS_NST, ab = g & 1;
            if (!wait_warp(smem_u32(&bars->full[s]), (g / PS_NST) & 1, abort, st, 0x4201)) break;
            if (!wait_warp(smem_u32(&bars->acc_empty[ab]), ((g >> 1) & 1) ^ 1, abort, st, 0x4202)) break;
            fence_proxy_async();
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_fp8_ss(tmem + ab * NQ, sdesc_sw128(s_a + s * PS_STAGE + ks * 32, 16, 1024),
                               sdesc_sw128(s_b + ks * 32, 16, 1024), idesc, ks > 0 ? 1u : 0u);
                mma_commit(smem_u32(&bars->empty[s]));
                mma_commit(smem_u32(&bars->acc_full[ab]));
            }
            __syncwarp();
        }
        if (*abort && lane == 0) {
            mma_commit(smem_u32(&bars->drain));
            mbar_wait(smem_u32(&bars->drain), 0, nullptr, st, 0x4203, 1ll << 28);
        }
    } else {
        // ================= epilogue: one thread per key (and 64 queries) =================
        const int quad = warp & 3, ch = warp >> 2;
        float* out = a.scores + (t_first - a.row_begin) * a.ld;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const float none = a.fill ? -INFINITY : 0.f;  // the selection's own scores are never negative
        // rows of this warp, from a whole group of 16
        const int c_beg = max(r_lo & ~15, ch * Lay::HALF), c_end = min(r_hi, (ch + 1) * Lay::HALF);
        // A key's scale takes two dependent loads: pages are read three tiles ahead,
        // scales two, so that neither is waited for.
        const int32_t* table = a.pv.table + b * a.pv.ld_table;
        auto page_at = [&](int64_t tile, int& slot) -> int32_t {
            const int64_t s = tile * PS_KEYS + quad * 32 + lane;
            slot = 0;
            if (tile >= t_act || s > pos_last) return 0;  // no row sees it
            uint32_t p, o;
            page_split(a.pv, (uint32_t)s, p, o);
            slot = (int)o;
            return (int64_t)p < a.pv.ld_table ? __ldg(table + p) : -1;
        };
        auto scale_at = [&](int64_t tile, int32_t pg, int slot, bool& have) -> float {
            const int64_t s = tile * PS_KEYS + quad * 32 + lane;
            have = true;
            if (tile >= t_act || s > pos_last) return 0.f;
            have = (uint32_t)pg < (uint32_t)a.pv.num_pages;
            if (!have) {
                report(st, DSA_ERR_INDEX, t_first);
                return 0.f;
            }
            return __ldg(a.k_scale + (int64_t)pg * a.scale_page_stride + slot);
        };
        int sl0, sl1, sl2;
        const int32_t pg0 = page_at(t_lo, sl0), pg1 = page_at(t_lo + 1, sl1);
        int32_t pg2 = page_at(t_lo + 2, sl2);
        bool h0, h1;
        float k0 = scale_at(t_lo, pg0, sl0, h0), k1 = scale_at(t_lo + 1, pg1, sl1, h1);
        uint32_t g = 0;
        bool ok = true;
        for (int64_t tile = t_lo; ok && tile < t_act; ++tile, ++g) {
            const uint32_t ab = g & 1;
            const float ks = k0;
            const bool have = h0;
            k0 = k1, h0 = h1;
            k1 = scale_at(tile + 2, pg2, sl2, h1);
            pg2 = page_at(tile + 3, sl2);
            if (!wait_warp(smem_u32(&bars->acc_full[ab]), (g >> 1) & 1, abort, st, 0x4301)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int64_t s = tile * PS_KEYS + quad * 32 + lane;
            const bool in = s < a.cols;
            const int64_t end = (tile + 1) * PS_KEYS;  // every row asked for sees the whole tile
            const bool whole = end <= a.cols && end - 1 <= pos_first + r_lo;
            if (c_beg >= c_end) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->acc_empty[ab]));
            }
            for (int c0 = c_beg; c0 < c_end; c0 += 16) {
                uint32_t acc[16];
                tmem_ld16(tmem + lane_off + ab * NQ + c0, acc);
                tmem_wait_ld();
                if (c0 + 16 >= c_end) {  // the last columns read: hand the accumulator back
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars->acc_empty[ab]));
                }
                if (whole && c0 >= r_lo && c0 + 16 <= r_hi) {
                    float* o = out + (int64_t)c0 * a.ld + s;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 f = *(const float4*)(srow + c0 + 4 * q);
                        const float fr[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = ps_relu(__fmul_rn(__fmul_rn(__uint_as_float(acc[4 * q + e]), ks), fr[e]));
                            *o = have ? x : none;
                            o += a.ld;
                        }
                    }
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int r = c0 + e;
                    if (r >= r_lo && r < r_hi) {
                        const float x = ps_relu(__fmul_rn(__fmul_rn(__uint_as_float(acc[e]), ks), srow[r]));
                        const bool seen = s <= pos_first + r;
                        if (in && (seen || a.fill)) out[(int64_t)r * a.ld + s] = seen && have ? x : none;
                    }
                }
            }
        }
        if (a.fill)  // tiles past every row's position
            for (int64_t tile = t_act; tile < t_hi; ++tile) {
                const int64_t s = tile * PS_KEYS + quad * 32 + lane;
                if (s < a.cols)
                    for (int r = max(r_lo, ch * Lay::HALF); r < c_end; ++r) out[(int64_t)r * a.ld + s] = -INFINITY;
            }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == PS_MMA_WARP) tmem_dealloc(tmem, Lay::TMEM_COLS);
}

// ---------------------------------------------------------------------------
// fp32 keys (the small fp32 configuration): 8 lanes a key, 16 columns each,
// one query a block; exact fp32 products and sums.
// ---------------------------------------------------------------------------
constexpr int PSF_KEYS = 256;  // keys per block

__global__ void __launch_bounds__(256) paged_scores_f32_kernel(const PagedScoresArgs a) {
    const int64_t t = a.row_begin + blockIdx.y;
    const RowInfo ri = row_info(a.sv, t);
    if (!ri.ok) {
        if (threadIdx.x == 0) report(a.st, DSA_ERR_INDEX, t);
        return;
    }
    const int sub = threadIdx.x & 7;
    float q[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = __ldg((const float4*)((const float*)a.u + t * 128 + sub * 16) + i);
        q[4 * i] = v.x, q[4 * i + 1] = v.y, q[4 * i + 2] = v.z, q[4 * i + 3] = v.w;
    }
    const float sr = a.s_row ? __ldg(a.s_row + t) : 1.f;
    float* out = a.scores + (int64_t)blockIdx.y * a.ld;
    const int64_t s_end = min((int64_t)(blockIdx.x + 1) * PSF_KEYS, a.cols);
    for (int64_t s0 = (int64_t)blockIdx.x * PSF_KEYS; s0 < s_end; s0 += 32) {
        const int64_t s = s0 + (threadIdx.x >> 3);
        float acc = 0.f;
        bool have = true;
        if (s <= ri.pos && s < s_end) {
            const PageRef pr = page_of(a.pv, ri.b, s);
            have = pr.page >= 0;
            if (have) {
                const float4* k = (const float4*)((const float*)a.k + pr.page * a.k_page_stride + (int64_t)pr.slot * 128 +
                                                  sub * 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 v = __ldg(k + i);
                    acc = fmaf(q[4 * i], v.x, acc);
                    acc = fmaf(q[4 * i + 1], v.y, acc);
                    acc = fmaf(q[4 * i + 2], v.z, acc);
                    acc = fmaf(q[4 * i + 3], v.w, acc);
                }
            } else {
                report(a.st, DSA_ERR_INDEX, t);
            }
        }
        acc += __shfl_xor_sync(0xffffffffu, acc, 1);
        acc += __shfl_xor_sync(0xffffffffu, acc, 2);
        acc += __shfl_xor_sync(0xffffffffu, acc, 4);
        if (sub == 0 && s < s_end) {
            const bool seen = s <= ri.pos;
            if (seen || a.fill) out[s] = seen && have ? ps_relu(__fmul_rn(acc, sr)) : a.fill ? -INFINITY : 0.f;
        }
    }
}

// ---------------------------------------------------------------------------
// At most 16 queries a sequence
// ---------------------------------------------------------------------------
struct PfwSmem {
    static constexpr uint32_t STAGE = PS_STAGE + 16 * 128;  // keys, then the queries (128-byte swizzled rows)
    static constexpr uint32_t OFF_BAR = PS_NST * STAGE;
    static constexpr uint32_t OFF_CUT = OFF_BAR + 128;
    static constexpr uint32_t SMEM = OFF_CUT + 64 + 1024;   // + alignment
};
static_assert(sizeof(PsBars) <= 128, "barrier block");
constexpr int PFW_EPI = 4, PFW_MMA = PFW_EPI + PS_PROD, PFW_THREADS = 32 * (PFW_MMA + 1);
// Resident an SM: the shared memory of four stages allows three.  Four CTAs of two
// stages measured 84 us against 66 for the decode above, five 75.
constexpr int PFW_CTAS = 3;

// A sequence's rows that are asked for, and its key tiles: those that some row
// sees, then (fill) those that none does.
struct PfwSeq {
    int64_t t0, pos0;   // token and position of query 0
    int r_lo, r_hi;     // rows asked for
    int64_t act, fill;
};
DSA_DEV PfwSeq pfw_seq(const PagedScoresArgs& a, int b, int64_t tiles) {
    PfwSeq s;
    s.t0 = __ldg(a.sv.cu_q + b);
    const int64_t q1 = __ldg(a.sv.cu_q + b + 1), lk = __ldg(a.sv.cu_k + b + 1) - __ldg(a.sv.cu_k + b);
    s.pos0 = lk - (q1 - s.t0);
    const int64_t n = s.t0 < 0 ? 0 : min(min(q1 - s.t0, (int64_t)16), a.total_q - s.t0);
    s.r_lo = (int)min(max(max((int64_t)0, -s.pos0), a.row_begin - s.t0), (int64_t)16);
    s.r_hi = (int)min(n, a.row_begin + a.row_count - s.t0);
    s.act = s.fill = 0;
    if (s.r_lo < s.r_hi) {
        s.act = min(tiles, (s.pos0 + s.r_hi - 1) / PS_KEYS + 1);
        s.fill = a.fill ? tiles - s.act : 0;
    }
    return s;
}
struct PfwCut {
    int b;         // sequence (batch: the end)
    int64_t tile;  // tiles of it before the cut
};

__global__ void __launch_bounds__(PFW_THREADS) paged_scores_few_kernel(const PagedScoresArgs a) {
    using Lay = PfwSmem;
    extern __shared__ uint8_t ps_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)ps_raw + 1023) & ~(uintptr_t)1023);
    PsBars* bars = (PsBars*)(smem + Lay::OFF_BAR);
    PfwCut* cuts = (PfwCut*)(smem + Lay::OFF_CUT);  // [4] visible tiles from, to; filled tiles from, to
    const int warp = __shfl_sync(0xffffffffu, (int)warp_id(), 0), lane = (int)lane_id();
    volatile int* abort = &bars->abort;
    StatusHdr* st = a.st;
    const int64_t tiles = (a.cols + PS_KEYS - 1) / PS_KEYS;
    const int batch = a.sv.batch;
    if (blockIdx.x == 0 && threadIdx.x == 32 * PFW_MMA - 1) report_no_sequence(a.sv, a.row_begin, a.row_begin + a.row_count, st);
    if (threadIdx.x == 0) {
        for (int i = 0; i < PS_NST; ++i) {
            mbar_init(smem_u32(&bars->full[i]), PS_PROD * 32);
            mbar_init(smem_u32(&bars->empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars->acc_full[i]), 1);
            mbar_init(smem_u32(&bars->acc_empty[i]), PFW_EPI);
        }
        mbar_init(smem_u32(&bars->drain), 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == PFW_MMA) {
        tmem_alloc(smem_u32(&bars->tmem_base), 32);
        tmem_relinquish();  // several CTAs share an SM
    }
    if (warp == PFW_EPI) {  // this CTA's stretch
        auto weight = [&](int b, int64_t& act, int64_t& fill) {
            act = fill = 0;
            if (b >= batch) return;
            const PfwSeq s = pfw_seq(a, b, tiles);
            act = s.act, fill = s.fill;
            if (blockIdx.x == 0 && (s.pos0 < 0 || s.t0 < 0)) report(st, DSA_ERR_INDEX, s.t0);  // no such position
        };
        int64_t total[2] = {0, 0};
        for (int b0 = 0; b0 < batch; b0 += 32) {
            int64_t w[2];
            weight(b0 + lane, w[0], w[1]);
            total[0] += w[0], total[1] += w[1];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            total[0] += __shfl_xor_sync(0xffffffffu, total[0], o);
            total[1] += __shfl_xor_sync(0xffffffffu, total[1], o);
        }
        const int64_t g = gridDim.x;
        if (lane < 4) cuts[lane].b = batch, cuts[lane].tile = 0;
        __syncwarp();
        int64_t base[2] = {0, 0};
        for (int b0 = 0; b0 < batch; b0 += 32) {
            int64_t w[2];
            weight(b0 + lane, w[0], w[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                int64_t incl = w[k];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += v;
                }
                incl += base[k];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int64_t p = blockIdx.x + i, target = total[k] / g * p + total[k] % g * p / g;
                    const uint32_t past = __ballot_sync(0xffffffffu, incl > target);
                    if (past && base[k] <= target && lane == __ffs((int)past) - 1) {
                        cuts[2 * k + i].b = b0 + lane;
                        cuts[2 * k + i].tile = target - (incl - w[k]);
                    }
                }
                base[k] = __shfl_sync(0xffffffffu, incl, 31);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base, s0 = smem_u32(smem);
    const PfwCut from = cuts[0], to = cuts[1];
    // the tiles [lo, hi) of sequence b that are this CTA's
    auto range = [&](const PfwCut& f, const PfwCut& t, int b, int64_t n, int64_t& lo, int64_t& hi) {
        lo = b == f.b ? f.tile : 0;
        hi = b == t.b ? t.tile : n;
    };

    if (warp >= PFW_EPI && warp < PFW_MMA) {
        // ================= producers =================
        const int pw = warp - PFW_EPI, sub = lane >> 3, chunk = lane & 7;
        const uint8_t* pool = (const uint8_t*)a.k;
        uint32_t g = 0;
        bool ok = true;
        for (int b = from.b; ok && b <= min(to.b, batch - 1); ++b) {
            const PfwSeq q = pfw_seq(a, b, tiles);
            int64_t lo, hi;
            range(from, to, b, q.act, lo, hi);
            const int64_t pos_last = q.pos0 + q.r_hi - 1;
            const int32_t* table = a.pv.table + b * a.pv.ld_table;
            // this lane's key of a tile: its page (read two tiles ahead) and row
            auto page_at = [&](int64_t tile, int& slot) -> int32_t {
                const int64_t s = tile * PS_KEYS + pw * 32 + lane;
                uint32_t p, o;
                page_split(a.pv, (uint32_t)s, p, o);
                slot = (int)o;
                return tile < hi && s <= pos_last && (int64_t)p < a.pv.ld_table ? __ldg(table + p) : -1;
            };
            int sl0, sl1;
            int32_t pg0 = page_at(lo, sl0), pg1 = page_at(lo + 1, sl1);
            const int qr = pw * 4 + sub;  // this lane's query row
            const uint8_t* qrow = (const uint8_t*)a.u + (q.t0 + qr) * 128 + chunk * 16;
            for (int64_t tile = lo; tile < hi; ++tile, ++g) {
                const int64_t cur = (uint32_t)pg0 < (uint32_t)a.pv.num_pages ? pg0 * a.k_page_stride + (int64_t)sl0 * 128 : -1;
                pg0 = pg1, sl0 = sl1;
                pg1 = page_at(tile + 2, sl1);
                const uint32_t stg = s0 + g % PS_NST * Lay::STAGE;
                if (!wait_warp(smem_u32(&bars->empty[g % PS_NST]), ((g / PS_NST) & 1) ^ 1, abort, st, 0x4101)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int key = i * 4 + sub;
                    const int64_t off = __shfl_sync(0xffffffffu, cur, key);
                    const int r = pw * 32 + key;
                    if (off >= 0) cp_async16(stg + r * 128 + ((chunk ^ (r & 7)) << 4), pool + off + chunk * 16);
                }
                if (qr < q.r_hi) cp_async16(stg + PS_STAGE + qr * 128 + ((chunk ^ (qr & 7)) << 4), qrow);
                cp_async_arrive(smem_u32(&bars->full[g % PS_NST]));
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == PFW_MMA) {
        // ================= MMA issuer =================
        constexpr uint32_t idesc = idesc_make(0, 0, false, PS_KEYS, 16);
        uint32_t g = 0;
        bool ok = true;
        for (int b = from.b; ok && b <= min(to.b, batch - 1); ++b) {
            int64_t lo, hi;
            range(from, to, b, pfw_seq(a, b, tiles).act, lo, hi);
            for (int64_t tile = lo; tile < hi; ++tile, ++g) {
                const uint32_t s = g % PS_NST, ab = g & 1;
                if (!wait_warp(smem_u32(&bars->full[s]), (g / PS_NST) & 1, abort, st, 0x4201) ||
                    !wait_warp(smem_u32(&bars->acc_empty[ab]), ((g >> 1) & 1) ^ 1, abort, st, 0x4202)) {
                    ok = false;
                    break;
                }
                fence_proxy_async();
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t k = s0 + s * Lay::STAGE;
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_fp8_ss(tmem + ab * 16, sdesc_sw128(k + ks * 32, 16, 1024),
                                   sdesc_sw128(k + PS_STAGE + ks * 32, 16, 1024), idesc, ks > 0 ? 1u : 0u);
                    mma_commit(smem_u32(&bars->empty[s]));
                    mma_commit(smem_u32(&bars->acc_full[ab]));
                }
                __syncwarp();
            }
        }
        if (*abort && lane == 0) {
            mma_commit(smem_u32(&bars->drain));
            mbar_wait(smem_u32(&bars->drain), 0, nullptr, st, 0x4203, 1ll << 28);
        }
        __syncwarp();
    } else {
        // ================= epilogue: one thread per key =================
        const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
        const float none = a.fill ? -INFINITY : 0.f;  // the selection's own scores are never negative
        uint32_t g = 0;
        bool ok = true;
        for (int b = from.b; ok && b <= min(to.b, batch - 1); ++b) {
            const PfwSeq q = pfw_seq(a, b, tiles);
            int64_t lo, hi;
            range(from, to, b, q.act, lo, hi);
            if (lo >= hi) continue;
            const int64_t pos_last = q.pos0 + q.r_hi - 1;
            float* out = a.scores + (q.t0 - a.row_begin) * a.ld;
            const float sr = lane < q.r_hi ? __ldg(a.s_row + q.t0 + lane) : 0.f;  // lane r: row r's scale
            // a key's scale takes two dependent loads: pages are read three tiles ahead,
            // scales two, so that neither is waited for
            const int32_t* table = a.pv.table + b * a.pv.ld_table;
            auto page_at = [&](int64_t tile, int& slot) -> int32_t {
                const int64_t s = tile * PS_KEYS + warp * 32 + lane;
                slot = 0;
                if (tile >= hi || s > pos_last) return 0;  // no row sees it
                uint32_t p, o;
                page_split(a.pv, (uint32_t)s, p, o);
                slot = (int)o;
                return (int64_t)p < a.pv.ld_table ? __ldg(table + p) : -1;
            };
            auto scale_at = [&](int64_t tile, int32_t pg, int slot, bool& have) -> float {
                const int64_t s = tile * PS_KEYS + warp * 32 + lane;
                have = true;
                if (tile >= hi || s > pos_last) return 0.f;
                have = (uint32_t)pg < (uint32_t)a.pv.num_pages;
                if (!have) {
                    report(st, DSA_ERR_INDEX, q.t0);
                    return 0.f;
                }
                return __ldg(a.k_scale + (int64_t)pg * a.scale_page_stride + slot);
            };
            int sl0, sl1, sl2;
            const int32_t pg0 = page_at(lo, sl0), pg1 = page_at(lo + 1, sl1);
            int32_t pg2 = page_at(lo + 2, sl2);
            bool h0, h1;
            float k0 = scale_at(lo, pg0, sl0, h0), k1 = scale_at(lo + 1, pg1, sl1, h1);
            for (int64_t tile = lo; tile < hi; ++tile, ++g) {
                const uint32_t ab = g & 1;
                const float ks = k0;
                const bool have = h0;
                k0 = k1, h0 = h1;
                k1 = scale_at(tile + 2, pg2, sl2, h1);
                pg2 = page_at(tile + 3, sl2);
                if (!wait_warp(smem_u32(&bars->acc_full[ab]), (g >> 1) & 1, abort, st, 0x4301)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t acc[16];
                tmem_ld16(tmem + lane_off + ab * 16, acc);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->acc_empty[ab]));
                const int64_t s = tile * PS_KEYS + warp * 32 + lane;
                const bool in = s < a.cols;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float fr = __shfl_sync(0xffffffffu, sr, r);
                    if (r >= q.r_lo && r < q.r_hi) {
                        const float x = ps_relu(__fmul_rn(__fmul_rn(__uint_as_float(acc[r]), ks), fr));
                        const bool seen = s <= q.pos0 + r;
                        if (in && (seen || a.fill)) out[(int64_t)r * a.ld + s] = seen && have ? x : none;
                    }
                }
            }
        }
        // tiles past every row's position
        const PfwCut ff = cuts[2], ft = cuts[3];
        for (int b = ff.b; b <= min(ft.b, batch - 1); ++b) {
            const PfwSeq q = pfw_seq(a, b, tiles);
            int64_t lo, hi;
            range(ff, ft, b, q.fill, lo, hi);
            float* out = a.scores + (q.t0 - a.row_begin) * a.ld;
            const int64_t end = min((q.act + hi) * PS_KEYS, a.cols);
            for (int r = q.r_lo; r < q.r_hi; ++r)
                for (int64_t s = (q.act + lo) * PS_KEYS + threadIdx.x; s < end; s += 32 * PFW_EPI)
                    out[(int64_t)r * a.ld + s] = -INFINITY;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == PFW_MMA) tmem_dealloc(tmem, 32);
}

static bool pfw_launch(const PagedScoresArgs& a, cudaStream_t s) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaFuncSetAttribute(paged_scores_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PfwSmem::SMEM) !=
            cudaSuccess)
        return false;
    const int64_t tiles = (a.cols + PS_KEYS - 1) / PS_KEYS * a.sv.batch, most = (int64_t)sms * PFW_CTAS;
    paged_scores_few_kernel<<<(unsigned)(tiles < most ? tiles : most), PFW_THREADS, PfwSmem::SMEM, s>>>(a);
    return cudaGetLastError() == cudaSuccess;
}

template <int NQ>
static bool ps_launch(PagedScoresArgs a, cudaStream_t s) {
    const int64_t tiles = (a.cols + PS_KEYS - 1) / PS_KEYS;
    const int64_t units = (a.max_seqlen_q + NQ - 1) / NQ * a.sv.batch;
    if (tiles <= 0 || units <= 0) return true;
    // Key tiles a CTA: as many CTAs as are resident for one sequence (1000 x 32000:
    // 33 us against 36 with four an SM), twice that for several, whose lengths may
    // differ much: 63 single tokens and a chunk of 17 over 16K to 64K keys 154 us
    // against 165.  Sequences alike pay for it (queries x keys: 3 x 385 x 20K 42.9
    // against 40.7, 8 x 128 x 10K 25.5 against 24.4, 32 x 20 x 5K 22.6 against 20.4).
    const int64_t ctas = 148 * (a.sv.batch == 1 ? 2 : 4);
    int64_t per = (tiles * units + ctas - 1) / ctas;
    per = per < 2 ? 2 : per > 64 ? 64 : per;
    a.tiles_per_cta = (int)per;
    const int64_t grid = (tiles + per - 1) / per * units;
    if (grid >= ((int64_t)1 << 31)) return false;
    if (cudaFuncSetAttribute(paged_scores_kernel<NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)PsSmem<NQ>::SMEM) != cudaSuccess)
        return false;
    paged_scores_kernel<NQ><<<(unsigned)grid, PsSmem<NQ>::THREADS, PsSmem<NQ>::SMEM, s>>>(a);
    return cudaGetLastError() == cudaSuccess;
}

bool launch_paged_scores(const PagedScoresArgs& a, bool e4m3, cudaStream_t s) {
    if (a.row_count <= 0 || a.cols <= 0) return true;
    // By the longest query count, the only one that the host has.  A sequence of more
    // than 16 takes the others with it: 63 single tokens and one of 16 over 16K to 64K
    // keys 108 us, with one of 17 154 us (the same on the kernel for few queries would
    // read the longer one's keys twice, and 64 times for 1000).
    if (e4m3) return a.max_seqlen_q <= 16 ? pfw_launch(a, s) : ps_launch<128>(a, s);
    const int64_t gx = (a.cols + PSF_KEYS - 1) / PSF_KEYS;
    // rows on the grid's second axis, at most 65535 a launch
    for (int64_t r = 0; r < a.row_count; r += 65535) {
        PagedScoresArgs p = a;
        p.row_begin = a.row_begin + r;
        p.row_count = a.row_count - r < 65535 ? a.row_count - r : 65535;
        p.scores = a.scores + r * a.ld;
        paged_scores_f32_kernel<<<dim3((unsigned)gx, (unsigned)p.row_count), 256, 0, s>>>(p);
        if (cudaGetLastError() != cudaSuccess) return false;
    }
    return true;
}

}  // namespace dsa
