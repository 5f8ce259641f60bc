// attn_paged_f32.cu -- attention over a paged cache in exact fp32 (the small fp32
// configuration: up to 32 heads share one K row and one V row, dk and dv of 32 to
// 128), dense causal or over selected positions.
//
// One block takes one query token and a part of its keys, in tiles of 32 keys
// that all heads share: rows arrive in shared memory by cp.async, two tiles in
// flight; a warp scores 32 keys at a time (lane = key), keeps the running
// maximum and sum of its heads, and adds P V with lane = column.  Bound by
// latency (a few hundred keys a block); parts are cut so that short batches
// still fill the GPU, and joined by a second kernel.  Eight heads a warp are compiled
// in whatever the call has: dk = dv = 64 takes 199 registers, 128 and 128 spill 1160
// bytes (64 queries x 2048 slots: 50 us with 4 heads of 64, 319 with 32 of 128).
#include "rows.cuh"

namespace dsa {

constexpr int PF_WARPS = 4;
constexpr int PF_KEYS = 32;
constexpr int PF_HEADS = 8;  // heads per warp at most

DSA_DEV void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"((uint64_t)src) : "memory");
}

template <int DK, int DV>
struct PfSmem {
    static constexpr int KP = DK + 4, VP = DV + 4;  // row pitches (floats): 16-byte reads of 8 rows hit all banks
    float k[2][PF_KEYS * KP];
    float v[2][PF_KEYS * VP];
    int ok[2][PF_KEYS];
    float q[32 * DK];
};

template <int DK, int DV>
__global__ void __launch_bounds__(PF_WARPS * 32) attn_paged_f32_kernel(const PagedAttnArgs a, int vec) {
    extern __shared__ __align__(16) uint8_t pf_raw[];
    using Sm = PfSmem<DK, DV>;
    Sm& sm = *(Sm*)pf_raw;
    constexpr int NV = DV / 32;
    const int warp = (int)warp_id(), lane = (int)lane_id();
    next_grid();
    const int64_t t = blockIdx.x / (unsigned)a.splits;
    const int part = (int)(blockIdx.x - t * a.splits);
    const RowInfo ri = row_info_guess(a.sv, t, a.total_q);
    if (!ri.ok) {  // rows without a valid position are left as they were
        if (threadIdx.x == 0) report(a.st, DSA_ERR_INDEX, t);
        return;
    }
    // this part's keys or slots [lo, hi)
    const int64_t n = a.idx ? a.k_sel : ri.pos + 1;
    const int64_t per = ((n + PF_KEYS - 1) / PF_KEYS + a.splits - 1) / a.splits * PF_KEYS;
    const int64_t lo = min((int64_t)part * per, n), hi = min(lo + per, n);
    const int32_t* irow = a.idx ? a.idx + t * a.ld_idx : nullptr;
    const int tiles = (int)((hi - lo + PF_KEYS - 1) / PF_KEYS);

    for (int i = threadIdx.x; i < a.heads * DK; i += PF_WARPS * 32) {
        const int h = i / DK, c = i - h * DK;
        sm.q[i] = ((const float*)a.q)[t * a.q_stride_tok + h * a.q_stride_head + c];
    }
    // rows warp, warp + 4, ... of a tile: lane i < 8 looks up row warp + 4 i
    auto fetch = [&](int tile, int buf) {
        int64_t ko = 0, vo = 0;
        int have = 0;
        const int r = warp + PF_WARPS * (lane & 7);
        const int64_t j = lo + (int64_t)tile * PF_KEYS + r;
        if (j < hi) {
            int64_t s = j;
            if (irow) {
                const int32_t v = __ldg(irow + j);
                s = v;
                if (v >= ri.seqlen_k) {
                    if (lane < 8) report(a.st, DSA_ERR_INDEX, t);
                    s = -1;
                }
            }
            if (s >= 0) {
                const PageRef pr = page_of(a.pv, ri.b, s);
                have = pr.page >= 0;
                if (have) {
                    ko = pr.page * a.k_page_stride + (int64_t)pr.slot * a.k_stride;
                    vo = pr.page * a.v_page_stride + (int64_t)pr.slot * a.v_stride;
                } else if (lane < 8) {
                    report(a.st, DSA_ERR_INDEX, t);
                }
            }
        }
        if (lane < 8) sm.ok[buf][r] = have;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = warp + PF_WARPS * i;
            const int64_t k0 = __shfl_sync(0xffffffffu, ko, i), v0 = __shfl_sync(0xffffffffu, vo, i);
            float* kd = sm.k[buf] + row * Sm::KP;
            float* vd = sm.v[buf] + row * Sm::VP;
            if (__shfl_sync(0xffffffffu, have, i)) {
                const float *ks = (const float*)a.k + k0, *vs = (const float*)a.v + v0;
                if (vec) {
                    if (4 * lane < DK) cp_async16(smem_u32(kd + 4 * lane), ks + 4 * lane);
                    if (4 * lane < DV) cp_async16(smem_u32(vd + 4 * lane), vs + 4 * lane);
                } else {
                    for (int c = lane; c < DK; c += 32) cp_async4(smem_u32(kd + c), ks + c);
                    for (int c = lane; c < DV; c += 32) cp_async4(smem_u32(vd + c), vs + c);
                }
            } else {  // no row: zeros, so that a zero probability meets no stray NaN
                for (int c = lane; c < DV; c += 32) vd[c] = 0.f;
                for (int c = lane; c < DK; c += 32) kd[c] = 0.f;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    float m[PF_HEADS], l[PF_HEADS], o[PF_HEADS][NV];
#pragma unroll
    for (int i = 0; i < PF_HEADS; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < NV; ++c) o[i][c] = 0.f;
    }
    if (tiles > 0) fetch(0, 0);
    for (int tile = 0; tile < tiles; ++tile) {
        const int buf = tile & 1;
        if (tile + 1 < tiles) {
            fetch(tile + 1, buf ^ 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        const bool ok = sm.ok[buf][lane] != 0;
        const float* kr = sm.k[buf] + lane * Sm::KP;
#pragma unroll
        for (int i = 0; i < PF_HEADS; ++i) {
            const int h = warp + PF_WARPS * i;
            if (h >= a.heads) break;
            const float* qr = sm.q + h * DK;
            float d = 0.f;
#pragma unroll
            for (int c = 0; c < DK; c += 4) {
                const float4 kv = *(const float4*)(kr + c), qv = *(const float4*)(qr + c);
                d = fmaf(qv.x, kv.x, d);
                d = fmaf(qv.y, kv.y, d);
                d = fmaf(qv.z, kv.z, d);
                d = fmaf(qv.w, kv.w, d);
            }
            const float z = ok ? d * a.scale : -INFINITY;
            float mt = z;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
            if (mt > m[i]) {  // warp-uniform
                const float c = m[i] == -INFINITY ? 0.f : expf(m[i] - mt);
                l[i] *= c;
#pragma unroll
                for (int x = 0; x < NV; ++x) o[i][x] *= c;
                m[i] = mt;
            }
            // (a score of -inf adds nothing, also while there is no maximum; a NaN stays NaN)
            const float p = z == -INFINITY ? 0.f : expf(z - m[i]);
            float ps = p;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, x);
            l[i] += ps;
#pragma unroll
            for (int j = 0; j < PF_KEYS; ++j) {
                const float pj = __shfl_sync(0xffffffffu, p, j);
#pragma unroll
                for (int x = 0; x < NV; ++x) o[i][x] = fmaf(pj, sm.v[buf][j * Sm::VP + lane + 32 * x], o[i][x]);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < PF_HEADS; ++i) {
        const int h = warp + PF_WARPS * i;
        if (h >= a.heads) break;
        const float inv = l[i] != 0.f ? 1.0f / l[i] : 0.f;  // a NaN sum stays NaN
        const float lse = l[i] != 0.f ? m[i] + logf(l[i]) : -INFINITY;
        float* op;
        if (a.splits > 1) {
            const int64_t r = ((int64_t)blockIdx.x * a.heads + h);
            op = a.part_o + r * DV;
            if (lane == 0) a.part_lse[r] = lse;
        } else {
            op = (float*)a.out + t * a.out_stride_tok + h * a.out_stride_head;
            if (a.lse && lane == 0) a.lse[t * a.heads + h] = lse;
        }
#pragma unroll
        for (int x = 0; x < NV; ++x) op[lane + 32 * x] = o[i][x] * inv;
    }
}

// Joins the parts of a token's heads; one block a token, a warp a head.
__global__ void __launch_bounds__(128) attn_paged_f32_combine_kernel(const PagedAttnArgs a) {
    const int64_t t = blockIdx.x;
    const int lane = (int)lane_id();
    const bool ok = row_info_guess(a.sv, t, a.total_q).ok;
    grid_wait();
    if (!ok) return;  // left as it was
    for (int h = (int)warp_id(); h < a.heads; h += 4) {
        // lane p holds the weights of parts p and p + 32
        float z[2], m = -INFINITY;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int p = lane + 32 * i;
            z[i] = p < a.splits ? a.part_lse[(t * a.splits + p) * a.heads + h] : -INFINITY;
            m = fmaxf(m, z[i]);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        float w[2], l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i] = z[i] == -INFINITY ? 0.f : expf(z[i] - m);  // an empty part; NaN stays NaN
#pragma unroll 4
        for (int p = 0; p < a.splits; ++p) {
            const float wp = __shfl_sync(0xffffffffu, p < 32 ? w[0] : w[1], p & 31);
            const int64_t r = (t * a.splits + p) * a.heads + h;
            l += wp;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (lane + 32 * x < a.dv) o[x] = fmaf(wp, a.part_o[r * a.dv + lane + 32 * x], o[x]);
        }
        const float inv = l != 0.f ? 1.0f / l : 0.f;
        float* op = (float*)a.out + t * a.out_stride_tok + h * a.out_stride_head;
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (lane + 32 * x < a.dv) op[lane + 32 * x] = o[x] * inv;
        if (a.lse && lane == 0) a.lse[t * a.heads + h] = l != 0.f ? m + logf(l) : -INFINITY;
    }
}

template <int DK, int DV>
static bool pf_launch(const PagedAttnArgs& a, cudaStream_t s) {
    auto al = [](const void* p) { return ((uintptr_t)p & 15) == 0; };
    const int vec = al(a.k) && al(a.v) && a.k_stride % 4 == 0 && a.v_stride % 4 == 0 && a.k_page_stride % 4 == 0 &&
                    a.v_page_stride % 4 == 0;
    const int64_t grid = a.total_q * a.splits;
    if (grid >= ((int64_t)1 << 31)) return false;
    const int smem = (int)sizeof(PfSmem<DK, DV>);
    if (cudaFuncSetAttribute(attn_paged_f32_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
        return false;
    attn_paged_f32_kernel<DK, DV><<<(unsigned)grid, PF_WARPS * 32, smem, s>>>(a, vec);
    if (cudaGetLastError() != cudaSuccess) return false;
    return a.splits == 1 || launch_after(attn_paged_f32_combine_kernel, dim3((unsigned)a.total_q), dim3(128), s, a);
}

template <int DK>
static bool pf_launch_dv(const PagedAttnArgs& a, cudaStream_t s) {
    switch (a.dv) {
        case 32: return pf_launch<DK, 32>(a, s);
        case 64: return pf_launch<DK, 64>(a, s);
        case 96: return pf_launch<DK, 96>(a, s);
        case 128: return pf_launch<DK, 128>(a, s);
    }
    return false;
}

bool launch_paged_attn_f32(const PagedAttnArgs& a, cudaStream_t s) {
    if (a.total_q <= 0) return true;
    switch (a.dk) {
        case 32: return pf_launch_dv<32>(a, s);
        case 64: return pf_launch_dv<64>(a, s);
        case 96: return pf_launch_dv<96>(a, s);
        case 128: return pf_launch_dv<128>(a, s);
    }
    return false;
}

}  // namespace dsa
