// cache_append.cu -- append a step's new tokens to the paged cache: the KV row
// (RMS norm of its leading columns, rotation of its rope columns, one rounding
// to the pool's type) and the indexer key (norm, rotation, and for an FP8 pool
// the e4m3 codes with one fp32 scale per token, amax / 448).
//
// One warp per token, its row and key in registers (a warp for each of the two
// looks the position up twice: graph replays 14.6 us against 13.0 for 9154 tokens).
// Bound by latency: a decode step moves a few hundred KB; a prefill chunk's warps
// each wait for the sequence, the page and the row in turn (27 MB in 15 us, 0.28 of
// the copy bandwidth).
//
// The indexer key is computed in 64 bits.  Its codes are a rounding to 4
// significant bits: an fp32 error of 1e-7 moves about one value in a million
// across a rounding border, a change of up to 1/16 of that value, and the same
// token appended in another batch must give the same code.  At 128 columns a
// token the fp64 work (one division a column) hides behind the loads.  The
// 64-bit quotient is brought to fp32 by rounding to odd, so that the following
// rounding to e4m3 is that of the quotient itself (no double rounding).
#include <cuda_fp8.h>

#include "rows.cuh"

namespace dsa {

constexpr int AP_WARPS = 4;

DSA_DEV double warp_sum_f64(double x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
DSA_DEV double warp_max_f64(double x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmax(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

DSA_DEV uint32_t e4m3_of(double q) {
    float f = __double2float_rz(q);
    if ((double)f != q) f = __uint_as_float(__float_as_uint(f) | 1u);  // odd: never on a border of e4m3
    return (uint32_t)__nv_cvt_float_to_fp8(f, __NV_SATFINITE, __NV_E4M3);
}

// The indexer key of one token by one warp: lane l holds columns 4l..4l+3.
DSA_DEV void append_key(const AppendArgs& a, const float (&x)[4], const float* __restrict__ cs, const PageRef& pr, int lane,
                        double* sm) {
    const RowXform& ra = a.idx_row;
    double v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (double)x[e];
    if (ra.norm_dim > 0) {
        double ss = 0.0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (4 * lane + e < ra.norm_dim) ss += v[e] * v[e];
        const double rstd = 1.0 / sqrt(warp_sum_f64(ss) / (double)ra.norm_dim + (double)ra.eps);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = 4 * lane + e;
            if (c < ra.norm_dim) v[e] *= ra.weight ? rstd * (double)__ldg(ra.weight + c) : rstd;
        }
    }
    if (ra.rope_dim > 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sm[4 * lane + e] = v[e];
        __syncwarp();
        const int h = ra.rope_dim >> 1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = 4 * lane + e, o = c - ra.rope_begin;
            if (o >= 0 && o < ra.rope_dim) {
                const int j = ra.interleaved ? o >> 1 : (o < h ? o : o - h);
                const bool first = ra.interleaved ? (o & 1) == 0 : o < h;
                const int d = ra.interleaved ? 1 : h;
                const double p = sm[first ? c + d : c - d], co = (double)__ldg(cs + j), si = (double)__ldg(cs + h + j);
                v[e] = first ? v[e] * co - p * si : v[e] * co + p * si;
            }
        }
    }
    const int64_t row = pr.slot;
    if (a.idx_dtype == DSA_F32) {
        float* y = (float*)a.idx + pr.page * a.idx_page_stride + row * 128 + 4 * lane;
        *(float4*)y = make_float4((float)v[0], (float)v[1], (float)v[2], (float)v[3]);
        return;
    }
    const double amax = warp_max_f64(fmax(fmax(fabs(v[0]), fabs(v[1])), fmax(fabs(v[2]), fabs(v[3]))));
    float sc = (float)(amax / 448.0);
    if (!(sc > 0.f)) sc = 1.f;  // an all-zero key
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) w |= e4m3_of(v[e] / (double)sc) << (8 * e);
    *(uint32_t*)((uint8_t*)a.idx + pr.page * a.idx_page_stride + row * 128 + 4 * lane) = w;
    if (lane == 0) a.idx_scale[pr.page * a.scale_page_stride + row] = sc;
}

// NC > 0: KV rows of at most NC * 256 columns in chunks; NC = 0: scalar.
template <class T, int NC>
__global__ void __launch_bounds__(AP_WARPS * 32) cache_append_kernel(const AppendArgs a) {
    extern __shared__ __align__(16) uint8_t ap_sm[];
    const int lane = (int)lane_id(), warp = (int)warp_id();
    const int64_t t = (int64_t)blockIdx.x * AP_WARPS + warp;
    if (t >= a.total_q) return;
    // the token's row first: its place takes three or more dependent loads
    const T* x = (const T*)a.kv_new + t * a.kv_new_stride;
    Raw8<T> row[NC > 0 ? NC : 1];
    float kx[4];
    if (a.idx_new) {
#pragma unroll
        for (int e = 0; e < 4; ++e) kx[e] = load1((const T*)a.idx_new + t * a.idx_new_stride + 4 * lane + e);
    }
    if constexpr (NC > 0) load_row<T, 32, NC>(row, x, a.dim, lane, a.kv_new != nullptr);
    const RowInfo ri = row_info_guess(a.sv, t, a.total_q);
    PageRef pr;
    pr.page = -1;
    pr.slot = 0;
    // (a table that a part without rotation does not read has no end)
    bool ok = ri.ok;
    if (a.kv_new && a.kv_row.rope_dim) ok = ok && ri.pos < a.kv_row.rope_positions;
    if (a.idx_new && a.idx_row.rope_dim) ok = ok && ri.pos < a.idx_row.rope_positions;
    if (ok) pr = page_of(a.pv, ri.b, ri.pos);
    if (!ok || pr.page < 0) {
        if (lane == 0) report(a.st, DSA_ERR_INDEX, t);
        return;
    }
    auto angles = [&](const RowXform& ra) { return ra.rope_dim ? ra.cos_sin + ri.pos * ra.rope_dim : nullptr; };
    uint8_t* sm = ap_sm + warp * a.warp_smem;
    if (a.idx_new) append_key(a, kx, angles(a.idx_row), pr, lane, (double*)sm);
    if (!a.kv_new) return;
    __syncwarp();
    const RowXform& ra = a.kv_row;
    const float* cs = angles(ra);
    T* y = (T*)a.kv + pr.page * a.kv_page_stride + (int64_t)pr.slot * a.kv_stride;
    if constexpr (NC > 0) {
        row_forward<T, 32, NC>(row, y, ra, a.dim, cs, lane, true, (float*)sm);
    } else row_forward_scalar<T>(x, y, ra, a.dim, cs, lane);
}

template <class T, int NC>
static bool ap_launch(const AppendArgs& a, cudaStream_t s) {
    const int64_t blocks = (a.total_q + AP_WARPS - 1) / AP_WARPS;
    if (blocks >= ((int64_t)1 << 31)) return false;
    cache_append_kernel<T, NC><<<(unsigned)blocks, AP_WARPS * 32, AP_WARPS * a.warp_smem, s>>>(a);
    return cudaGetLastError() == cudaSuccess;
}

template <class T>
static bool ap_launch_dim(const AppendArgs& a, bool chunked, cudaStream_t s) {
    if (!chunked) return ap_launch<T, 0>(a, s);
    if (a.dim <= 256) return ap_launch<T, 1>(a, s);
    if (a.dim <= 768) return ap_launch<T, 3>(a, s);
    return ap_launch<T, 8>(a, s);
}

bool launch_cache_append(const AppendArgs& in, bool bf16, cudaStream_t s) {
    AppendArgs a = in;
    if (a.total_q <= 0) return true;
    const int64_t e = bf16 ? 8 : 4;
    auto al = [](const void* p) { return ((uintptr_t)p & 15) == 0; };
    const bool chunked = row_xform_chunked(a.kv_row, a.dim) && al(a.kv_new) && al(a.kv) && a.kv_new_stride % e == 0 &&
                         a.kv_stride % e == 0 && a.kv_page_stride % e == 0;
    // per warp: the key's 128 doubles, or the half-split exchange of the KV row
    a.warp_smem = 128 * 8;
    if (chunked && !a.kv_row.interleaved && a.kv_row.rope_dim * 4 > a.warp_smem) a.warp_smem = a.kv_row.rope_dim * 4;
    return bf16 ? ap_launch_dim<__nv_bfloat16>(a, chunked, s) : ap_launch_dim<float>(a, chunked, s);
}

}  // namespace dsa
