// norm_rope.cu -- RMS norm of every head's row and the position rotation in
// one pass, and its gradients.
//
// Rows x[t, h, 0:dim] (heads may be 1, as for the shared KV row).  With
// n = norm_dim, r = 1/sqrt(mean(x[0:n]^2) + eps):
//     u_c = x_c r w_c (c < n),  u_c = x_c (c >= n)
//     (y_a, y_b) = (u_a cos - u_b sin, u_b cos + u_a sin)
// for every pair (a, b) of the rotated columns, y_c = u_c elsewhere; the
// angles are those of the token's position.  Backward, with g = the transposed
// rotation of dy and x^ = x r:
//     dx_c = r (g_c w_c - x^_c mean_n(g w x^)) (c < n),  dx_c = g_c (c >= n)
//     dw_c = sum over rows of g_c x^_c
//
// Both are bound by HBM: a row is read once and written once (backward: x and
// dy once, dx once); a group of 8 lanes (dim <= 256) or 32 lanes holds a row in
// registers as 16-byte chunks, so the norm's reduction and the rotation need
// no second read.  All arithmetic is fp32; the result is rounded once.  8192 x 128
// rows of 576 in bf16: 439 us, 0.84 of the copy bandwidth; the backward of 232K
// rows of 128 in bf16: 43 us, 0.64 (16 warps an SM at 128 registers).  The times
// beside the choices below are of graph replays (429 and 41.6 us for these two).
//
// dw is summed in a fixed order, whatever the launch: each lane sums its
// columns over its block's rows, the block's groups are added in order, and a
// second kernel adds the blocks' partial rows (in 64 bits).
#include "rows.cuh"

namespace dsa {

constexpr int NR_THREADS = 256;
constexpr int NR_WARPS = NR_THREADS / 32;

// Token t's position row of the cos | sin table, or false (reported once).
struct TokenPos {
    int64_t t = -1;
    bool ok = false;
    const float* cs = nullptr;
};
DSA_DEV void token_pos(TokenPos& tp, int64_t t, const NormRopeArgs& a) {
    const RowXform& ra = a.ra;
    if (t == tp.t) return;
    tp.t = t;
    const RowInfo ri = row_info_guess(a.sv, t, a.total_q);
    tp.ok = ri.ok && (ra.rope_dim == 0 || ri.pos < ra.rope_positions);
    if (!tp.ok) report(a.st, DSA_ERR_INDEX, t);
    tp.cs = tp.ok && ra.rope_dim ? ra.cos_sin + ri.pos * ra.rope_dim : nullptr;
}

// A lane group's walk over rows, N arrays' offsets with it: all by addition (a
// 64-bit division a row costs more than the row's arithmetic).
template <int N>
struct RowWalk {
    int64_t t;
    int h;
    int64_t off[N], head[N], wrap[N];  // elements: the row's offset; a head's; from a token's end to the next
};
template <int N>
DSA_DEV RowWalk<N> walk_from(int64_t r, int heads, const int64_t (&st)[N], const int64_t (&sh)[N]) {
    RowWalk<N> w;
    w.t = r / heads;
    w.h = (int)(r - w.t * heads);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        w.off[i] = w.t * st[i] + w.h * sh[i];
        w.head[i] = sh[i];
        w.wrap[i] = st[i] - heads * sh[i];
    }
    return w;
}
template <int N>
DSA_DEV void walk_on(RowWalk<N>& w, int n, int heads) {
    w.h += n;
#pragma unroll
    for (int i = 0; i < N; ++i) w.off[i] += n * w.head[i];
    while (w.h >= heads) {
        w.h -= heads;
        ++w.t;
#pragma unroll
        for (int i = 0; i < N; ++i) w.off[i] += w.wrap[i];
    }
}

template <class T, int G, int NC>
__global__ void __launch_bounds__(NR_THREADS, NC <= 3 ? 4 : 1) norm_rope_kernel(const NormRopeArgs a) {
    extern __shared__ __align__(16) float nr_sm[];
    constexpr int RPW = 32 / G;  // rows per warp and step
    const int lane = (int)lane_id(), gl = lane % G, sub = lane / G, warp = (int)warp_id();
    float* sm = nr_sm + (warp * RPW + sub) * a.ra.rope_dim;
    const int64_t rows = a.total_q * a.heads;
    const int64_t r0 = ((int64_t)blockIdx.x * NR_WARPS + warp) * a.rows_per_warp;
    const int n = (int)max(min(rows - r0, a.rows_per_warp), (int64_t)0);  // rows of this warp
    const int64_t st[2] = {a.x_stride_tok, a.y_stride_tok}, sh[2] = {a.x_stride_head, a.y_stride_head};
    RowWalk<2> w = walk_from(r0 + sub, a.heads, st, sh);
    TokenPos tp;
    // One row at a time: many small warps hide the loads better than rows in flight
    // (a row ahead: 120 registers, 565 us for 8192 x 128 x 576 in bf16 against 427).
    for (int i = sub; i < n + sub; i += RPW) {
        bool live = i < n;
        Raw8<T> cur[NC];
        load_row<T, G, NC>(cur, (const T*)a.x + w.off[0], a.dim, gl, live);
        if (live) {
            token_pos(tp, w.t, a);
            live = tp.ok;
        }
        row_forward<T, G, NC>(cur, (T*)a.y + w.off[1], a.ra, a.dim, tp.cs, gl, live, sm);
        walk_on(w, RPW, a.heads);
    }
}

template <class T>
__global__ void __launch_bounds__(NR_THREADS) norm_rope_scalar_kernel(const NormRopeArgs a) {
    const int64_t rows = a.total_q * a.heads;
    const int64_t step = (int64_t)gridDim.x * NR_WARPS;
    TokenPos tp;
    for (int64_t r = (int64_t)blockIdx.x * NR_WARPS + warp_id(); r < rows; r += step) {
        const int64_t t = r / a.heads, h = r - t * a.heads;
        token_pos(tp, t, a);
        if (!tp.ok) continue;
        row_forward_scalar<T>((const T*)a.x + t * a.x_stride_tok + h * a.x_stride_head,
                              (T*)a.y + t * a.y_stride_tok + h * a.y_stride_head, a.ra, a.dim, tp.cs, (int)lane_id());
    }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
template <class T, int G, int NC>
__global__ void __launch_bounds__(NR_THREADS, NC <= 3 ? 2 : 1) norm_rope_bwd_kernel(const NormRopeArgs a) {
    extern __shared__ __align__(16) float nr_sm[];
    constexpr int RPW = 32 / G;
    const int lane = (int)lane_id(), gl = lane % G, sub = lane / G, warp = (int)warp_id();
    float* sm = nr_sm + (warp * RPW + sub) * a.ra.rope_dim;
    const int n = a.ra.norm_dim;
    next_grid();
    const int64_t rows = a.total_q * a.heads;
    float acc[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
    const int64_t r0 = ((int64_t)blockIdx.x * NR_WARPS + warp) * a.rows_per_warp;
    const int count = (int)max(min(rows - r0, a.rows_per_warp), (int64_t)0);  // rows of this warp
    const int64_t st[3] = {a.x_stride_tok, a.dy_stride_tok, a.y_stride_tok};
    const int64_t sh[3] = {a.x_stride_head, a.dy_stride_head, a.y_stride_head};
    RowWalk<3> w = walk_from(r0 + sub, a.heads, st, sh);
    const float inv_n = n > 0 ? 1.0f / (float)n : 0.f;
    // the weight stays in registers where they allow
    constexpr bool KEEP_W = NC <= 2;
    float wt[KEEP_W ? NC : 1][8];
    if (KEEP_W)
#pragma unroll
        for (int i = 0; i < (KEEP_W ? NC : 1); ++i) {
            const int c = (gl + G * i) * 8;
#pragma unroll
            for (int x = 0; x < 8; ++x) wt[i][x] = 1.f;
            if (a.ra.weight && c < n) load_weight8(a.ra.weight, c, wt[i]);
        }
    // The next row is in flight while this one is worked on where that does not
    // spill.  In bf16 without and with, us: 232K heads of 128 51, 41; 116K heads of 192
    // 70, 58 and of 256 72, 62; 29K rows of 1024 70, 60 (one block an SM either way).
    // 576 columns in fp32 spill: 14, 21.
    constexpr bool AHEAD = sizeof(T) == 2 ? NC <= 2 || NC == 4 : NC == 1;
    Raw8<T> cx[NC], cg[NC];
    auto fetch = [&](bool have) {
        load_row<T, G, NC>(cg, (const T*)a.dy + w.off[1], a.dim, gl, have);
        load_row<T, G, NC>(cx, (const T*)a.x + w.off[0], n, gl, have);
    };
    if (AHEAD) fetch(sub < count);
    TokenPos tp;
    for (int i0 = sub; i0 < count + sub; i0 += RPW) {
        bool live = i0 < count;
        if (live) {
            token_pos(tp, w.t, a);
            live = tp.ok;
        }
        T* dx = (T*)a.y + w.off[2];
        if (!AHEAD) fetch(live);
        float g[NC][8], xv[NC][8];
#pragma unroll
        for (int i = 0; i < NC; ++i) unpack8(cg[i], g[i]), unpack8(cx[i], xv[i]);
        if (AHEAD && !live) {  // a token without a position adds nothing, whatever its rows hold
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) g[i][e] = xv[i][e] = 0.f;
        }
        walk_on(w, RPW, a.heads);
        if (AHEAD) fetch(i0 + RPW < count);
        if (a.ra.rope_dim > 0) rotate_chunks<G, NC>(g, a.ra, tp.cs, gl, -1.f, live, sm);
        if (n > 0) {
            float ss = 0.f, dot = 0.f;
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if ((gl + G * i) * 8 < n)
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(xv[i][e], xv[i][e], ss);
            ss = group_sum<G>(ss);
            const float rstd = live ? row_rstd(fmaf(ss, inv_n, a.ra.eps)) : 0.f;  // no row: zeros throughout
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = (gl + G * i) * 8;
                if (c < n) {
                    float(&wc)[8] = wt[KEEP_W ? i : 0];
                    if (!KEEP_W && a.ra.weight) load_weight8(a.ra.weight, c, wc);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        xv[i][e] *= rstd;  // x^
                        acc[i][e] = fmaf(g[i][e], xv[i][e], acc[i][e]);
                        if (KEEP_W || a.ra.weight) g[i][e] *= wc[e];
                        dot = fmaf(g[i][e], xv[i][e], dot);
                    }
                }
            }
            const float k = rstd * (group_sum<G>(dot) * inv_n);  // r times the mean of g w x^
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if ((gl + G * i) * 8 < n)
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[i][e] = fmaf(-xv[i][e], k, rstd * g[i][e]);
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (gl + G * i) * 8;
            if (live && c < a.dim) store8(dx + c, g[i]);
        }
    }
    if (!a.dw_part) return;
    // the block's groups, added in order; each warp's RPW row groups first
    __syncthreads();
    float* red = nr_sm;  // [NR_WARPS][n]
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = (gl + G * i) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = acc[i][e];
#pragma unroll
            for (int o = 16; o >= G; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            acc[i][e] = v;
        }
        if (sub == 0 && c < n) store8(red + warp * n + c, acc[i]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < n; c += NR_THREADS) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < NR_WARPS; ++w) v += red[w * n + c];
        a.dw_part[(int64_t)blockIdx.x * n + c] = v;
    }
}

template <class T>
__global__ void __launch_bounds__(NR_THREADS) norm_rope_bwd_scalar_kernel(const NormRopeArgs a) {
    extern __shared__ __align__(16) float nr_sm[];
    const int lane = (int)lane_id(), warp = (int)warp_id(), n = a.ra.norm_dim;
    const RowXform& ra = a.ra;
    const int h = ra.rope_dim >> 1;
    const float inv_n = n > 0 ? 1.0f / (float)n : 0.f;
    next_grid();
    float* acc = nr_sm + warp * n;
    for (int c = lane; c < n; c += 32) acc[c] = 0.f;
    const int64_t rows = a.total_q * a.heads;
    const int64_t step = (int64_t)gridDim.x * NR_WARPS;
    TokenPos tp;
    for (int64_t r = (int64_t)blockIdx.x * NR_WARPS + warp; r < rows; r += step) {
        const int64_t t = r / a.heads, hd = r - t * a.heads;
        token_pos(tp, t, a);
        if (!tp.ok) continue;
        const T* x = (const T*)a.x + t * a.x_stride_tok + hd * a.x_stride_head;
        const T* dy = (const T*)a.dy + t * a.dy_stride_tok + hd * a.dy_stride_head;
        T* dx = (T*)a.y + t * a.y_stride_tok + hd * a.y_stride_head;
        auto grad = [&](int c) {  // the transposed rotation of dy at column c
            const int o = c - ra.rope_begin;
            if (o < 0 || o >= ra.rope_dim) return load1(dy + c);
            const int j = ra.interleaved ? o >> 1 : (o < h ? o : o - h);
            const bool first = ra.interleaved ? (o & 1) == 0 : o < h;
            const int d = ra.interleaved ? 1 : h;
            const float p = load1(dy + (first ? c + d : c - d)), co = __ldg(tp.cs + j), si = __ldg(tp.cs + h + j);
            return first ? load1(dy + c) * co + p * si : load1(dy + c) * co - p * si;
        };
        float rstd = 0.f, k = 0.f;
        if (n > 0) {
            float ss = 0.f, dot = 0.f;
            for (int c = lane; c < n; c += 32) {
                const float v = load1(x + c), w = ra.weight ? __ldg(ra.weight + c) : 1.f;
                ss = fmaf(v, v, ss);
                dot = fmaf(grad(c) * w, v, dot);
            }
            ss = group_sum<32>(ss);
            dot = group_sum<32>(dot);
            rstd = row_rstd(fmaf(ss, inv_n, ra.eps));
            k = dot * rstd * inv_n;
        }
        for (int c = lane; c < a.dim; c += 32) {
            const float g = grad(c);
            if (c < n) {
                const float xh = load1(x + c) * rstd, w = ra.weight ? __ldg(ra.weight + c) : 1.f;
                acc[c] = fmaf(g, xh, acc[c]);  // column c of a warp is lane c % 32's alone
                store1(dx + c, rstd * (g * w - xh * k));
            } else {
                store1(dx + c, g);
            }
        }
    }
    if (!a.dw_part) return;
    __syncthreads();
    for (int c = threadIdx.x; c < n; c += NR_THREADS) {
        float v = 0.f;
        for (int w = 0; w < NR_WARPS; ++w) v += nr_sm[w * n + c];
        a.dw_part[(int64_t)blockIdx.x * n + c] = v;
    }
}

// dw[c] = sum over the blocks' partial rows, in a fixed order: 32 strided sums
// in 64 bits, then those in order.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* part, int blocks, int n,
                                                            float* __restrict__ dw) {
    __shared__ double sm[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    double v = 0.0;
    grid_wait();
    if (c < n) {
#pragma unroll 5
        for (int b = threadIdx.y; b < blocks; b += 32) v += (double)part[(int64_t)b * n + c];
    }
    sm[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && c < n) {
        v = 0.0;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += sm[i][threadIdx.x];
        dw[c] = (float)v;
    }
}

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------
template <class T, int G, int NC>
static bool nr_launch(NormRopeArgs a, bool bwd, int blocks, cudaStream_t s) {
    const int groups = NR_THREADS / G;
    const int d = rope_in_lane<G>(a.ra);
    size_t smem = a.ra.interleaved || (d > 0 && d < NC && NC > 1) ? 0 : (size_t)groups * a.ra.rope_dim * 4;
    if (bwd && a.dw_part && smem < (size_t)NR_WARPS * a.ra.norm_dim * 4) smem = (size_t)NR_WARPS * a.ra.norm_dim * 4;
    const void* fn = bwd ? (const void*)norm_rope_bwd_kernel<T, G, NC> : (const void*)norm_rope_kernel<T, G, NC>;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return false;
    if (bwd) norm_rope_bwd_kernel<T, G, NC><<<blocks, NR_THREADS, smem, s>>>(a);
    else norm_rope_kernel<T, G, NC><<<blocks, NR_THREADS, smem, s>>>(a);
    return cudaGetLastError() == cudaSuccess;
}

template <class T>
static bool nr_launch_dim(const NormRopeArgs& a, bool bwd, int blocks, cudaStream_t s) {
    if (a.dim <= 64) return nr_launch<T, 8, 1>(a, bwd, blocks, s);
    if (a.dim <= 128) return nr_launch<T, 8, 2>(a, bwd, blocks, s);
    if (a.dim <= 256) return nr_launch<T, 8, 4>(a, bwd, blocks, s);
    if (a.dim <= 512) return nr_launch<T, 32, 2>(a, bwd, blocks, s);
    if (a.dim <= 768) return nr_launch<T, 32, 3>(a, bwd, blocks, s);
    if (a.dim <= 1024) return nr_launch<T, 32, 4>(a, bwd, blocks, s);
    return nr_launch<T, 32, 8>(a, bwd, blocks, s);
}

static bool nr_chunked(const NormRopeArgs& a, bool bf16, bool bwd) {
    const int64_t e = bf16 ? 8 : 4;  // elements of 16 bytes
    auto al = [](const void* p) { return ((uintptr_t)p & 15) == 0; };
    bool ok = row_xform_chunked(a.ra, a.dim) && al(a.x) && al(a.y) && a.x_stride_tok % e == 0 &&
              a.x_stride_head % e == 0 && a.y_stride_tok % e == 0 && a.y_stride_head % e == 0;
    if (bwd) ok = ok && al(a.dy) && a.dy_stride_tok % e == 0 && a.dy_stride_head % e == 0;
    return ok;
}

// Blocks of the backward: enough warps to fill the GPU, and no more, because
// each block adds one partial row to dw.
int norm_rope_bwd_blocks(int64_t rows) {
    const int64_t want = (rows + NR_WARPS - 1) / NR_WARPS;
    return (int)(want < kNormRopeBwdBlocks ? (want > 0 ? want : 1) : kNormRopeBwdBlocks);
}

bool launch_norm_rope(const NormRopeArgs& in, bool bf16, cudaStream_t s) {
    NormRopeArgs a = in;
    const int64_t rows = a.total_q * a.heads;
    if (rows <= 0) return true;
    if (!nr_chunked(a, bf16, false)) {
        const int64_t blocks = (rows + NR_WARPS - 1) / NR_WARPS;
        const unsigned g = (unsigned)(blocks < 148 * 16 ? blocks : 148 * 16);
        if (bf16) norm_rope_scalar_kernel<__nv_bfloat16><<<g, NR_THREADS, 0, s>>>(a);
        else norm_rope_scalar_kernel<float><<<g, NR_THREADS, 0, s>>>(a);
        return cudaGetLastError() == cudaSuccess;
    }
    const int rpw = a.dim <= 256 ? 4 : 1;
    int64_t per = (rows + (int64_t)148 * 64 * 4 - 1) / ((int64_t)148 * 64 * 4);  // rows a warp: a few waves of warps
    if (per > 16) per = 16;
    a.rows_per_warp = (int)((per + rpw - 1) / rpw * rpw);
    const int64_t blocks = (rows + (int64_t)a.rows_per_warp * NR_WARPS - 1) / ((int64_t)a.rows_per_warp * NR_WARPS);
    if (blocks >= ((int64_t)1 << 31)) return false;
    return bf16 ? nr_launch_dim<__nv_bfloat16>(a, false, (int)blocks, s) : nr_launch_dim<float>(a, false, (int)blocks, s);
}

bool launch_norm_rope_bwd(const NormRopeArgs& in, bool bf16, float* dw, cudaStream_t s) {
    NormRopeArgs a = in;
    const int64_t rows = a.total_q * a.heads;
    const int n = a.ra.norm_dim;
    if (rows <= 0) return !dw || n == 0 || cudaMemsetAsync(dw, 0, (size_t)n * 4, s) == cudaSuccess;
    int blocks = norm_rope_bwd_blocks(rows);
    if (!dw || n == 0) a.dw_part = nullptr;
    bool ok;
    if (!nr_chunked(a, bf16, true)) {
        const size_t smem = (size_t)NR_WARPS * n * 4;
        const void* fn = bf16 ? (const void*)norm_rope_bwd_scalar_kernel<__nv_bfloat16>
                              : (const void*)norm_rope_bwd_scalar_kernel<float>;
        if (smem > 48 * 1024 &&
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
            return false;
        if (bf16) norm_rope_bwd_scalar_kernel<__nv_bfloat16><<<blocks, NR_THREADS, smem, s>>>(a);
        else norm_rope_bwd_scalar_kernel<float><<<blocks, NR_THREADS, smem, s>>>(a);
        ok = cudaGetLastError() == cudaSuccess;
    } else {
        const int rpw = a.dim <= 256 ? 4 : 1;
        const int64_t warps = (int64_t)blocks * NR_WARPS;
        const int64_t per = (rows + warps - 1) / warps;
        a.rows_per_warp = (per + rpw - 1) / rpw * rpw;
        ok = bf16 ? nr_launch_dim<__nv_bfloat16>(a, true, blocks, s) : nr_launch_dim<float>(a, true, blocks, s);
    }
    if (!ok || !a.dw_part) return ok;
    return launch_after(norm_rope_dw_kernel, dim3((n + 31) / 32), dim3(32, 32), s, (const float*)a.dw_part, blocks, n, dw);
}

}  // namespace dsa
