// rows.cuh -- the per-row transform of queries and keys (RMS norm over the
// leading columns, then the position rotation of a column range), shared by
// the query/key transform (norm_rope.cu) and the paged-cache append
// (cache_append.cu), and the lookup of a cache row through the page table.
#pragma once
#include "dsa_kernels.h"

namespace dsa {

// ---------------------------------------------------------------------------
// A kernel that starts while the one before it on the stream runs (which allows
// it by next_grid()): every block calls grid_wait(), before it reads what that one
// wrote and in any case before it leaves.
// ---------------------------------------------------------------------------
DSA_DEV void next_grid() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
DSA_DEV void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <class... P, class... A>
bool launch_after(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, (P)args...) == cudaSuccess;
}

// row_info of token t of total_q, after a first guess: sequences of equal length
// (a decode batch) need no search, whose every step waits for a load.
DSA_DEV RowInfo row_info_guess(const SeqView& sv, int64_t t, int64_t total_q) {
    const int b = min(max((int)((float)t * ((float)sv.batch / (float)total_q)), 0), sv.batch - 1);
    const int64_t q0 = __ldg(sv.cu_q + b), q1 = __ldg(sv.cu_q + b + 1), k0 = __ldg(sv.cu_k + b), k1 = __ldg(sv.cu_k + b + 1);
    if (t < q0 || t >= q1) return row_info(sv, t);
    RowInfo r;
    r.b = b;
    r.key_base = k0;
    r.seqlen_k = k1 - k0;
    r.pos = (k1 - k0) - (q1 - q0) + (t - q0);
    r.ok = r.pos >= 0 && r.pos < r.seqlen_k;
    return r;
}

// Records the first of the tokens [first, end) that no sequence holds, for kernels
// that walk over sequences and would pass it by.
DSA_DEV void report_no_sequence(const SeqView& sv, int64_t first, int64_t end, StatusHdr* st) {
    const int64_t lo = __ldg(sv.cu_q), hi = __ldg(sv.cu_q + sv.batch);
    if (first < min(lo, end)) report(st, DSA_ERR_INDEX, first);
    else if (end > max(hi, first)) report(st, DSA_ERR_INDEX, max(hi, first));
}

// ---------------------------------------------------------------------------
// Page table: the pool row of a sequence's position.
// ---------------------------------------------------------------------------
struct PageRef {
    int64_t page;  // -1: no valid page
    int32_t slot;  // row inside the page
};
DSA_DEV void page_split(const PageView& pv, uint32_t s, uint32_t& p, uint32_t& o) {  // s = p * page_size + o
    if (pv.shift >= 0) {
        p = s >> pv.shift;
        o = s & (uint32_t)(pv.page_size - 1);
    } else {
        p = s / (uint32_t)pv.page_size;
        o = s - p * (uint32_t)pv.page_size;
    }
}
DSA_DEV PageRef page_of(const PageView& pv, int b, int64_t s) {
    uint32_t p, o;
    page_split(pv, (uint32_t)s, p, o);
    PageRef r;
    r.slot = (int32_t)o;
    r.page = (int64_t)p < pv.ld_table ? (int64_t)__ldg(pv.table + b * pv.ld_table + p) : -1;
    if (r.page >= pv.num_pages || r.page < 0) r.page = -1;
    return r;
}

// ---------------------------------------------------------------------------
// 8 consecutive elements (two 16-byte accesses for fp32, one for bf16)
// ---------------------------------------------------------------------------
DSA_DEV void load8(const float* p, float (&v)[8]) {
    const float4 a = *(const float4*)p, b = *(const float4*)(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
DSA_DEV void store8(float* p, const float (&v)[8]) {
    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
    *(float4*)(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
DSA_DEV void store8(__nv_bfloat16* p, const float (&v)[8]) {
    *(uint4*)p = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
DSA_DEV float load1(const float* p) { return *p; }
DSA_DEV float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
DSA_DEV void store1(float* p, float v) { *p = v; }
DSA_DEV void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <int G>
DSA_DEV float group_sum(float x) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// A row's reciprocal root mean square, from mean square + eps.  rsqrtf is within 2
// ulp; 1 / sqrtf measured 43.6 us against 41.6 (graph replays, backward of 232K heads
// of 128 in bf16) and 33.8 against 33.1 (forward).  Every path takes this one, so that a row's
// alignment does not change it.
DSA_DEV float row_rstd(float ms) { return rsqrtf(ms); }

// Rotate the chunks of this row that lie in the rotated columns, in place;
// sgn = 1 rotates by the position's angles, -1 back (the transpose).
// Interleaved pairs lie inside an 8-column chunk.  Half-split pairs are
// rope_dim / 2 columns apart: in another chunk of the same lane where that is
// a multiple of 8 G columns (heads of 128 and 256 columns, rotated whole), else in
// another lane's chunk, and the rotated columns pass through `sm`, this row
// group's rope_dim floats of shared memory.  All lanes of the warp call this
// together.
template <int G, int NC, int D>
DSA_DEV void rotate_in_lane(float (&v)[NC][8], const RowXform& ra, const float* __restrict__ cs, int gl, float sgn, bool live) {
    const int h = ra.rope_dim >> 1;
#pragma unroll
    for (int i = 0; i + D < NC; ++i) {
        const int o = (gl + G * i) * 8 - ra.rope_begin;  // the partner is at o + h
        if (live && o >= 0 && o < h) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float4 c4 = __ldg((const float4*)(cs + o) + x), s4 = __ldg((const float4*)(cs + h + o) + x);
                const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x * sgn, s4.y * sgn, s4.z * sgn, s4.w * sgn};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a = v[i][4 * x + e], b = v[i + D][4 * x + e];
                    v[i][4 * x + e] = a * c[e] - b * s[e];
                    v[i + D][4 * x + e] = b * c[e] + a * s[e];
                }
            }
        }
    }
}
// chunks between the halves of a pair, 0: in another lane
template <int G>
__host__ __device__ inline int rope_in_lane(const RowXform& ra) {
    const int h = ra.rope_dim >> 1;
    return !ra.interleaved && (h == 8 * G || h == 16 * G) ? h / (8 * G) : 0;
}
template <int G, int NC>
DSA_DEV void rotate_chunks(float (&v)[NC][8], const RowXform& ra, const float* __restrict__ cs, int gl, float sgn, bool live,
                           float* sm) {
    const int h = ra.rope_dim >> 1;
    if (ra.interleaved) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int o = (gl + G * i) * 8 - ra.rope_begin;
            if (live && o >= 0 && o < ra.rope_dim) {
                const float4 c = __ldg((const float4*)(cs + (o >> 1)));
                const float4 s = __ldg((const float4*)(cs + h + (o >> 1)));
                const float cc[4] = {c.x, c.y, c.z, c.w};
                const float ss[4] = {s.x * sgn, s.y * sgn, s.z * sgn, s.w * sgn};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a = v[i][2 * e], b = v[i][2 * e + 1];
                    v[i][2 * e] = a * cc[e] - b * ss[e];
                    v[i][2 * e + 1] = b * cc[e] + a * ss[e];
                }
            }
        }
        return;
    }
    if constexpr (NC > 1) {
        const int d = rope_in_lane<G>(ra);
        if (d == 1) return rotate_in_lane<G, NC, 1>(v, ra, cs, gl, sgn, live);
        if (NC > 2 && d == 2) return rotate_in_lane<G, NC, 2>(v, ra, cs, gl, sgn, live);
    }
    __syncwarp();  // the previous row's reads of sm are done
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int o = (gl + G * i) * 8 - ra.rope_begin;
        if (live && o >= 0 && o < ra.rope_dim) store8(sm + o, v[i]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int o = (gl + G * i) * 8 - ra.rope_begin;
        if (live && o >= 0 && o < ra.rope_dim) {
            const bool lo = o < h;
            const int j = lo ? o : o - h;
            float p[8], c[8], s[8];
            load8(sm + (lo ? o + h : o - h), p);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float4 c4 = __ldg((const float4*)(cs + j) + e), s4 = __ldg((const float4*)(cs + h + j) + e);
                c[4 * e] = c4.x, c[4 * e + 1] = c4.y, c[4 * e + 2] = c4.z, c[4 * e + 3] = c4.w;
                s[4 * e] = s4.x, s[4 * e + 1] = s4.y, s[4 * e + 2] = s4.z, s[4 * e + 3] = s4.w;
            }
            const float sg = lo ? -sgn : sgn;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * c[e] + sg * (p[e] * s[e]);
        }
    }
}

// A row as loaded: this lane's chunks gl, gl + G, ... of 8 columns each,
// unconverted, so that the next row can be in flight while one is worked on.
template <class T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
};
template <>
struct Raw8<float> {
    float4 a, b;
};
DSA_DEV void unpack8(const Raw8<float>& r, float (&v)[8]) {
    v[0] = r.a.x, v[1] = r.a.y, v[2] = r.a.z, v[3] = r.a.w;
    v[4] = r.b.x, v[5] = r.b.y, v[6] = r.b.z, v[7] = r.b.w;
}
DSA_DEV void unpack8(const Raw8<__nv_bfloat16>& r, float (&v)[8]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
// columns [0, cols) of row x (zeros past them, or everywhere if !have)
template <class T, int G, int NC>
DSA_DEV void load_row(Raw8<T> (&r)[NC], const T* x, int cols, int gl, bool have) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = (gl + G * i) * 8;
        r[i] = Raw8<T>{};
        if (have && c < cols) r[i] = *(const Raw8<T>*)(x + c);
    }
}
DSA_DEV void load_weight8(const float* __restrict__ weight, int c, float (&w)[8]) {
    const float4 a = __ldg((const float4*)(weight + c)), b = __ldg((const float4*)(weight + c) + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}

// One loaded row by a group of G lanes: norm, weight, rotation, one rounding to
// T, stored to y if live.  cs: the position's cos | sin row.
template <class T, int G, int NC>
DSA_DEV void row_forward(const Raw8<T> (&r)[NC], T* y, const RowXform& ra, int dim, const float* __restrict__ cs, int gl,
                         bool live, float* sm) {
    float v[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) unpack8(r[i], v[i]);
    if (ra.norm_dim > 0) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if ((gl + G * i) * 8 < ra.norm_dim)
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
        ss = group_sum<G>(ss);
        const float rstd = row_rstd(ss / (float)ra.norm_dim + ra.eps);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = (gl + G * i) * 8;
            if (c < ra.norm_dim) {
                float w[8];
                if (ra.weight) load_weight8(ra.weight, c, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = ra.weight ? v[i][e] * rstd * w[e] : v[i][e] * rstd;
            }
        }
    }
    if (ra.rope_dim > 0) rotate_chunks<G, NC>(v, ra, cs, gl, 1.f, live, sm);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = (gl + G * i) * 8;
        if (live && c < dim) store8(y + c, v[i]);
    }
}

// The same row by one warp with scalar accesses, for sizes, strides or
// addresses that the chunked form does not take.  Every pair is read and
// written by one lane, so y may be x.
template <class T>
DSA_DEV void row_forward_scalar(const T* x, T* y, const RowXform& ra, int dim, const float* __restrict__ cs, int lane) {
    float rstd = 1.f;
    if (ra.norm_dim > 0) {
        float ss = 0.f;
        for (int c = lane; c < ra.norm_dim; c += 32) {
            const float a = load1(x + c);
            ss = fmaf(a, a, ss);
        }
        rstd = row_rstd(group_sum<32>(ss) / (float)ra.norm_dim + ra.eps);
    }
    __syncwarp();
    auto value = [&](int c) {
        const float a = load1(x + c);
        if (c >= ra.norm_dim) return a;
        return ra.weight ? a * rstd * __ldg(ra.weight + c) : a * rstd;
    };
    for (int c = lane; c < dim; c += 32)
        if (c < ra.rope_begin || c >= ra.rope_begin + ra.rope_dim) store1(y + c, value(c));
    const int h = ra.rope_dim >> 1;
    for (int j = lane; j < h; j += 32) {
        const int ca = ra.rope_begin + (ra.interleaved ? 2 * j : j), cb = ca + (ra.interleaved ? 1 : h);
        const float a = value(ca), b = value(cb), c = __ldg(cs + j), s = __ldg(cs + h + j);
        store1(y + ca, a * c - b * s);
        store1(y + cb, b * c + a * s);
    }
}

// Whether the chunked form takes these columns (strides and addresses are
// checked by its callers): whole chunks, pairs inside a chunk or a whole
// number of chunks apart.
inline bool row_xform_chunked(const RowXform& ra, int dim) {
    auto al = [](const void* p) { return ((uintptr_t)p & 15) == 0; };
    return dim % 8 == 0 && dim <= kRowMaxDim && ra.norm_dim % 8 == 0 && ra.rope_begin % 8 == 0 &&
           (ra.interleaved ? ra.rope_dim % 8 == 0 : ra.rope_dim % 16 == 0) && al(ra.weight) && al(ra.cos_sin);
}

}  // namespace dsa
