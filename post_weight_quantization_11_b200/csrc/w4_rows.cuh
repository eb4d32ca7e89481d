// The product of a few activation columns with packed INT4 rows, for kernels
// that stream the rows from HBM once ("INT4/INT8 量化推理" sec. 六):
//
//   y[r][n] = sum_k Q[r][k] x[n][k],  Q[r][k] = s (c - z) per group of g columns
//           = sum over groups of  s (sum_k c x  -  z sum_k x)
//
// A CTA has 8 warps = KW shares of the columns x RW row tiles of 16 rows.  A
// step is 128 columns of a row tile: 64 bytes a row, 1 KB a warp.
//  * Products on m16n8k16 mma.sync, fp16 x fp16 -> fp32, rows as A.  A nibble
//    alone in its half word is the fp16 subnormal c 2^-24, and four bits up it
//    is c 2^-20: one AND makes an operand register of two codes (nibbles 0 and
//    4, then 2 and 6, of the low positions; 1 and 5, 3 and 7 of the high ones),
//    with no OR, subtraction or conversion.  The two positions have their own
//    accumulators, joined when the group's scale is applied; the zero point is
//    applied there too, through the group's sum of x.  1.25 ALU instructions an
//    operand register, against 2.75 for codes in the mantissa of 1024.
//    Products (11 by 4 bits) are exact, sums fp32.
//  * Rows come straight from HBM into registers: the four 16-byte loads of a
//    step's row are the four lanes that hold the row's operand, so nothing
//    passes through shared memory.  Every lane keeps a ring of four steps in
//    flight (4 KB a warp), across row tiles.
//  * x is staged once per CTA in operand order: 16 bytes hold the eight columns
//    of one packed word for one n, so one LDS.128 feeds two products; the order
//    within the eight is the nibbles' pairing above.
// Groups that are a multiple of 128 columns (WIDE) fold once a step; smaller
// ones fold every 32 columns, for which a lane takes the words of a row that
// are 16 bytes apart (32-bit loads) so that a product stays inside 32 columns.
// SPLIT: x in two fp16 parts (22 bits) for fp32 activations, scaled by a power
// of two per column.
#pragma once

#include "common.cuh"
#include "tc_common.cuh"

namespace gptq {

constexpr int W4_KW = 4, W4_RW = 2;               // column shares, row tiles of a CTA
constexpr int W4_THREADS = 32 * W4_KW * W4_RW;
constexpr int W4_RING = 4;                        // steps in flight per lane
constexpr int W4_STEP = 128;                      // columns per step

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// D (16x8 fp32) += A (16x16 fp16, row) B (16x8 fp16, col)
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Streamed once: not kept in L1
__device__ __forceinline__ uint4 ld_stream16(const void* p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t ld_nc4(const void* p)
{
    uint32_t v;
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// floor(block * 32 / g) for blocks of 32 columns: block * mul >> 22, exact for
// block, g / 32 <= 1024 (the rounding of mul adds less than block g / 32 / 2^22
// of a group to the quotient, whose fraction is at most 1 - 32 / g)
struct W4Group { uint32_t mul; };
inline W4Group w4_group(int64_t g)
{
    const uint32_t n = uint32_t(g / 32);
    return W4Group{((1u << 22) + n - 1) / n};
}

// One packed layer
struct W4Layer {
    const uint32_t* qw;
    const __half* sc;
    const uint8_t* qz;
    int64_t rowb;          // bytes of a packed row
    int G, Gb;             // groups of a row, bytes of its zero points
    W4Group grp;
};

inline W4Layer w4_layer(const uint32_t* qw, const uint16_t* sc, const uint8_t* qz, int64_t d,
                        int64_t g)
{
    W4Layer l;
    l.qw = qw;
    l.sc = reinterpret_cast<const __half*>(sc);
    l.qz = qz;
    l.rowb = d / 2;
    l.G = int(d / g);
    l.Gb = (l.G + 1) / 2;
    l.grp = w4_group(g);
    return l;
}

// The two rows (g, g + 8 of the row tile) of a lane
struct W4Rows {
    const uint8_t* q[2];
    const __half* s[2];
    const uint8_t* z[2];
};

__device__ __forceinline__ W4Rows w4_rows(const W4Layer& l, int64_t ra, int64_t rb)
{
    W4Rows r;
    const uint8_t* q = reinterpret_cast<const uint8_t*>(l.qw);
    r.q[0] = q + ra * l.rowb;
    r.q[1] = q + rb * l.rowb;
    r.s[0] = l.sc + ra * l.G;
    r.s[1] = l.sc + rb * l.G;
    r.z[0] = l.qz + ra * l.Gb;
    r.z[1] = l.qz + rb * l.Gb;
    return r;
}

// A step of a lane: 16 bytes of each row and the scale and zero point (bits 0 ..
// 15 and 16 ..) of the step's group, or, where groups are smaller, of the 32
// columns of the lane's own number in the quad
struct W4Regs {
    uint4 q[2];
    uint32_t p[2];
};

template <bool WIDE>
__device__ __forceinline__ void w4_load(W4Regs& v, const W4Rows& r, const W4Layer& l, int step)
{
    const int t = threadIdx.x & 3;
    const int grp = int((uint32_t(step * 4 + (WIDE ? 0 : t)) * l.grp.mul) >> 22);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (WIDE) {
            v.q[i] = ld_stream16(r.q[i] + step * 64 + t * 16);
        } else {
            const uint8_t* p = r.q[i] + step * 64 + t * 4;
            v.q[i] = make_uint4(ld_nc4(p), ld_nc4(p + 16), ld_nc4(p + 32), ld_nc4(p + 48));
        }
        v.p[i] = uint32_t(__half_as_ushort(r.s[i][grp])) |
                 (((uint32_t(r.z[i][grp >> 1]) >> (4 * (grp & 1))) & 15u) << 16);
    }
}

// Staged activations: chunk ((step 4 + w) cols + n) 4 + t of 16 bytes holds, for
// column n, the columns 128 step + 32 t + 8 w .. (WIDE) or 128 step + 32 w + 8 t ..
// in the order 0 4 2 6 1 5 3 7; SPLIT: a second plane behind the first.  xs: the
// sums of a step's 128 (WIDE) or 32 columns, 8 NT floats each, zero behind cols.
struct W4Stage {
    const uint4* x;
    const float* xs;
    int cols;              // columns that are staged (the others are zero)
    int plane;             // chunks of one plane
};

template <int NT, bool WIDE, bool SPLIT>
__device__ __forceinline__ void w4_step(float (&y)[NT][4], const W4Regs& v, const W4Stage& st,
                                        int step)
{
    constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t qa[4] = {v.q[0].x, v.q[0].y, v.q[0].z, v.q[0].w};
    const uint32_t qb[4] = {v.q[1].x, v.q[1].y, v.q[1].z, v.q[1].w};
    float lo[NT][4], hi[NT][4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (!WIDE || w == 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) lo[n][i] = hi[n][i] = 0.f;
        }
        const uint32_t a = qa[w], b = qb[w], a8 = a >> 8, b8 = b >> 8;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bool on = n * 8 + g < st.cols;
            const int at = ((step * 4 + w) * st.cols + n * 8 + g) * 4 + t;
#pragma unroll
            for (int p = 0; p < (SPLIT ? 2 : 1); ++p) {
                const uint4 x = on ? st.x[at + p * st.plane] : make_uint4(0u, 0u, 0u, 0u);
                mma_16816(lo[n], a & LO, b & LO, a8 & LO, b8 & LO, x.x, x.y);
                mma_16816(hi[n], a & HI, b & HI, a8 & HI, b8 & HI, x.z, x.w);
            }
        }
        if (!WIDE || w == 3) {
            uint32_t pa = v.p[0], pb = v.p[1];
            if constexpr (!WIDE) {
                pa = __shfl_sync(0xffffffffu, pa, (lane & ~3) | w);
                pb = __shfl_sync(0xffffffffu, pb, (lane & ~3) | w);
            }
            const float s[2] = {__half2float(__ushort_as_half((unsigned short)(pa & 0xffffu))),
                                __half2float(__ushort_as_half((unsigned short)(pb & 0xffffu)))};
            const float z[2] = {s[0] * float(pa >> 16), s[1] * float(pb >> 16)};   // exact
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 xs = *reinterpret_cast<const float2*>(
                    st.xs + (WIDE ? step : step * 4 + w) * (8 * NT) + n * 8 + 2 * t);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float c = fmaf(hi[n][i], 0.0625f, lo[n][i]);             // 2^-24 sum c x
                    y[n][i] = fmaf(s[i >> 1] * 16777216.f, c, y[n][i]);
                    y[n][i] = fmaf(-z[i >> 1], (i & 1) ? xs.y : xs.x, y[n][i]);
                }
            }
        }
    }
}

// Where the chunk of the columns 8 kc .. of column n goes
template <bool WIDE> __device__ __forceinline__ int w4_chunk(int kc, int n, int cols)
{
    const int step = kc >> 4, hi = (kc >> 2) & 3, lo = kc & 3;
    const int w = WIDE ? lo : hi, t = WIDE ? hi : lo;
    return ((step * 4 + w) * cols + n) * 4 + t;
}

__device__ __forceinline__ uint32_t pack2(__half a, __half b)
{
    return uint32_t(__half_as_ushort(a)) | (uint32_t(__half_as_ushort(b)) << 16);
}

__device__ __forceinline__ uint4 w4_order(const __half (&h)[8])
{
    return make_uint4(pack2(h[0], h[4]), pack2(h[2], h[6]), pack2(h[1], h[5]), pack2(h[3], h[7]));
}

// The sums of x over 32 (or 128, WIDE) columns from each lane's sum over 8; lanes
// hold consecutive chunks, 16 to a step
template <bool WIDE> __device__ __forceinline__ float w4_join(float s)
{
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    if constexpr (WIDE) {
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
    }
    return s;
}

// Stages columns [k0, k0 + 128 steps) of `cols` fp16 rows (row(n): its first
// element), through perm when given.  All threads; ends without a barrier.
template <int NT, bool WIDE, class Row>
__device__ __forceinline__ void w4_stage_half(uint4* x, float* xs, Row row, const int32_t* perm,
                                              int k0, int steps, int cols, int d)
{
    constexpr int XS = 8 * NT;
    for (int i = threadIdx.x; i < steps * (WIDE ? 1 : 4) * XS; i += blockDim.x)
        if (i % XS >= cols) xs[i] = 0.f;
    const int nch = steps * 16, total = cols * nch;        // a multiple of 16
    for (int base = 0; base < total; base += blockDim.x) {
        const int i = base + threadIdx.x;
        const bool on = i < total;
        const int n = on ? i / nch : 0, kc = on ? i - n * nch : 0;
        float s = 0.f;
        if (on) {
            const __half* src = row(n);
            alignas(16) __half h[8];
            if (!perm) {
                *reinterpret_cast<uint4*>(h) = *reinterpret_cast<const uint4*>(src + k0 + kc * 8);
            } else {
                const int4 pa = *reinterpret_cast<const int4*>(perm + k0 + kc * 8);
                const int4 pb = *reinterpret_cast<const int4*>(perm + k0 + kc * 8 + 4);
                const int at[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool ok = at[j] >= 0 && at[j] < d;   // a bad index is not followed
                    if (!ok) atomicCAS(&g_device_status, 0, kErrIndex);
                    h[j] = ok ? src[at[j]] : __ushort_as_half(0);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) s += __half2float(h[j]);
            x[w4_chunk<WIDE>(kc, n, cols)] = w4_order(h);
        }
        s = w4_join<WIDE>(s);
        if (on && kc % (WIDE ? 16 : 4) == 0) xs[(kc / (WIDE ? 16 : 4)) * XS + n] = s;
    }
}

// Stages fp32 rows in two fp16 parts: column n scaled by the power of two that
// brings its largest magnitude to 2^14 .. 2^15 (undo[n]: its inverse; a column
// with an infinity or NaN is not scaled).  top: NT * 8 words of scratch.  Holds
// barriers; ends without one.
template <int NT, bool WIDE, class Row>
__device__ __forceinline__ void w4_stage_split(uint4* x, float* xs, float* undo, uint32_t* top,
                                               Row row, const int32_t* perm, int k0, int steps,
                                               int cols, int d)
{
    constexpr int XS = 8 * NT;
    for (int i = threadIdx.x; i < XS; i += blockDim.x) top[i] = 0u;
    __syncthreads();
    const int nch = steps * 16, total = cols * nch;
    auto load = [&](int n, int kc, float (&v)[8]) {
        const float* src = row(n);
        if (!perm) {
            const float4 a = *reinterpret_cast<const float4*>(src + k0 + kc * 8);
            const float4 b = *reinterpret_cast<const float4*>(src + k0 + kc * 8 + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int at = perm[k0 + kc * 8 + j];
                const bool ok = at >= 0 && at < d;
                if (!ok) atomicCAS(&g_device_status, 0, kErrIndex);
                v[j] = ok ? src[at] : 0.f;
            }
        }
    };
    for (int base = 0; base < total; base += blockDim.x) {
        const int i = base + threadIdx.x;
        const bool on = i < total;
        const int n = on ? i / nch : 0;
        uint32_t m = 0u;
        if (on) {
            float v[8];
            load(n, i - n * nch, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (on && (threadIdx.x & 15) == 0) atomicMax(&top[n], m);   // 16 lanes: one step of one n
    }
    __syncthreads();
    for (int i = threadIdx.x; i < steps * (WIDE ? 1 : 4) * XS; i += blockDim.x)
        if (i % XS >= cols) xs[i] = 0.f;
    auto factor = [&](int n) {                             // 2^(14 - exponent of the maximum)
        const uint32_t m = top[n];
        if (m == 0u || m >= 0x7f800000u) return 1.f;
        const int e = max(-100, int(m >> 23) - 127);       // tiny columns: the largest factor
        return __uint_as_float(uint32_t(127 + 14 - e) << 23);
    };
    if (threadIdx.x < XS) undo[threadIdx.x] = threadIdx.x < cols ? 1.f / factor(threadIdx.x) : 0.f;
    for (int base = 0; base < total; base += blockDim.x) {
        const int i = base + threadIdx.x;
        const bool on = i < total;
        const int n = on ? i / nch : 0, kc = on ? i - n * nch : 0;
        float s = 0.f;
        if (on) {
            float v[8];
            load(n, kc, v);
            const float f = factor(n);
            __half h[8], l[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float a = v[j] * f;                  // exact
                h[j] = __float2half_rn(a);
                l[j] = __float2half_rn(a - __half2float(h[j]));
                s += __half2float(h[j]) + __half2float(l[j]);
            }
            const int at = w4_chunk<WIDE>(kc, n, cols);
            x[at] = w4_order(h);
            x[at + cols * nch] = w4_order(l);
        }
        s = w4_join<WIDE>(s);
        if (on && kc % (WIDE ? 16 : 4) == 0) xs[(kc / (WIDE ? 16 : 4)) * XS + n] = s;
    }
}

// Shared memory of a staged slice
inline __host__ __device__ size_t w4_x_bytes(int steps, int cols, bool split)
{
    return size_t(steps) * 256 * cols * (split ? 2 : 1);
}
inline __host__ __device__ size_t w4_xs_bytes(int steps, int nt, bool wide)
{
    return size_t(steps) * (wide ? 1 : 4) * 8 * nt * 4;
}
constexpr size_t w4_red_bytes(int nt) { return size_t(2) * W4_THREADS * 4 * nt * 4; }

// Sweeps the row-tile groups [g0, g1) over a slice of `steps` steps that starts
// at step k0 of the rows.
//   rows(group, rw): the lane's two rows of row tile rw of the group;
//   stage(): stages x (called after the first loads are issued; ends with a
//            barrier);
//   done(group, y): this thread's share of the joined result: y[n][j], element
//            j = kw of the four of an m16n8 tile (row (lane >> 2) + 8 (j >> 1),
//            column 8 n + 2 (lane & 3) + (j & 1)) of row tile rw.
// PAIR: done gets elements kw and kw + 2 instead, in the warps kw < 2 only (rows
// r and r + 8: gate and up).
template <int NT, bool WIDE, bool SPLIT, bool PAIR, class RowsF, class StageF, class DoneF>
__device__ __forceinline__ void w4_sweep(const W4Layer& l, const W4Stage& st, float* red, int g0,
                                         int g1, int k0, int steps, RowsF rows, StageF stage,
                                         DoneF done)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kw = warp % W4_KW, rw = warp / W4_KW;
    const int s0 = steps * kw / W4_KW, n = steps * (kw + 1) / W4_KW - s0;
    W4Regs ring[W4_RING];
    W4Rows cur = rows(g0, rw);
#pragma unroll
    for (int r = 0; r < W4_RING; ++r)
        if (r < n) w4_load<WIDE>(ring[r], cur, l, k0 + s0 + r);
    stage();
    int buf = 0;
    for (int grp = g0; grp < g1; ++grp, buf ^= 1) {
        const bool more = grp + 1 < g1;
        const W4Rows next = more ? rows(grp + 1, rw) : cur;
        float y[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[i][j] = 0.f;
        for (int jb = 0; jb < n; jb += W4_RING) {
#pragma unroll
            for (int r = 0; r < W4_RING; ++r) {
                if (jb + r < n) {
                    w4_step<NT, WIDE, SPLIT>(y, ring[r], st, s0 + jb + r);
                    if (jb + W4_RING + r < n)
                        w4_load<WIDE>(ring[r], cur, l, k0 + s0 + jb + W4_RING + r);
                    else if (more)
                        w4_load<WIDE>(ring[r], next, l, k0 + s0 + r);
                }
            }
        }
        float* out = red + buf * (W4_THREADS * 4 * NT);
#pragma unroll
        for (int i = 0; i < NT; ++i)
            *reinterpret_cast<float4*>(out + ((i * 8 + warp) * 32 + lane) * 4) =
                make_float4(y[i][0], y[i][1], y[i][2], y[i][3]);
        __syncthreads();                                   // the buffer of two groups ago is free
        if constexpr (PAIR) {
            if (kw < 2) {
                float v[NT][2];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    v[i][0] = v[i][1] = 0.f;
#pragma unroll
                    for (int k = 0; k < W4_KW; ++k) {
                        const float* p = out + ((i * 8 + rw * W4_KW + k) * 32 + lane) * 4 + kw;
                        v[i][0] += p[0];
                        v[i][1] += p[2];
                    }
                }
                done(grp, v);
            }
        } else {
            float v[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                v[i] = 0.f;
#pragma unroll
                for (int k = 0; k < W4_KW; ++k)
                    v[i] += out[((i * 8 + rw * W4_KW + k) * 32 + lane) * 4 + kw];
            }
            done(grp, v);
        }
        cur = next;
    }
    __syncthreads();                                       // x and red free again
}

// A kernel on the stream that may start before its predecessor on it has ended
// (it waits by pdl_wait)
template <class... A>
inline cudaError_t launch_after(void (*kern)(A...), dim3 grid, dim3 block, size_t smem,
                                cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace gptq
