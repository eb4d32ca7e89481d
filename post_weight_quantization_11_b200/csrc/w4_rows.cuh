// The product of a few activation columns with packed INT4 rows, for kernels
// that stream the rows from HBM once ("INT4/INT8 量化推理" sec. 六):
//
//   y[r][n] = sum_k Q[r][k] x[n][k],  Q[r][k] = s (c - z) per group of g columns
//           = sum over groups of  s (sum_k c x  -  z sum_k x)
//
// A CTA has 16 warps = KW shares of the columns x RW row tiles of 16 rows.  A
// step is 128 columns of a row tile: 64 bytes a row, 1 KB a warp.
//  * Products on m16n8k16 mma.sync, fp16 x fp16 -> fp32, rows as A, up to eight
//    columns n.  A nibble alone in its half word is the fp16 subnormal c 2^-24,
//    and four bits up it is c 2^-20: one AND makes an operand register of two
//    codes (nibbles 0 and 4, then 2 and 6, of the low positions; 1 and 5, 3 and
//    7 of the high ones), with no OR, subtraction or conversion.  The two
//    positions have their own accumulators, joined when the group's scale is
//    applied; the zero point is applied there too, through the group's sum of
//    x.  1.25 ALU instructions an operand register, against 2.75 for codes in
//    the mantissa of 1024.  Products (11 by 4 bits) are exact, sums fp32.
//  * Every warp has its own ring of W4_RING steps in shared memory, filled by
//    16-byte asynchronous copies that run ahead across row tiles: no barrier
//    between warps, and no registers (a ring of four steps in registers was
//    bound by waiting for loads at 0.33 of HBM: a wait on one load waits for
//    the younger ones that share its scoreboard).
//  * x is staged once per CTA in operand order: 16 bytes hold the eight columns
//    of one packed word for one n, so one LDS.128 feeds two products; the order
//    within the eight is the nibbles' pairing above.
// Groups that are a multiple of 128 columns (WIDE) fold once a step; smaller
// ones fold every 32 columns, for which a lane takes words of a row that are 16
// bytes apart, so that a product stays inside 32 columns.
// SPLIT: x in two fp16 parts (22 bits) for fp32 activations, scaled by a power
// of two per column.
#pragma once

#include "common.cuh"
#include "tc_common.cuh"

namespace gptq {

constexpr int W4_THREADS = 512;
constexpr int W4_RING = 6;                        // steps in flight per warp
constexpr int W4_STEP = 128;                      // columns per step
constexpr int W4_COLS = 8;                        // columns n of a product

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

// D = A B
__device__ __forceinline__ void mma_16816_first(float (&c)[4], uint32_t a0, uint32_t a1,
                                                uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 16 bytes global -> shared, asynchronous
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// The rows of a group of row tiles: a uniform base for the first and the second
// row of every lane, and the lane's own offsets from it (32 bits: an address is
// a uniform register plus one lane register)
struct W4Rows {
    const uint8_t* q[2];
    const __half* s[2];
    const uint8_t* z[2];
    uint32_t oq[2], os[2], oz[2];
};

// base[i]: uniform row; row[i]: the lane's row from there on
__device__ __forceinline__ W4Rows w4_rows(const W4Layer& l, const int64_t (&base)[2],
                                          const uint32_t (&row)[2])
{
    W4Rows r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        r.q[i] = reinterpret_cast<const uint8_t*>(l.qw) + base[i] * l.rowb;
        r.s[i] = l.sc + base[i] * l.G;
        r.z[i] = l.qz + base[i] * l.Gb;
        r.oq[i] = row[i] * uint32_t(l.rowb) + (threadIdx.x & 3) * 16;
        r.os[i] = row[i] * uint32_t(l.G);
        r.oz[i] = row[i] * uint32_t(l.Gb);
    }
    return r;
}

// Scale and zero point of a group, as two halves of a register: of the group of
// column block 4 step + block (of 32 columns), for each of the lane's rows
__device__ __forceinline__ void w4_load_params(uint32_t (&p)[2], const W4Rows& r, const W4Layer& l,
                                               int block)
{
    const uint32_t grp = (uint32_t(block) * l.grp.mul) >> 22;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t z = (r.z[i][r.oz[i] + (grp >> 1)] >> (4 * (grp & 1))) & 15u;
        p[i] = uint32_t(__half_as_ushort(r.s[i][r.os[i] + grp])) | (z << 16);
    }
}

// Staged activations: chunk ((step 4 + w) cols + n) 4 + t of 16 bytes holds, for
// column n, the columns 128 step + 32 t + 8 w .. (WIDE) or 128 step + 32 w + 8 t ..
// in the order 0 4 2 6 1 5 3 7; SPLIT: a second plane behind the first.  xs: 2^-24
// times the sums of a step's 128 (WIDE) or 32 columns, 8 floats each.  Lanes of
// columns behind cols read another column; their results are not used.
struct W4Stage {
    const uint4* x;
    const float* xs;
    int cols;              // columns that are staged
    int plane;             // chunks of one plane
};

// A slot of the ring: row 8 i + g (the lane's row i) at 64 (8 i + g), its 16-byte
// parts t exchanged by t ^ (g >> 1) so that the 32-bit reads of the narrow form
// hit 32 banks
__device__ __forceinline__ uint32_t w4_part(int g, int t) { return uint32_t(t ^ ((g >> 1) & 3)) * 16; }

// y += 2^-24 times the step's product.  qa, qb: the lane's words of its rows.  p:
// w4_load_params, held by lane t of the quad for (WIDE) step src of four or
// (otherwise) block t of this step.
template <bool WIDE, bool SPLIT>
__device__ __forceinline__ void w4_step(float (&y)[4], const uint32_t (&qa)[4],
                                        const uint32_t (&qb)[4], const uint32_t (&p)[2], int src,
                                        const uint4* x, const float* xs, const W4Stage& st)
{
    constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u;
    const int lane = threadIdx.x & 31, t = lane & 3;
    float lo[4], hi[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const uint32_t a = qa[w], b = qb[w], a8 = a >> 8, b8 = b >> 8;
#pragma unroll
        for (int h = 0; h < (SPLIT ? 2 : 1); ++h) {
            const uint4 f = x[h * st.plane];
            if (h == 0 && (!WIDE || w == 0)) {
                mma_16816_first(lo, a & LO, b & LO, a8 & LO, b8 & LO, f.x, f.y);
                mma_16816_first(hi, a & HI, b & HI, a8 & HI, b8 & HI, f.z, f.w);
            } else {
                mma_16816(lo, a & LO, b & LO, a8 & LO, b8 & LO, f.x, f.y);
                mma_16816(hi, a & HI, b & HI, a8 & HI, b8 & HI, f.z, f.w);
            }
        }
        x += st.cols * 4;
        if (!WIDE || w == 3) {
            float s[2], z[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t u = __shfl_sync(0xffffffffu, p[i], (lane & ~3) | (WIDE ? src : w));
                s[i] = __half2float(__ushort_as_half((unsigned short)(u & 0xffffu)));
                z[i] = -float(u >> 16);
            }
            const float2 k = *reinterpret_cast<const float2*>(xs + 2 * t);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float c = fmaf(hi[i], 0.0625f, lo[i]);                 // 2^-24 sum c x
                y[i] = fmaf(s[i >> 1], fmaf(z[i >> 1], (i & 1) ? k.y : k.x, c), y[i]);
            }
            xs += W4_COLS;
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
template <bool WIDE, class Row>
__device__ __forceinline__ void w4_stage_half(uint4* x, float* xs, Row row, const int32_t* perm,
                                              int k0, int steps, int cols, int d)
{
    constexpr int XS = W4_COLS;
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
        if (on && kc % (WIDE ? 16 : 4) == 0) xs[(kc / (WIDE ? 16 : 4)) * XS + n] = s * 0x1p-24f;
    }
}

// Stages fp32 rows in two fp16 parts: column n scaled by the power of two that
// brings its largest magnitude to 2^14 .. 2^15 (undo[n]: its inverse; a column
// with an infinity or NaN is not scaled).  top: W4_COLS words of scratch.  Holds
// barriers; ends without one.
template <bool WIDE, class Row>
__device__ __forceinline__ void w4_stage_split(uint4* x, float* xs, float* undo, uint32_t* top,
                                               Row row, const int32_t* perm, int k0, int steps,
                                               int cols, int d)
{
    constexpr int XS = W4_COLS;
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
        if (on && kc % (WIDE ? 16 : 4) == 0) xs[(kc / (WIDE ? 16 : 4)) * XS + n] = s * 0x1p-24f;
    }
}

// Dynamic shared memory of a sweep, in this order
inline __host__ __device__ size_t w4_x_bytes(int steps, int cols, bool split)
{
    return size_t(steps) * 256 * cols * (split ? 2 : 1);
}
inline __host__ __device__ size_t w4_xs_bytes(int steps, bool wide)
{
    return size_t(steps) * (wide ? 1 : 4) * W4_COLS * 4;
}
constexpr size_t W4_RED_BYTES = size_t(2) * W4_THREADS * 16;
constexpr size_t W4_RING_BYTES = size_t(W4_THREADS / 32) * W4_RING * 1024;
inline __host__ __device__ size_t w4_smem(int steps, int cols, bool wide, bool split)
{
    return w4_x_bytes(steps, cols, split) + w4_xs_bytes(steps, wide) + W4_RED_BYTES + W4_RING_BYTES;
}

// Sweeps the row-tile groups [g0, g1) over a slice of `steps` steps that starts
// at step k0 of the rows.  red: W4_RED_BYTES, then the ring.
//   rows(group): the lane's rows of a group of RW row tiles;
//   stage(): stages x (called after the first copies are issued; ends with a
//            barrier);
//   done(group, j, v): v the joined element j of the four of an m16n8 tile (row
//            (lane >> 2) + 8 (j >> 1), column 2 (lane & 3) + (j & 1)) of row tile
//            rw = warp / KW, times 2^24.  The KW warps of a tile share its four
//            elements.
// PAIR: done(group, j, v, v2) gets elements j and j + 2 together (rows r and r +
// 8: gate and up).
template <int KW, bool WIDE, bool SPLIT, bool PAIR, class RowsF, class StageF, class DoneF>
__device__ __forceinline__ void w4_sweep(const W4Layer& l, const W4Stage& st, float* red, int g0,
                                         int g1, int k0, int steps, RowsF rows, StageF stage,
                                         DoneF done)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 3, g = lane >> 2;
    const int kw = warp % KW, rw = warp / KW;
    const int s0 = steps * kw / KW, n = steps * (kw + 1) / KW - s0;
    uint8_t* ring = reinterpret_cast<uint8_t*>(red) + W4_RED_BYTES + warp * (W4_RING * 1024);
    const uint32_t put = smem_u32(ring) + g * 64 + w4_part(g, t);
    // producer: step pj of group pg goes into slot ps
    int pg = n ? g0 : g1, pj = 0, ps = 0;
    W4Rows prod = rows(g0);
    auto issue = [&]() {
        if (pg < g1) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                cp_async16(put + ps * 1024 + i * 512, prod.q[i] + (k0 + s0 + pj) * 64 + prod.oq[i]);
            if (++pj == n) {
                pj = 0;
                if (++pg < g1) prod = rows(pg);
            }
        }
        ps = ps + 1 == W4_RING ? 0 : ps + 1;
        cp_async_commit();                                 // one (maybe empty) group per step
    };
#pragma unroll
    for (int i = 0; i < W4_RING; ++i) issue();
    // scales and zero points of four steps (WIDE: lane t those of step t; else
    // block t of each), loaded four steps ahead
    constexpr int PR = WIDE ? 1 : 4;
    uint32_t par[PR][2] = {};
    auto params = [&](uint32_t (&p)[PR][2], const W4Rows& r, int j) {
#pragma unroll
        for (int i = 0; i < PR; ++i)
            w4_load_params(p[i], r, l, (k0 + s0 + min(j + (WIDE ? t : i), n - 1)) * 4 + (WIDE ? 0 : t));
    };
    W4Rows cur = prod;
    if (n) params(par, rows(g0), 0);
    stage();
    const uint4* xw = st.x + (min(g, st.cols - 1) * 4 + t) + s0 * st.cols * 16;
    const float* xsw = st.xs + s0 * (WIDE ? 1 : 4) * W4_COLS;
    int slot = 0;
    for (int grp = g0; grp < g1; ++grp) {
        const W4Rows next = rows(min(grp + 1, g1 - 1));
        float y[4] = {0.f, 0.f, 0.f, 0.f};
        const uint4* x = xw;
        const float* xs = xsw;
        for (int jb = 0; jb < n; jb += 4) {
            uint32_t ahead[PR][2];
            if (jb + 4 < n) params(ahead, cur, jb + 4);
            else params(ahead, next, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (jb + r < n) {
                    cp_async_wait<W4_RING - 1>();
                    if (!WIDE) __syncwarp();
                    uint32_t q[2][4];
                    const uint8_t* from = ring + slot * 1024 + g * 64;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if constexpr (WIDE) {
                            const uint4 v =
                                *reinterpret_cast<const uint4*>(from + i * 512 + w4_part(g, t));
                            q[i][0] = v.x; q[i][1] = v.y; q[i][2] = v.z; q[i][3] = v.w;
                        } else {
#pragma unroll
                            for (int w = 0; w < 4; ++w)
                                q[i][w] = *reinterpret_cast<const uint32_t*>(
                                    from + i * 512 + w4_part(g, w) + t * 4);
                        }
                    }
                    if (!WIDE) __syncwarp();
                    slot = slot + 1 == W4_RING ? 0 : slot + 1;
                    issue();                               // into the slot just read
                    w4_step<WIDE, SPLIT>(y, q[0], q[1], par[WIDE ? 0 : r], r, x, xs, st);
                    x += st.cols * 16;
                    xs += (WIDE ? 1 : 4) * W4_COLS;
                }
            }
#pragma unroll
            for (int i = 0; i < PR; ++i) { par[i][0] = ahead[i][0]; par[i][1] = ahead[i][1]; }
        }
        float* out = red + ((grp - g0) & 1) * (W4_THREADS * 4);
        *reinterpret_cast<float4*>(out + threadIdx.x * 4) = make_float4(y[0], y[1], y[2], y[3]);
        __syncthreads();                                   // the buffer of two groups ago is free
        constexpr int OUT = PAIR ? 2 : 4;                  // results per lane of a tile
        for (int j = kw; j < OUT; j += KW) {
            float v = 0.f, v2 = 0.f;
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                const float* p = out + ((rw * KW + k) * 32 + lane) * 4 + j;
                v += p[0];
                if (PAIR) v2 += p[2];
            }
            if constexpr (PAIR) done(grp, j, v * 0x1p24f, v2 * 0x1p24f);
            else done(grp, j, v * 0x1p24f);
        }
        cur = next;
    }
    cp_async_wait<0>();
    __syncthreads();                                       // x, red and the ring free again
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
