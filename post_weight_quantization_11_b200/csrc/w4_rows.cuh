// The product of a few activation columns with packed INT4 rows, for kernels
// that stream the rows from HBM once ("INT4/INT8 量化推理" sec. 六):
//
//   y[r][n] = sum_k Q[r][k] x[n][k],  Q[r][k] = s (c - z) per group of g columns
//           = sum over groups of  s (sum_k c x  -  z sum_k x)
//
// A CTA has 16 warps = KW shares of the columns x RW row tiles of 32 rows.  A
// step is 128 columns of a row tile: 64 bytes a row, 2 KB a warp.
//  * Products on m16n8k16 mma.sync, fp16 x fp16 -> fp32, rows as A, up to 8
//    NT columns n.  A nibble alone in its half word is the fp16 subnormal c 2^-24,
//    and four bits up it is c 2^-20: one AND makes an operand register of two
//    codes (nibbles 0 and 4, then 2 and 6, of the low positions; 1 and 5, 3 and
//    7 of the high ones).  The two positions have their own accumulators, joined
//    when the group's scale is applied; the zero point is applied there too,
//    through the group's sum of x.  Products (11 by 4 bits) are exact.  The
//    matrix pipe aligns a subnormal operand's products by the exponent field, so
//    its sums lose the operand's leading zero bits: 7 to 10 in the low position,
//    which is therefore made normal (times 2^10, one packed multiplication on the
//    otherwise idle FMA pipe), 3 to 6 in the high one, which is left.  Relative
//    error of a 4096-column product against float64: 4.3e-6 without the
//    multiplication.
//  * Every warp has its own ring of W4_RING slots of two steps in shared memory,
//    filled by TMA copies that run ahead across row tiles: no barrier between
//    warps and no registers.  With the 128-byte swizzle, and lane g of an operand
//    on row (g >> 1) + 4 (g & 1) of its eight, the reads hit every bank once.
//    (A ring of four steps in registers was bound by waiting for loads: a wait
//    on one load waits for the younger ones that share its scoreboard.)
//  * 32 rows a warp share each read of x.
//  * x is staged once per CTA in operand order: 16 bytes hold the eight columns
//    of one packed word for one n, so one LDS.128 feeds two products; the order
//    within the eight is the nibbles' pairing above.
// The scales are applied every 32 FOLD columns: once a step for groups that are a
// multiple of 128 columns (FOLD = 4); for a multiple of 64 or 32 (2, 1) a lane takes
// words of a row that are 16 bytes apart, so that a product stays inside 32 columns.
// What it reaches: a pass over 32 KB (a step of every warp) takes 0.55 us from shared
// memory alone, 8.8 TB/s on 148 SMs; in a sweep of 14336 x 4096 rows 4.3 TB/s (0.65 of the
// measured copy rate) with 258 instructions a step and warp (of which 128 unpack and
// multiply), issued in 59 % of the cycles; four warps a scheduler do not hide more.
// SPLIT: x in two fp16 parts (22 bits) for fp32 activations, scaled by a power
// of two per column: W4_TWICE: each read of the rows is multiplied with both;
// W4_BESIDE: up to four columns, the second parts are operand columns 4 .. 7 (half
// the products; one token of 8 experts of 14336 x 4096: 58 us against 63 in all).
#pragma once

#include <atomic>

#include "common.cuh"
#include "tc_common.cuh"

namespace gptq {

constexpr int W4_THREADS = 512;
constexpr int W4_RING = 2;                        // slots in flight per warp
constexpr int W4_SLOT = 4096;                     // bytes of one: two steps of 32 rows
constexpr int W4_MAX_SMEM = 226 * 1024;           // dynamic shared memory of a CTA
constexpr int W4_STEP = 128;                      // columns per step
constexpr int W4_COLS = 8;                        // columns n of an operand
enum W4Split : int { W4_WHOLE = 0, W4_TWICE = 1, W4_BESIDE = 2 };

// Two fp32 FMAs in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return d;
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

// Two codes c 2^-24 -> c 2^-14
__device__ __forceinline__ uint32_t w4_normal(uint32_t v)
{
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(1024.f));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Shared memory by its 32-bit address
__device__ __forceinline__ uint4 lds16(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float lds_f(uint32_t a) { return __uint_as_float(lds4(a)); }
__device__ __forceinline__ float2 lds_f2(uint32_t a)
{
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts_f(uint32_t a, float v)
{
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
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

// Blocks of 32 columns that share a scale, at most a step
inline int w4_fold(int64_t g) { return g % 128 == 0 ? 4 : g % 64 == 0 ? 2 : 1; }

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

// Scale and byte of zero points of a group of the lane's four rows, as loaded: what
// is computed from them waits for the loads, so that is done a round later
struct W4Raw {
    uint32_t s[2][2], z[2][2];
    uint32_t shift;                        // of the zero point in its byte
};

__device__ __forceinline__ uint32_t ld_nc_u16(const void* p)
{
    uint16_t v;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ld_nc_u8(const void* p)
{
    uint32_t v;
    asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// Scale (low half) and minus the zero point (high half) as fp16
__device__ __forceinline__ uint32_t w4_param(uint32_t s, uint32_t z, uint32_t shift)
{
    const __half m = __hsub(__ushort_as_half((unsigned short)0x6400),      // 1024 - (1024 + z)
                            __ushort_as_half((unsigned short)(0x6400u | ((z >> shift) & 15u))));
    return s | (uint32_t(__half_as_ushort(m)) << 16);
}

// Staged activations: chunk ((step 4 + w) cols + n) 4 + t of 16 bytes holds, for
// column n, the columns 128 step + 32 t + 8 w .. (FOLD 4) or 128 step + 32 w + 8 t ..
// in the order 0 4 2 6 1 5 3 7; SPLIT: a second plane behind the first.  xs: 2^-14
// times the sums of 32 FOLD columns each, 8 NT floats.  Lanes of
// columns behind cols read another column; their results are not used.
struct W4Stage {
    uint32_t x, xs;        // shared addresses
    int cols;              // columns that are staged
    uint32_t plane;        // bytes of one plane
};

// A slot: rows of 128 bytes (two steps), the 16-byte part 4 u + t of row r (part t of
// step u) at 128 r + 16 ((4 u + t) ^ (r & 7)).  Row 8 i + w4_rho(g) of the warp's m16
// tile m is row 16 m + 8 i + w4_rho(g) of a slot; PAIR: row 8 m + w4_rho(g) of the gate
// rows (i = 0) or of the up rows, which have the slot's second half.
__device__ __forceinline__ int w4_rho(int g) { return (g >> 1) + 4 * (g & 1); }
template <bool PAIR> __host__ __device__ constexpr int w4_row(int m, int i)
{
    return PAIR ? i * 16 + m * 8 : m * 16 + i * 8;
}

// y += 2^-14 times the step's product.  slot: shared address of the lane's row; FOLD 4:
// of its part t of the step, else of word t of the row.  u: the step of the slot.  p: w4_param of
// the lane's rows, of the groups of the step, held by lanes src on of the quad.
// x[c]: shared address of the lane's part of operand column 8 c + g.
template <int NT, int FOLD, int SPLIT, bool PAIR>
__device__ __forceinline__ void w4_step(float (&y)[NT][2][4], uint32_t slot, int u,
                                        const uint32_t (&p)[2][2], int src, uint32_t (&x)[NT],
                                        uint32_t xs, uint32_t xw, uint32_t plane)
{
    constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u;
    const int rho = w4_rho((threadIdx.x & 31) >> 2);
    uint32_t q[2][2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (FOLD == 4) {
                const uint4 v = lds16(slot + w4_row<PAIR>(m, i) * 128);
                q[m][i][0] = v.x; q[m][i][1] = v.y; q[m][i][2] = v.z; q[m][i][3] = v.w;
            } else {
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    q[m][i][w] = lds4(slot + w4_row<PAIR>(m, i) * 128 + ((4 * u + w) ^ rho) * 16);
            }
        }
    float lo[NT][2][4], hi[NT][2][4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t a[2][4], b[2][4];                         // operands of the low and high nibbles
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const uint32_t v0 = q[m][0][w], v1 = q[m][1][w], w0 = v0 >> 8, w1 = v1 >> 8;
            a[m][0] = w4_normal(v0 & LO); a[m][1] = w4_normal(v1 & LO);
            a[m][2] = w4_normal(w0 & LO); a[m][3] = w4_normal(w1 & LO);
            b[m][0] = v0 & HI; b[m][1] = v1 & HI; b[m][2] = w0 & HI; b[m][3] = w1 & HI;
        }
#pragma unroll
        for (int c = 0; c < NT; ++c) {
#pragma unroll
            for (int h = 0; h < (SPLIT == W4_TWICE ? 2 : 1); ++h) {
                const uint4 f = lds16(h ? x[c] + plane : x[c]);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    if (h == 0 && w % FOLD == 0) {
                        mma_16816_first(lo[c][m], a[m][0], a[m][1], a[m][2], a[m][3], f.x, f.y);
                        mma_16816_first(hi[c][m], b[m][0], b[m][1], b[m][2], b[m][3], f.z, f.w);
                    } else {
                        mma_16816(lo[c][m], a[m][0], a[m][1], a[m][2], a[m][3], f.x, f.y);
                        mma_16816(hi[c][m], b[m][0], b[m][1], b[m][2], b[m][3], f.z, f.w);
                    }
                }
            }
            x[c] += xw;
        }
        if (w % FOLD == FOLD - 1) {
            float2 sz[2][2];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t v = __shfl_sync(0xffffffffu, p[m][i], src + w / FOLD, 4);
                    sz[m][i] = __half22float2(*reinterpret_cast<const __half2*>(&v));
                }
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                const float2 k = lds_f2(xs + (w / FOLD * NT + c) * (W4_COLS * 4));
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 h = make_float2(hi[c][m][2 * i], hi[c][m][2 * i + 1]);
                        const float2 o = make_float2(lo[c][m][2 * i], lo[c][m][2 * i + 1]);
                        float2 v = fma2(h, make_float2(64.f, 64.f), o);      // 2^-14 sum c x
                        v = fma2(make_float2(sz[m][i].y, sz[m][i].y), k, v);
                        v = fma2(make_float2(sz[m][i].x, sz[m][i].x), v,
                                 make_float2(y[c][m][2 * i], y[c][m][2 * i + 1]));
                        y[c][m][2 * i] = v.x;
                        y[c][m][2 * i + 1] = v.y;
                    }
            }
        }
    }
}

// Where the chunk of the columns 8 kc .. of column n goes
template <int FOLD> __device__ __forceinline__ int w4_chunk(int kc, int n, int cols)
{
    const int step = kc >> 4, hi = (kc >> 2) & 3, lo = kc & 3;
    const int w = FOLD == 4 ? lo : hi, t = FOLD == 4 ? hi : lo;
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

// The sums of x over 32 FOLD columns from each lane's sum over 8; lanes
// hold consecutive chunks, 16 to a step
template <int FOLD> __device__ __forceinline__ float w4_join(float s)
{
#pragma unroll
    for (int o = 1; o < 4 * FOLD; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Stages columns [k0, k0 + 128 steps) of `cols` fp16 rows (row(n): its first
// element), through perm when given.  All threads; ends without a barrier.
template <int NT, int FOLD, class Row>
__device__ __forceinline__ void w4_stage_half(uint4* x, float* xs, Row row, const int32_t* perm,
                                              int k0, int steps, int cols, int d)
{
    constexpr int XS = W4_COLS * NT;
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
            x[w4_chunk<FOLD>(kc, n, cols)] = w4_order(h);
        }
        s = w4_join<FOLD>(s);
        if (on && kc % (4 * FOLD) == 0) xs[(kc / (4 * FOLD)) * XS + n] = s * 0x1p-14f;
    }
}

// Stages fp32 rows in two fp16 parts: column n scaled by the power of two that
// brings its largest magnitude to 2^14 .. 2^15 (undo[n]: its inverse; a column
// with an infinity or NaN is not scaled).  top: 8 NT words of scratch.  Holds
// barriers; ends without one.
template <int NT, int FOLD, class Row>
__device__ __forceinline__ void w4_stage_split(uint4* x, float* xs, float* undo, uint32_t* top,
                                               Row row, const int32_t* perm, int k0, int steps,
                                               int cols, int d, bool beside)
{
    constexpr int XS = W4_COLS * NT;
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
        float s = 0.f, s2 = 0.f;                           // of the first and the second parts
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
                s += __half2float(h[j]);
                s2 += __half2float(l[j]);
            }
            const int at = w4_chunk<FOLD>(kc, n, cols);
            x[at] = w4_order(h);
            x[at + cols * nch] = w4_order(l);
        }
        s = w4_join<FOLD>(s);
        s2 = w4_join<FOLD>(s2);
        if (on && kc % (4 * FOLD) == 0) {
            float* to = xs + (kc / (4 * FOLD)) * XS + n;
            to[0] = (beside ? s : s + s2) * 0x1p-14f;
            if (beside) to[4] = s2 * 0x1p-14f;
        }
    }
}

// Dynamic shared memory of a kernel with sweeps: the ring, the joining buffer,
// the barriers, then the staged activations and their sums
constexpr int W4_WARPS = W4_THREADS / 32;
constexpr size_t W4_AT_RED = size_t(W4_WARPS) * W4_RING * W4_SLOT;
constexpr size_t w4_at_bar(int nt) { return W4_AT_RED + size_t(W4_WARPS) * 32 * 8 * 4 * nt; }
constexpr size_t w4_at_x(int nt) { return w4_at_bar(nt) + 512; }
static_assert(W4_WARPS * W4_RING * 8 <= 512, "barriers");
inline __host__ __device__ size_t w4_x_bytes(int steps, int cols, bool split)
{
    return size_t(steps) * 256 * cols * (split ? 2 : 1);
}
inline __host__ __device__ size_t w4_xs_bytes(int steps, int nt, int fold)
{
    return size_t(steps) * (4 / fold) * W4_COLS * nt * 4;
}
// (and up to 1023 bytes in front, for the alignment of the ring)
inline size_t w4_smem(int steps, int cols, int nt, int fold, bool split)
{
    return 1024 + w4_at_x(nt) + w4_x_bytes(steps, cols, split) + w4_xs_bytes(steps, nt, fold);
}

// The packed rows as a TMA tensor, in boxes of `rows` rows and two steps
inline int w4_tmap(CUtensorMap* tm, const uint32_t* qw, int64_t rows, int64_t d, int box_rows)
{
    return encode_tmap_2d(tm, CU_TENSOR_MAP_DATA_TYPE_UINT32, qw, uint64_t(d / 8), uint64_t(rows),
                          uint64_t(d / 2), 32, uint32_t(box_rows), CU_TENSOR_MAP_SWIZZLE_128B);
}

__device__ __forceinline__ bool w4_elect()
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok));
    return ok != 0;
}

constexpr uint32_t W4_GONE = 2;

// A warp's ring (shared addresses)
struct W4Pipe {
    uint32_t ring, bar, red;
    uint32_t put, get;         // next slot to fill, to read
    uint32_t phase;            // parity of the slot to read; from W4_GONE on: a wait gave up, no more
                               // waits and copies of this lane (the device status says so)
    int* abort;
};

// All threads; with a barrier
template <int NT> __device__ __forceinline__ W4Pipe w4_pipe(uint8_t* smem, int* abort)
{
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);    // uniform
    W4Pipe p;
    p.ring = smem_u32(smem) + warp * (W4_RING * W4_SLOT);
    p.red = smem_u32(smem) + uint32_t(W4_AT_RED);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + w4_at_bar(NT)) + warp * W4_RING;
    p.bar = smem_u32(bar);
    p.abort = abort;
    p.put = p.get = 0;
    p.phase = 0;
    if ((threadIdx.x & 31) == 0)
        for (int i = 0; i < W4_RING; ++i) mbar_init(&bar[i], 1);
    if (threadIdx.x == 0) *abort = 0;
    fence_mbar_init();
    __syncthreads();
    return p;
}

__device__ __forceinline__ bool w4_try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// The rest of a wait that did not succeed at once, bounded like every wait of the
// library.  False: it gave up, or another wait of the CTA has
static __device__ __noinline__ bool w4_wait_long(uint32_t bar, uint32_t parity, volatile int* abort)
{
    const unsigned long long t0 = globaltimer_ns();
    for (unsigned i = 1; !w4_try_wait(bar, parity); ++i)
        if ((i & 63u) == 0) {
            if (*abort) return false;
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
                atomicCAS(&g_device_status, 0, kErrWaitFull);
                *abort = 1;
                return false;
            }
        }
    return true;
}

// For a copy in flight behind a wait that gave up: it should land before the CTA's shared
// memory is released.  Bounded, too
static __device__ __noinline__ void w4_land(uint32_t bar, uint32_t parity)
{
    const unsigned long long t0 = globaltimer_ns();
    while (!w4_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > kWaitLimitNs) return;
}

// Sweeps the groups [0, groups) of RW row tiles over a slice of `steps` steps that
// starts at step k0 of the rows.  Group 0 begins at row0 (of tm and l; end: the rows
// behind it are not read).  PAIR: a tile is 16 rows from row0 on and the 16 rows that
// lie `pair` rows further on.
// The scales of the rows from row0 on that it reads span less than 2^32 bytes.
//   stage(): stages x (called after the first copies are issued; ends with a
//            barrier);
//   done(group, r, n, v): the joined result of row r of the group (PAIR: of the
//            group's gate rows), column n; PAIR: done(group, r, n, v, v2) with the up
//            row's.
template <int NT, int KW, int FOLD, int SPLIT, bool PAIR, class StageF, class DoneF>
__device__ __forceinline__ void w4_sweep(W4Pipe& pipe, const CUtensorMap* tm, const W4Layer& l,
                                         int64_t row0, int64_t end, uint32_t pair,
                                         const W4Stage& st, int groups, int k0, int steps,
                                         StageF stage, DoneF done)
{
    constexpr int RW = W4_WARPS / KW, ROWS = PAIR ? 16 : 32;
    const int lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);    // uniform
    const int kw = warp % KW, rw = warp / KW;
    const int s0 = steps * kw / KW, n = steps * (kw + 1) / KW - s0;
    // producer: the rows and step of the next copy, steps left of the row tile,
    // row tiles left
    const int first_step = k0 + s0;
    int prow = int(row0) + rw * ROWS, pstep = first_step, pleft = n, tiles = n ? groups : 0;
    auto issue = [&]() {
        if (tiles == 0) return;
        if (w4_elect() && pipe.phase < W4_GONE) {          // (always the same lane)
            const uint32_t dst = pipe.ring + pipe.put * W4_SLOT, bar = pipe.bar + pipe.put * 8;
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                         "r"(W4_SLOT)
                         : "memory");
            auto copy = [&](uint32_t to, int row) {
                asm volatile(
                    "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
                    " [%0], [%1, {%3, %4}], [%2];" ::"r"(to),
                    "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(pstep * 16), "r"(row)
                    : "memory");
            };
            copy(dst, prow);
            if (PAIR) copy(dst + W4_SLOT / 2, prow + int(pair));
        }
        pipe.put ^= 1u;
        pstep += 2;
        pleft -= 2;
        if (pleft <= 0) { pleft = n; pstep = first_step; prow += RW * ROWS; --tiles; }
    };
    static_assert(W4_RING == 2, "pipe.put and get");
    issue();
    issue();
    // scales and zero points of FOLD steps at a time, as many steps ahead: PER groups a
    // step, lane t of a quad those of group t % PER of step t / PER
    constexpr int PER = 4 / FOLD;
    const uint8_t* sc = reinterpret_cast<const uint8_t*>(l.sc) + row0 * (l.G * 2);
    const uint8_t* qz = l.qz + row0 * l.Gb;
    const uint32_t last = uint32_t(end - row0 - 1);
    auto params = [&](W4Raw& p, int grp, int j) {
        const uint32_t block = (first_step + min(j + t / PER, n - 1)) * 4 + (t % PER) * FOLD;
        const uint32_t at = (block * l.grp.mul) >> 22;
        const uint32_t first = (grp * RW + rw) * ROWS + w4_rho(g);
        p.shift = 4 * (at & 1);
        // bytes from the sweep's first row on: a uniform base and one 32-bit register
        const uint32_t gs = uint32_t(l.G) * 2, gz = uint32_t(l.Gb);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t r = PAIR ? first + m * 8 + i * pair
                                        : min(first + m * 16 + i * 8, last);
                p.s[m][i] = ld_nc_u16(sc + (r * gs + at * 2));
                p.z[m][i] = ld_nc_u8(qz + (r * gz + (at >> 1)));
            }
    };
    uint32_t par[2][2] = {};
    W4Raw ahead{};
    if (n) params(ahead, 0, 0);
    stage();
    const uint32_t xw = st.cols * 64;
    uint32_t x0[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c)
        x0[c] = st.x + (min(SPLIT == W4_BESIDE ? g & 3 : c * 8 + g, st.cols - 1) * 4 + t) * 16 +
                s0 * 4 * xw + (SPLIT == W4_BESIDE && g >= 4 ? st.plane : 0u);
    const uint32_t xs0 = st.xs + s0 * PER * W4_COLS * NT * 4 + t * 8;
    const uint32_t from = pipe.ring + w4_rho(g) * 128 + (FOLD == 4 ? (t ^ w4_rho(g)) * 16 : t * 4);
    const uint32_t red = pipe.red + (warp * 32 + lane) * 4;
    for (int grp = 0; grp < groups; ++grp) {
        float y[NT][2][4] = {};
        uint32_t x[NT], xs = xs0;
#pragma unroll
        for (int c = 0; c < NT; ++c) x[c] = x0[c];
#pragma unroll 1
        for (int j = 0; j < n; j += 2) {
            if (pipe.phase < W4_GONE && !w4_try_wait(pipe.bar + pipe.get * 8, pipe.phase) &&
                !w4_wait_long(pipe.bar + pipe.get * 8, pipe.phase, pipe.abort)) {
                w4_land(pipe.bar + pipe.get * 8, pipe.phase);
                if (grp + 1 < groups || j + 2 < n)
                    w4_land(pipe.bar + (pipe.get ^ 1u) * 8, pipe.phase ^ pipe.get);
                pipe.phase |= W4_GONE;                     // no copies behind this one and the next
            }
            const uint32_t slot = from + pipe.get * W4_SLOT;
            auto next_params = [&](int jj) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        par[m][i] = w4_param(ahead.s[m][i], ahead.z[m][i], ahead.shift);
                if (jj + FOLD < n) params(ahead, grp, jj + FOLD);
                else params(ahead, min(grp + 1, groups - 1), 0);
            };
            auto step = [&](int u) {
                w4_step<NT, FOLD, SPLIT, PAIR>(y, FOLD == 4 ? slot ^ (64 * u) : slot, u, par,
                                               (((j & 2) + u) % FOLD) * PER, x, xs, xw, st.plane);
                xs += PER * W4_COLS * NT * 4;
            };
            if (FOLD < 4 || (j & 2) == 0) next_params(j);
            step(0);
            if (j + 1 < n) {
                if (FOLD == 1) next_params(j + 1);
                step(1);
            }
            pipe.phase ^= pipe.get;
            pipe.get ^= 1u;
            __syncwarp();                                  // every lane has read its slot
            issue();
        }
        if (grp) __syncthreads();                          // the last group's sums have been read
#pragma unroll
        for (int e = 0; e < 8 * NT; ++e)
            sts_f(red + e * W4_WARPS * 128, y[e >> 3][(e >> 2) & 1][e & 3]);
        __syncthreads();
        constexpr int EL = (PAIR ? 4 : 8) * NT;            // results per lane of a tile
#pragma unroll
        for (int u = 0; u < (RW * EL + W4_WARPS - 1) / W4_WARPS; ++u) {
            const int o = warp + u * W4_WARPS;
            if (o >= RW * EL) break;
            const int w = o / EL, r = o % EL, c = r / (EL / NT), m = (r / (EL / NT / 2)) & 1;
            const int j = r % (EL / NT / 2);
            const uint32_t p = red + ((c * 8 + m * 4 + j) * W4_WARPS + w * KW - warp) * 128;
            float v = 0.f, v2 = 0.f;
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                v += lds_f(p + k * 128);
                if (PAIR) v2 += lds_f(p + (2 * W4_WARPS + k) * 128);
            }
            if constexpr (PAIR)
                done(grp, w * 16 + m * 8 + w4_rho(g), c * 8 + 2 * t + j, v * 0x1p14f, v2 * 0x1p14f);
            else {
                if (SPLIT == W4_BESIDE) v += __shfl_xor_sync(0xffffffffu, v, 2);   // column n + 4
                done(grp, w * 32 + m * 16 + (j >> 1) * 8 + w4_rho(g), c * 8 + 2 * t + (j & 1),
                     v * 0x1p14f);
            }
        }
    }
    __syncthreads();                                       // x and red free again
}

// The opt-in to dynamic shared memory, set once per kernel and device (most:
// the largest that any call of the kernel asks for)
inline bool smem_opt_in(const void* kern, int most, std::atomic<bool> (&done)[64])
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
        return false;
    if (dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
    return true;
}

}  // namespace gptq
