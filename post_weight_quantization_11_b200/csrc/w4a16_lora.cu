// W4A16 product with low-rank adapters of many requests -- the packed product
// of "INT4/INT8 量化推理" sec. 六 plus each row's adapter:
//
//   y[b] = x[b] Q^T + scaling[a] (x[b] A_a^T) B_a^T,   a = adapter[b]
//
// Up to LORA_SWEEP rows of x two kernels (three with an act-order permutation, which the
// first applies): one sweeps the packed rows (w4_rows.cuh) for chunks of up to
// 16 rows of x and slices of the columns, and computes t[b] = scaling A_a x[b]
// beside it; the other joins the slices and adds B_a t.  Beyond, the product is
// the tcgen05 kernel's (w4a16_tc.cu), with t computed where the activations are put
// in its order.  Partial results go through memory, not atomics: their order is
// fixed.
// Measured (B200): 10 us for one row and rank 16 of 4096 x 4096 (8.9 MB; gptq_w4a16_gemm
// without adapters 11.7), 25 us for 8 requests of 14336 x 4096 with act-order (35 MB: two
// rounds of row groups where 1.5 would do, the gather 3), 52 us for 93 rows of rank 64 of
// 4096 x 11008 (36 of them the tcgen05 product).
#include "common.cuh"
#include "tc_common.cuh"
#include "w4_rows.cuh"
#include "w4a16_tc.cuh"

namespace gptq {

constexpr int LORA_KW = 8, LORA_ROWS = 32 * (W4_WARPS / LORA_KW);   // of w4_sweep
constexpr int LORA_JOIN = 4, LORA_MANY = 8;      // rows of x per CTA of the join, few and many
constexpr int LORA_JOIN_ROWS = 128;              // rows of the layer
constexpr int LORA_TC_PARTS = 4;                 // slices of the columns of x A^T (tcgen05 product)
constexpr int LORA_SWEEP = 16;                   // most rows of x of the row sweep
constexpr int LORA_MAX_RANK = 256;
constexpr int LORA_SMS = 148;                    // the plan does not depend on the device that is current

struct LoraParams {
    const __half* x;
    const int32_t* perm;
    const __half* a;
    const __half* b;
    const float* scaling;
    const int32_t* adapter;
    int64_t batch, m, d, n;
    int rank;
    W4Layer lay;
    int chunk, chunks, slice, slices, groups;
    int run;           // most row groups of one sweep
    float* t;          // batch x rank (the tcgen05 product: LORA_TC_PARTS of them)
    __half* xp;        // batch x d: x in the order of the sweep or of the tcgen05 product, or null
    int tc;
    float* part;       // slices x batch x m
    float* y;
};

// t[b][r] = scaling (A_a[r] . x[b]).  A unit is a tile of eight rows b, 16 rank rows and
// a slice of the columns, whose sums stay apart in t; for each adapter among the rows
// S = A x^T on m16n8k16 mma.sync, the slice split over the CTA's 16 warps.  A lane's
// 16-byte load is eight neighbouring columns of its row, for A and x alike: operands of
// two products, whose order of the columns does not matter.  Rows of other adapters are
// computed along and dropped.  All threads; red: 16 x 128 floats, ids: 8 ints.
__device__ __forceinline__ void lora_shrink(const LoraParams& p, float* red, int* ids)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int tiles = int((p.batch + 7) / 8), rts = (p.rank + 15) / 16;
    for (int u = blockIdx.x; u < tiles * rts * LORA_TC_PARTS; u += gridDim.x) {
        const int part = u % LORA_TC_PARTS, rest = u / LORA_TC_PARTS;
        const int64_t b0 = int64_t(rest / rts) * 8;
        const int r0 = rest % rts * 16, rounds = int(p.d / 32);
        const int n0 = rounds * part / LORA_TC_PARTS, n = rounds * (part + 1) / LORA_TC_PARTS - n0;
        const int k0 = n0 + n * warp / W4_WARPS, k1 = n0 + n * (warp + 1) / W4_WARPS;
        __syncthreads();                                   // the last unit's ids have been read
        if (threadIdx.x < 8) {
            int id = b0 + threadIdx.x < p.batch ? p.adapter[b0 + threadIdx.x] : -1;
            if (id < -1 || id >= p.n) {
                atomicCAS(&g_device_status, 0, kErrIndex);
                id = -1;
            }
            ids[threadIdx.x] = id;
        }
        __syncthreads();
        const __half* x = p.x + min(b0 + g, p.batch - 1) * p.d + t * 8;
        for (int slot = 0; slot < 8; ++slot) {
            const int id = ids[slot];
            bool first = id >= 0;                          // of the tile's rows with this adapter
            for (int j = 0; j < slot; ++j) first = first && ids[j] != id;
            if (!first) continue;
            const __half* a0 = p.a + (int64_t(id) * p.rank + min(r0 + g, p.rank - 1)) * p.d + t * 8;
            const __half* a1 = p.a + (int64_t(id) * p.rank + min(r0 + g + 8, p.rank - 1)) * p.d + t * 8;
            float s[4] = {0.f, 0.f, 0.f, 0.f};
            for (int k = k0; k < k1; k += 3) {             // three rounds of 32 columns in flight
                uint4 av[3], bv[3], xv[3];
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (k + i < k1) {
                        av[i] = __ldg(reinterpret_cast<const uint4*>(a0 + (k + i) * 32));
                        bv[i] = __ldg(reinterpret_cast<const uint4*>(a1 + (k + i) * 32));
                        xv[i] = __ldg(reinterpret_cast<const uint4*>(x + (k + i) * 32));
                    }
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (k + i < k1) {
                        mma_16816(s, av[i].x, bv[i].x, av[i].y, bv[i].y, xv[i].x, xv[i].y);
                        mma_16816(s, av[i].z, bv[i].z, av[i].w, bv[i].w, xv[i].z, xv[i].w);
                    }
            }
            __syncthreads();                               // the last adapter's sums have been read
            *reinterpret_cast<float4*>(red + (warp * 32 + lane) * 4) =
                make_float4(s[0], s[1], s[2], s[3]);
            __syncthreads();
            if (threadIdx.x < 128) {                       // element e of lane l
                const int l = threadIdx.x >> 2, e = threadIdx.x & 3;
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < W4_WARPS; ++w) v += red[w * 128 + threadIdx.x];
                const int r = r0 + (l >> 2) + 8 * (e >> 1), j = 2 * (l & 3) + (e & 1);
                if (r < p.rank && ids[j] == id)
                    p.t[(part * p.batch + b0 + j) * p.rank + r] = v * p.scaling[id];
            }
        }
    }
}

// t[b][r] = scaling (A_a[r] . x[b]): one warp per (r, b), dealt out over the CTAs from the
// last one on, for the first ones gather beside it (up to LORA_SWEEP rows: 8 rows of rank
// 16 and 4096 columns leave the whole call 9 us faster than lora_shrink, which has a CTA
// per unit)
__device__ __forceinline__ void lora_shrink_few(const LoraParams& p)
{
    const int lane = threadIdx.x & 31;
    const int64_t items = p.batch * p.rank;
    for (int64_t it = int64_t(threadIdx.x >> 5) * gridDim.x + (gridDim.x - 1 - blockIdx.x); it < items;
         it += int64_t(gridDim.x) * W4_WARPS) {
        const int r = int(it / p.batch);
        const int64_t b = it - r * p.batch;
        int id = p.adapter[b];
        if (id < -1 || id >= p.n) {
            if (lane == 0) atomicCAS(&g_device_status, 0, kErrIndex);
            id = -1;
        }
        float s = 0.f;
        if (id >= 0) {
            const __half* a = p.a + (int64_t(id) * p.rank + r) * p.d + lane * 8;
            const __half* x = p.x + b * p.d + lane * 8;
            auto add = [&](uint4 av, uint4 xv) {
                const __half2* ah = reinterpret_cast<const __half2*>(&av);
                const __half2* xh = reinterpret_cast<const __half2*>(&xv);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 u = __half22float2(ah[e]), v = __half22float2(xh[e]);
                    s = fmaf(u.x, v.x, s);
                    s = fmaf(u.y, v.y, s);
                }
            };
            const int n = int(p.d / 256);                  // rounds of the warp, eight in flight
            int k = 0;
            for (; k + 8 <= n; k += 8) {
                uint4 av[8], xv[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    av[u] = __ldg(reinterpret_cast<const uint4*>(a + (k + u) * 256));
                    xv[u] = __ldg(reinterpret_cast<const uint4*>(x + (k + u) * 256));
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) add(av[u], xv[u]);
            }
            for (; k * 256 + lane * 8 < p.d; ++k)
                add(__ldg(reinterpret_cast<const uint4*>(a + k * 256)),
                    __ldg(reinterpret_cast<const uint4*>(x + k * 256)));
            s *= p.scaling[id];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) p.t[b * p.rank + r] = s;
    }
}

template <int NT, int FOLD>
__global__ void __launch_bounds__(W4_THREADS, 1)
lora_product_kernel(const __grid_constant__ CUtensorMap tm, const LoraParams p)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort;
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int nsteps = int(p.d / W4_STEP);
    uint4* x = reinterpret_cast<uint4*>(smem + w4_at_x(NT));
    float* xs = reinterpret_cast<float*>(smem + w4_at_x(NT) + w4_x_bytes(p.slice, p.chunk, false));
    W4Pipe pipe = w4_pipe<NT>(smem, &abort);
    // units in the order (slice, chunk of x, row group), shared evenly
    pdl_go();
    const int64_t units = int64_t(p.slices) * p.groups * p.chunks;
    int64_t u = units * blockIdx.x / gridDim.x;
    const int64_t u1 = units * (blockIdx.x + 1) / gridDim.x;
    bool shrunk = false;
    while (u < u1) {
        // a run of row groups of one (chunk, slice)
        const int64_t cs = u / p.groups;
        const int g0 = int(u - cs * p.groups);
        const int g1 = int(min(int64_t(p.groups), g0 + min(u1 - u, int64_t(p.run))));
        const int c = int(cs % p.chunks), sl = int(cs / p.chunks);
        const int k0 = sl * p.slice, steps = min(p.slice, nsteps - k0);
        const int64_t b0 = int64_t(c) * p.chunk;
        const int cols = int(min(int64_t(p.chunk), p.batch - b0));
        const W4Stage st{smem_u32(x), smem_u32(xs), cols, 0u};
        w4_sweep<NT, LORA_KW, FOLD, W4_WHOLE, false>(
            pipe, &tm, p.lay, int64_t(g0) * LORA_ROWS, p.m, 0u, st, g1 - g0, k0, steps,
            [&]() {
                if (!shrunk) {                             // beside the first copies
                    if (p.xp) pdl_wait();                  // what the front kernel wrote
                    else lora_shrink_few(p);
                    shrunk = true;
                }
                const __half* src = p.xp ? p.xp : p.x;
                w4_stage_half<NT, FOLD>(x, xs, [&](int n) { return src + (b0 + n) * p.d; }, nullptr,
                                        k0 * W4_STEP, steps, cols, int(p.d));
                __syncthreads();
            },
            [&](int grp, int r, int n, float v) {
                const int64_t row = int64_t(g0 + grp) * LORA_ROWS + r;
                if (n < cols && row < p.m) p.part[(int64_t(sl) * p.batch + b0 + n) * p.m + row] = v;
            });
        u += g1 - g0;
    }
    if (!shrunk && p.xp) pdl_wait();
    else if (!shrunk) lora_shrink_few(p);
}

// t, and the activations in the order of the product that follows, eight at a time
__global__ void __launch_bounds__(W4_THREADS, 2) lora_front_kernel(const LoraParams p)
{
    __shared__ __align__(16) float red[W4_WARPS * 128];
    __shared__ int ids[8];
    pdl_go();
    const int64_t total = p.batch * p.d;
    for (int64_t i = (int64_t(blockIdx.x) * W4_THREADS + threadIdx.x) * 8; i < total;
         i += int64_t(gridDim.x) * (W4_THREADS * 8)) {
        alignas(16) __half h[8];
        if (p.perm) {
            const int64_t b = i / p.d;
            const int k = int(i - b * p.d);
            const int4 lo = *reinterpret_cast<const int4*>(p.perm + k);
            const int4 hi = *reinterpret_cast<const int4*>(p.perm + k + 4);
            const int at[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = p.tc ? at[(j & 1) ? 4 + (j >> 1) : (j >> 1)] : at[j];
                const bool ok = c >= 0 && c < p.d;         // a bad index is not followed
                if (!ok) atomicCAS(&g_device_status, 0, kErrIndex);
                h[j] = ok ? p.x[b * p.d + c] : __ushort_as_half(0);
            }
        } else {                                           // (the tcgen05 product)
            const uint4 v = *reinterpret_cast<const uint4*>(p.x + i);
            const __half* s = reinterpret_cast<const __half*>(&v);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = s[(j & 1) ? 4 + (j >> 1) : (j >> 1)];
        }
        *reinterpret_cast<uint4*>(p.xp + i) = *reinterpret_cast<const uint4*>(h);
    }
    if (p.tc) lora_shrink(p, red, ids);
    else lora_shrink_few(p);
}

// y[b][r] = sum of part over the slices + B_a[r] . t[b].  A CTA has 128 rows r and
// LORA_JOIN rows b.  B_a is read whole lines at a time: a row's 16-byte chunks lie in
// neighbouring lanes (LANES of them, a power of two), whose sums are joined by shuffles
// and meet the slices' sums, one row r a thread, in shared memory (one thread per row of
// B: 32 lines a load, 20 us against 8 for 93 rows of rank 64).
template <int LANES> __global__ void __launch_bounds__(LORA_JOIN_ROWS) lora_join_kernel(const LoraParams p)
{
    __shared__ float4 ts[LORA_JOIN][LORA_MAX_RANK / 4];
    __shared__ float low[LORA_JOIN][LORA_JOIN_ROWS];
    const int tid = threadIdx.x;
    const int64_t r0 = int64_t(blockIdx.x) * LORA_JOIN_ROWS, r = r0 + tid;
    const int64_t b0 = int64_t(blockIdx.y) * LORA_JOIN;
    const int rows = int(min(int64_t(LORA_JOIN), p.batch - b0)), chunks = p.rank / 8;
    int id[LORA_JOIN];
    bool any = false;
#pragma unroll
    for (int i = 0; i < LORA_JOIN; ++i) {
        id[i] = i < rows ? p.adapter[b0 + i] : -1;
        if (id[i] >= p.n) id[i] = -1;
        any = any || id[i] >= 0;
    }
    pdl_wait();
    float y[LORA_JOIN] = {};
    if (r < p.m) {
        const float* src = p.part + b0 * p.m + r;
        const int64_t slice = p.batch * p.m;
#pragma unroll 4
        for (int s = 0; s < p.slices; ++s, src += slice)
#pragma unroll
            for (int i = 0; i < LORA_JOIN; ++i)
                if (i < rows) y[i] += src[i * p.m];
    }
    if (any) {                                             // (of the CTA)
        for (int i = tid; i < rows * (p.rank / 4); i += LORA_JOIN_ROWS)
            ts[i / (p.rank / 4)][i % (p.rank / 4)] =
                *reinterpret_cast<const float4*>(p.t + b0 * p.rank + int64_t(i) * 4);
        __syncthreads();
        const int c0 = tid % LANES;
#pragma unroll 4
        for (int pass = 0; pass < LANES; ++pass) {
            const int row = pass * (LORA_JOIN_ROWS / LANES) + tid / LANES;
            const int64_t at = min(r0 + row, p.m - 1);
            float v[LORA_JOIN] = {};
            for (int c = c0; c < chunks; c += LANES) {
                uint4 bv[LORA_JOIN];
#pragma unroll
                for (int i = 0; i < LORA_JOIN; ++i)        // all on their way before the first is used
                    if (id[i] >= 0 && (i == 0 || id[i] != id[i - 1]))
                        bv[i] = __ldg(reinterpret_cast<const uint4*>(
                            p.b + (int64_t(id[i]) * p.m + at) * p.rank + c * 8));
#pragma unroll
                for (int i = 0; i < LORA_JOIN; ++i) {
                    if (id[i] < 0) continue;
                    if (i > 0 && id[i] == id[i - 1]) bv[i] = bv[i - 1];   // neighbours share the load
                    const float4 t0 = ts[i][2 * c], t1 = ts[i][2 * c + 1];
                    const __half2* h = reinterpret_cast<const __half2*>(&bv[i]);
                    const float2 v0 = __half22float2(h[0]), v1 = __half22float2(h[1]);
                    const float2 v2 = __half22float2(h[2]), v3 = __half22float2(h[3]);
                    v[i] = fmaf(v0.x, t0.x, v[i]); v[i] = fmaf(v0.y, t0.y, v[i]);
                    v[i] = fmaf(v1.x, t0.z, v[i]); v[i] = fmaf(v1.y, t0.w, v[i]);
                    v[i] = fmaf(v2.x, t1.x, v[i]); v[i] = fmaf(v2.y, t1.y, v[i]);
                    v[i] = fmaf(v3.x, t1.z, v[i]); v[i] = fmaf(v3.y, t1.w, v[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < LORA_JOIN; ++i) {
#pragma unroll
                for (int o = 1; o < LANES; o <<= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
                if (c0 == 0) low[i][row] = v[i];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < LORA_JOIN; ++i)
            if (id[i] >= 0) y[i] += low[i][tid];
    }
    if (r < p.m)
#pragma unroll
        for (int i = 0; i < LORA_JOIN; ++i)
            if (i < rows) p.y[(b0 + i) * p.m + r] = y[i];
}

// The same for many rows of x, eight a CTA, on m16n8k16 mma.sync: the rows of B_a by t,
// which is split into two fp16 parts (22 bits) after a power of two has taken its largest
// element to 2^13 .. 2^14.  A run of rows with one adapter shares the loads of B_a; the
// other rows are computed along and dropped (on FMA units, like the few rows' join: 17 us
// against 8 for 93 rows of rank 64).
__global__ void __launch_bounds__(LORA_JOIN_ROWS) lora_join_many_kernel(const LoraParams p)
{
    constexpr int J = LORA_MANY;
    __shared__ uint4 th[J][LORA_MAX_RANK / 8 + 1], tl[J][LORA_MAX_RANK / 8 + 1];
    __shared__ float low[J][LORA_JOIN_ROWS], back[J];
    __shared__ int ids[J];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int64_t r0 = int64_t(blockIdx.x) * LORA_JOIN_ROWS, r = r0 + tid;
    const int64_t b0 = int64_t(blockIdx.y) * J;
    const int rows = int(min(int64_t(J), p.batch - b0)), chunks = p.rank / 8;
    if (tid < J) {
        const int id = tid < rows ? p.adapter[b0 + tid] : -1;
        ids[tid] = id < p.n ? id : -1;
    }
    pdl_wait();
    float y[J] = {};
    if (r < p.m) {
        const float* src = p.part + b0 * p.m + r;
        const int64_t slice = p.batch * p.m;
#pragma unroll 4
        for (int s = 0; s < p.slices; ++s, src += slice)
#pragma unroll
            for (int i = 0; i < J; ++i)
                if (i < rows) y[i] += src[i * p.m];
    }
    __syncthreads();
    for (int i = warp; i < rows; i += LORA_JOIN_ROWS / 32) {   // a lane's chunk of 8 elements
        if (ids[i] < 0) continue;
        float v[8] = {}, top = 0.f;
        if (lane < chunks) {
            const float* src = p.t + (b0 + i) * p.rank + lane * 8;
#pragma unroll
            for (int s = 0; s < LORA_TC_PARTS; ++s, src += p.batch * p.rank) {
                const float4 u = *reinterpret_cast<const float4*>(src);
                const float4 w = *reinterpret_cast<const float4*>(src + 4);
                v[0] += u.x; v[1] += u.y; v[2] += u.z; v[3] += u.w;
                v[4] += w.x; v[5] += w.y; v[6] += w.z; v[7] += w.w;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (isfinite(v[e])) top = fmaxf(top, fabsf(v[e]));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int ex = top > 0.f ? max(-126, min(126, 13 - ilogbf(top))) : 0;
        const float scale = __int_as_float((127 + ex) << 23);
        if (lane == 0) back[i] = __int_as_float((127 - ex) << 23);
        alignas(16) __half hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float w = v[e] * scale;
            hi[e] = __float2half_rn(w);
            lo[e] = __float2half_rn(isfinite(w) ? w - __half2float(hi[e]) : 0.f);
        }
        if (lane < chunks) {
            th[i][lane] = *reinterpret_cast<const uint4*>(hi);
            tl[i][lane] = *reinterpret_cast<const uint4*>(lo);
        }
    }
    __syncthreads();
    const uint4 none = make_uint4(0, 0, 0, 0);
    for (int i0 = 0, i1; i0 < rows; i0 = i1) {             // a run of one adapter
        const int id = ids[i0];
        for (i1 = i0 + 1; i1 < rows && ids[i1] == id; ++i1) {}
        if (id < 0) continue;
        const __half* src[4];                              // rows g and g + 8 of the warp's two tiles
#pragma unroll
        for (int q = 0; q < 4; ++q)
            src[q] = p.b + (int64_t(id) * p.m + min(r0 + warp * 32 + q * 8 + g, p.m - 1)) * p.rank;
        float acc[2][4] = {};
#pragma unroll 2
        for (int c = t; c - t < chunks; c += 4) {          // 32 columns of B_a
            const bool in = c < chunks;
            uint4 bv[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                bv[q] = in ? __ldg(reinterpret_cast<const uint4*>(src[q] + c * 8)) : none;
            const uint4 h = in && g < rows ? th[g][c] : none, l = in && g < rows ? tl[g][c] : none;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                mma_16816(acc[q], bv[2 * q].x, bv[2 * q + 1].x, bv[2 * q].y, bv[2 * q + 1].y, h.x, h.y);
                mma_16816(acc[q], bv[2 * q].z, bv[2 * q + 1].z, bv[2 * q].w, bv[2 * q + 1].w, h.z, h.w);
                mma_16816(acc[q], bv[2 * q].x, bv[2 * q + 1].x, bv[2 * q].y, bv[2 * q + 1].y, l.x, l.y);
                mma_16816(acc[q], bv[2 * q].z, bv[2 * q + 1].z, bv[2 * q].w, bv[2 * q + 1].w, l.z, l.w);
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 2 * t + (e & 1);
                if (i >= i0 && i < i1)
                    low[i][warp * 32 + q * 16 + g + 8 * (e >> 1)] = acc[q][e] * back[i];
            }
    }
    __syncthreads();
    if (r < p.m)
#pragma unroll
        for (int i = 0; i < J; ++i)
            if (i < rows) p.y[(b0 + i) * p.m + r] = ids[i] >= 0 ? y[i] + low[i][tid] : y[i];
}

struct LoraPlan {
    bool tc;                                     // the tcgen05 product
    WqPlan wq;
    int nt, chunk, chunks, slice, slices, groups;
    size_t at_xp, at_part;
};

// Rows of x that the sweep stages together (one operand of 8, or two)
struct LoraChunk {
    int nt, rows;
    int slices, most;        // slices of the columns: the fewest that fit beside the ring, the most
                             // that a plan has (steps of fewer columns than the shares gain nothing)
};

LoraChunk lora_chunk(int64_t T, int64_t d)
{
    LoraChunk c{};
    c.nt = T > W4_COLS ? 2 : 1;
    c.rows = int(std::min<int64_t>(T, W4_COLS * c.nt));
    const int so = int(d / W4_STEP), room = (c.nt == 1 ? 72 : 56) * 1024;
    const int steps = std::min(so, room / (256 * c.rows + 128 * c.nt));
    c.slices = (so + steps - 1) / steps;
    c.most = std::max(c.slices, (so + LORA_KW - 1) / LORA_KW);
    return c;
}

bool lora_tc(int64_t T, int64_t g) { return T > LORA_SWEEP && g % 64 == 0; }

// Slices of the columns: as few as fit, or more where few row groups would leave
// CTAs idle.  A group costs about 190 instructions a step and warp (two operands:
// 260, bound by the matrix pipe) and 150 to join, and the slowest CTA counts.
// More than 16 rows: the tcgen05 product, which needs groups of a multiple of 64.  Whole
// calls, the sweep against that product: 14336 x 4096, rank 16: 36 us against 57 at 16
// rows, 55 against 58 at 24, 60 against 58 at 32, 178 against 86 at 128; 4096 x 4096: 19
// against 31, 25 against 31, 26 against 33, 62 against 38; 4096 x 11008, rank 64, groups of
// 64: 52 against 61, 63 against 64, 65 against 65, 158 against 77.  (Every row with an
// adapter of its own but for eight; the limit could be 24.)
LoraPlan lora_plan(int64_t T, int64_t m, int64_t d, int64_t g, int rank)
{
    LoraPlan p{};
    p.tc = lora_tc(T, g);
    p.at_xp = align_up(size_t(T) * rank * 4 * (p.tc ? LORA_TC_PARTS : 1), 256);
    p.at_part = p.at_xp + align_up(size_t(T) * d * 2, 1024);
    if (p.tc) {
        p.wq = wq_plan(T, m, d, g, LORA_SMS);
        p.slices = p.wq.ksplit;
        return p;
    }
    const LoraChunk c = lora_chunk(T, d);
    p.nt = c.nt;
    p.chunk = c.rows;
    p.chunks = int((T + p.chunk - 1) / p.chunk);
    p.groups = int((m + LORA_ROWS - 1) / LORA_ROWS);
    const int so = int(d / W4_STEP);
    double best = 1e300;
    for (int s = c.slices; s <= c.most; ++s) {
        const int steps = (so + s - 1) / s;
        const int64_t rounds = ((int64_t(p.chunks) * s * p.groups) + LORA_SMS - 1) / LORA_SMS;
        const double cost = double(rounds) * (((steps + LORA_KW - 1) / LORA_KW) * (p.nt == 1 ? 190 : 260) + 150);
        if (cost < best * 0.97) { best = cost; p.slice = steps; }
    }
    p.slices = (so + p.slice - 1) / p.slice;
    return p;
}

// Bytes that serve T rows and every smaller batch: each part's largest.  The tcgen05
// product splits K into more parts where its tiles are few, a tile more per 128 rows.
size_t lora_bytes(int64_t T, int64_t m, int64_t d, int64_t g, int rank)
{
    const bool tc = lora_tc(T, g);
    const size_t front = align_up(size_t(T) * rank * 4 * (tc ? LORA_TC_PARTS : 1), 256) +
                         align_up(size_t(T) * d * 2, 1024);
    int64_t rows = 0;                            // of partial results: slices x rows of x
    auto add = [&](int64_t slices, int64_t n) { if (slices > 1) rows = std::max(rows, slices * n); };
    const int64_t sweep = tc ? LORA_SWEEP : T;
    add(lora_chunk(sweep, d).most, sweep);
    if (tc)
        for (int64_t n = std::min<int64_t>(T, 128);; n = std::min(T, n + 128)) {
            const WqPlan wq = wq_plan(n, m, d, g, LORA_SMS);
            add(wq.ksplit, n);
            if (n == T || int64_t(wq.n_rt) * wq.n_nt >= 2 * LORA_SMS) break;   // (no splits from here on)
        }
    return front + align_up(size_t(rows) * m * 4, 256);
}

}  // namespace gptq

extern "C" size_t gptq_w4a16_lora_workspace_bytes(int64_t batch, int64_t d_out, int64_t d_in,
                                                  int group_size, int rank)
{
    using namespace gptq;
    const int64_t g = group_size == -1 ? d_in : group_size;
    if (batch <= 0 || batch > 65535 || d_out <= 0 || d_out > kMaxRows || d_in <= 0 ||
        d_in > kMaxDim || d_in % 128 != 0 || g < 32 || g % 32 != 0 || d_in % g != 0 || rank <= 0 ||
        rank > LORA_MAX_RANK)
        return 0;
    return lora_bytes(batch, d_out, d_in, g, rank);
}

extern "C" int gptq_w4a16_lora(const uint16_t* x, int64_t batch, const uint32_t* qweight,
                               const uint16_t* scales, const uint8_t* qzeros, const int32_t* perm,
                               int64_t d_out, int64_t d_in, int group_size, const uint16_t* lora_a,
                               const uint16_t* lora_b, const float* lora_scaling,
                               const int32_t* adapter, int64_t n_adapters, int rank, float* y,
                               void* ws, size_t ws_bytes, void* stream)
{
    using namespace gptq;
    if (batch < 0 || batch > 65535 || n_adapters < 0 || n_adapters > 65536) return GPTQ_ERR_SHAPE;
    if (d_in < 128 || d_in > kMaxDim || d_in % 128 != 0 || d_out < 1 || d_out > kMaxRows)
        return GPTQ_ERR_SHAPE;
    const int64_t g = (group_size == -1) ? d_in : group_size;
    if (g < 32 || g % 32 != 0 || d_in % g != 0) return GPTQ_ERR_UNSUPPORTED;
    if (rank < 8 || rank > LORA_MAX_RANK || rank % 8 != 0) return GPTQ_ERR_UNSUPPORTED;
    if (batch == 0) return GPTQ_OK;
    if (!x || !qweight || !scales || !qzeros || !y || !ws || !adapter ||
        (n_adapters > 0 && (!lora_a || !lora_b || !lora_scaling)))
        return GPTQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(qweight) || !aligned16(scales) || !aligned16(qzeros) ||
        !aligned16(y) || !aligned16(ws) || !aligned16(perm) || !aligned16(lora_a) ||
        !aligned16(lora_b) || !aligned(lora_scaling, 4) || !aligned(adapter, 4))
        return GPTQ_ERR_INVALID_ARG;
    if (ws_bytes < lora_bytes(batch, d_out, d_in, g, rank)) return GPTQ_ERR_INVALID_ARG;
    const LoraPlan plan = lora_plan(batch, d_out, d_in, g, rank);
    LoraParams p{};
    p.x = reinterpret_cast<const __half*>(x);
    p.perm = perm;
    p.a = reinterpret_cast<const __half*>(lora_a);
    p.b = reinterpret_cast<const __half*>(lora_b);
    p.scaling = lora_scaling; p.adapter = adapter;
    p.batch = batch; p.m = d_out; p.d = d_in; p.n = n_adapters; p.rank = rank;
    p.lay = w4_layer(qweight, scales, qzeros, d_in, g);
    p.chunk = plan.chunk; p.chunks = plan.chunks; p.slice = plan.slice; p.slices = plan.slices;
    p.groups = plan.groups;
    // (a sweep's offsets into the scales are 32 bits: 2^21 rows of 32768 columns in groups of 32)
    p.run = int(std::min<int64_t>(int64_t(1) << 30, (int64_t(1) << 32) / (LORA_ROWS * 2 * p.lay.G)));
    p.t = static_cast<float*>(ws);
    p.tc = plan.tc;
    p.xp = plan.tc || perm ? reinterpret_cast<__half*>(static_cast<uint8_t*>(ws) + plan.at_xp) : nullptr;
    // one slice: in y, where the join finds it (each thread reads and writes its own elements)
    p.part = plan.slices > 1
                 ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + plan.at_part) : y;
    p.y = y;
    cudaStream_t st = as_stream(stream);
    KernelTimer kt(kKLora, st);
    if (p.xp) {
        lora_front_kernel<<<(unsigned)(device_sm_count() * (plan.tc ? 2 : 1)), W4_THREADS, 0, st>>>(p);
        count_launches();
        if (launch_status() != GPTQ_OK) return GPTQ_ERR_CUDA;
    }
    if (plan.tc) {
        const int rc = wq_run(plan.wq, p.xp, batch, qweight, p.lay.sc, qzeros, d_out, d_in, g, p.part,
                              batch * d_out, st);
        if (rc != GPTQ_OK) return rc;
    } else {
        CUtensorMap tm;
        if (w4_tmap(&tm, qweight, d_out, d_in, 32) != GPTQ_OK) return GPTQ_ERR_CUDA;
        const int fold = w4_fold(g);
        const size_t smem = w4_smem(plan.slice, plan.chunk, plan.nt, fold, false);
        if (smem > W4_MAX_SMEM) return GPTQ_ERR_SHAPE;
        auto kern = plan.nt == 1 ? (fold == 4   ? lora_product_kernel<1, 4>
                                    : fold == 2 ? lora_product_kernel<1, 2>
                                                : lora_product_kernel<1, 1>)
                                 : (fold == 4   ? lora_product_kernel<2, 4>
                                    : fold == 2 ? lora_product_kernel<2, 2>
                                                : lora_product_kernel<2, 1>);
        static std::atomic<bool> done[10][64];
        if (!smem_opt_in(reinterpret_cast<const void*>(kern), W4_MAX_SMEM,
                         done[(plan.nt - 1) * 5 + fold]))
            return GPTQ_ERR_CUDA;
        const int64_t units = int64_t(plan.chunks) * plan.slices * plan.groups;
        const unsigned grid = (unsigned)std::min<int64_t>(device_sm_count(), units);
        if (p.xp) {
            if (launch_after(kern, grid, W4_THREADS, smem, st, tm, p) != cudaSuccess)
                return GPTQ_ERR_CUDA;
        } else {
            kern<<<grid, W4_THREADS, smem, st>>>(tm, p);
        }
        count_launches();
        if (launch_status() != GPTQ_OK) return GPTQ_ERR_CUDA;
    }
    const bool many = plan.tc;
    auto join = many           ? lora_join_many_kernel
                : rank >= 64   ? lora_join_kernel<8>
                : rank >= 32   ? lora_join_kernel<4>
                : rank >= 16   ? lora_join_kernel<2>
                               : lora_join_kernel<1>;
    if (launch_after(join,
                     dim3((unsigned)ceil_div(d_out, LORA_JOIN_ROWS),
                          (unsigned)ceil_div(batch, many ? LORA_MANY : LORA_JOIN)),
                     LORA_JOIN_ROWS, 0, st, p) != cudaSuccess)
        return GPTQ_ERR_CUDA;
    count_launches();
    return launch_status();
}
