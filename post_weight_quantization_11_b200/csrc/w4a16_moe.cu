// A whole mixture-of-experts layer of packed experts for a few tokens -- top-k
// routed experts ("INT4/INT8 量化推理" sec. 五) with weights in 4 bits and fp16
// activations (sec. 六 of the same page):
//
//   p = softmax(logits), S = top_k of it,  y = sum_S w_e D_e (silu(G_e x) * U_e x)
//
// Three kernels, each begun while the one before it drains: routes and h, the second
// product over slices of its columns, and the joined y.  Every CTA of the first two works
// out the routes for itself (a warp a token; the second while the first ends, 4 us of 24
// tokens' time less than with the first's routes read behind it), the products are sweeps
// of the packed rows (w4_rows.cuh): only the experts that a token chose are read, each once
// per eight of its tokens (by the first product up to d_model 4096: rows of x are staged
// whole, and six of 5120, four of 7168, one from 16384 on fit beside the ring).  h stays
// fp32 between them, as two fp16 parts in the second.  Partial results go through memory,
// not atomics: their order is fixed.
// Measured (B200, 8 experts of 14336 x 4096, top 2, groups of 128): 56 us for one token
// (two experts, 183 MB: 3.3 TB/s), 218 us for 24 (all eight, 732 MB: 3.4 TB/s; the copies
// alone, without the products, 163); bound by the instructions that unpack (see
// w4_rows.cuh) and, for one token, by the start and end of three kernels.
#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "tc_common.cuh"
#include "w4_rows.cuh"

namespace gptq {

constexpr int kMoeTokens = 64, kMoeExperts = 256, kMoeTopK = 8;
constexpr int64_t kMoeMaxModel = 20480;     // a row of x has to fit beside the ring
// Of w4_sweep: more column shares make finer row groups, fewer make longer ones
constexpr int MOE_MAX_SMEM = W4_MAX_SMEM - 11 * 1024;     // beside the routes
template <int KW> constexpr int kMoeInRows = 16 * (W4_WARPS / KW);
constexpr int MOE_OUT_KW = 4, MOE_OUT_ROWS = 32 * (W4_WARPS / MOE_OUT_KW);
constexpr int kMoeSms = 148;               // the plan does not depend on the device that is current
constexpr int kMoePairs = kMoeTokens * kMoeTopK;

struct MoeRoutes;

struct MoeParams {
    const __half* x;
    const float* logits;
    const int32_t* pi;
    const int32_t* po;
    int64_t d, f;
    int T, E, k, renorm;
    W4Layer in, out;
    int chunk;                             // tokens of an expert that are staged together
    int slice, slices;                     // steps of a slice of the second product
    MoeRoutes* routes;
    float* h;                              // T k x f
    float* part;                           // slices x T k x d
    float* y;
};

// One warp: the routes of token t into ids / w[0 .. k)
__device__ __forceinline__ void moe_route(const float* logits, int E, int k, int renorm, int16_t* ids,
                                          float* w)
{
    constexpr uint32_t ALL = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    float l[kMoeExperts / 32];
#pragma unroll
    for (int i = 0; i < kMoeExperts / 32; ++i) {
        const int e = i * 32 + lane;
        const float v = e < E ? logits[e] : -INFINITY;
        l[i] = v != v ? -INFINITY : fminf(v, FLT_MAX);     // masked; +inf: the largest finite
    }
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kMoeExperts / 32; ++i) top = fmaxf(top, l[i]);
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(ALL, top, o));
    if (top > -INFINITY) {
#pragma unroll
        for (int i = 0; i < kMoeExperts / 32; ++i) sum += l[i] > -INFINITY ? expf(l[i] - top) : 0.f;
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(ALL, sum, o);
    }
    float mine = 0.f, chosen = 0.f;
    int id = -1;
    for (int j = 0; j < k; ++j) {                          // the j-th largest; ties: lowest index
        float v = -INFINITY;
        int at = kMoeExperts;
#pragma unroll
        for (int i = 0; i < kMoeExperts / 32; ++i)
            if (l[i] > v) { v = l[i]; at = i * 32 + lane; }
        for (int o = 16; o; o >>= 1) {
            const float v2 = __shfl_xor_sync(ALL, v, o);
            const int a2 = __shfl_xor_sync(ALL, at, o);
            if (v2 > v || (v2 == v && a2 < at)) { v = v2; at = a2; }
        }
        if (!(v > -INFINITY)) break;                       // no expert left (whole warp)
        const float e = expf(v - top);
        chosen += e;
        if (lane == j) { id = at; mine = e; }
#pragma unroll
        for (int i = 0; i < kMoeExperts / 32; ++i)
            if (i * 32 + lane == at) l[i] = -INFINITY;
    }
    if (lane < k) {
        ids[lane] = id;
        w[lane] = id < 0 ? 0.f : mine / (renorm ? chosen : sum);
    }
}

// The routes: chunks of up to p.chunk pairs of one expert, in expert order
struct MoeRoutes {
    int chunks;
    int16_t expert[kMoePairs];
    int16_t start[kMoePairs];              // in list
    int16_t n[kMoePairs];
    int16_t list[kMoePairs];               // pairs (t k + j), expert by expert
    int16_t id[kMoePairs];                 // expert of each pair, -1: none
    float w[kMoePairs];
};

// All threads: routes of all tokens and the chunks, in shared memory
__device__ __forceinline__ void moe_routes(const MoeParams& p, MoeRoutes& r, int* cnt, int* off,
                                           int* coff)
{
    const int tid = threadIdx.x, lane = tid & 31, pairs = p.T * p.k;
    for (int e = tid; e < p.E; e += blockDim.x) cnt[e] = 0;
    for (int t = tid >> 5; t < p.T; t += blockDim.x >> 5)
        moe_route(p.logits + int64_t(t) * p.E, p.E, p.k, p.renorm, r.id + t * p.k, r.w + t * p.k);
    __syncthreads();
    int pos[kMoePairs / 32];                               // of the first warp: place in the expert's list
    if (tid < 32) {                                        // in pair order: every CTA has the same lists
#pragma unroll
        for (int u = 0; u < kMoePairs / 32; ++u) {
            const int i = u * 32 + lane;
            const int id = i < pairs ? r.id[i] : -1;
            if (u * 32 >= pairs) break;
            const uint32_t same = __match_any_sync(0xffffffffu, id);
            const int before = __popc(same & ((1u << lane) - 1u));
            pos[u] = id >= 0 ? cnt[id] + before : -1;
            __syncwarp();
            if (id >= 0 && before == 0) cnt[id] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    if (tid < 32) {                                        // prefix sums over the experts
        const int per = (p.E + 31) / 32, e0 = lane * per, e1 = min(p.E, e0 + per);
        int a = 0, c = 0;
        for (int e = e0; e < e1; ++e) { a += cnt[e]; c += (cnt[e] + p.chunk - 1) / p.chunk; }
        int pa = a, pc = c;
        for (int o = 1; o < 32; o <<= 1) {
            const int va = __shfl_up_sync(0xffffffffu, pa, o), vc = __shfl_up_sync(0xffffffffu, pc, o);
            if (lane >= o) { pa += va; pc += vc; }
        }
        if (lane == 31) r.chunks = pc;
        pa -= a;
        pc -= c;
        for (int e = e0; e < e1; ++e) {
            off[e] = pa;
            coff[e] = pc;
            pa += cnt[e];
            pc += (cnt[e] + p.chunk - 1) / p.chunk;
        }
    }
    __syncthreads();
    if (tid < 32) {
#pragma unroll
        for (int u = 0; u < kMoePairs / 32; ++u) {
            const int i = u * 32 + lane;
            if (i < pairs && pos[u] >= 0) r.list[off[r.id[i]] + pos[u]] = i;
        }
    }
    for (int e = tid; e < p.E; e += blockDim.x)
        for (int c = 0, left = cnt[e]; left > 0; ++c, left -= p.chunk) {
            r.expert[coff[e] + c] = e;
            r.start[coff[e] + c] = off[e] + c * p.chunk;
            r.n[coff[e] + c] = min(left, p.chunk);
        }
    __syncthreads();
}

// h = silu(G x) (U x) of every pair.  A row tile is 8 gate rows and the same 8
// up rows, so that a lane holds both of an element of h.  The CTAs share the
// row tiles of all chunks evenly; a CTA stages a chunk's tokens once.
template <int KW, int FOLD>
__global__ void __launch_bounds__(W4_THREADS, 1) moe_in_kernel(const __grid_constant__ CUtensorMap tm, const MoeParams p)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort;
    __shared__ MoeRoutes r;
    __shared__ int cnt[kMoeExperts], off[kMoeExperts], coff[kMoeExperts];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int steps = int(p.d / W4_STEP), groups = int(p.f / kMoeInRows<KW>);
    uint4* x = reinterpret_cast<uint4*>(smem + w4_at_x(1));
    float* xs = reinterpret_cast<float*>(smem + w4_at_x(1) + w4_x_bytes(steps, p.chunk, false));
    W4Pipe pipe = w4_pipe<1>(smem, &abort);
    pdl_go();
    moe_routes(p, r, cnt, off, coff);
    if (blockIdx.x == 0) {                                 // for the joining kernel
        const int* src = reinterpret_cast<const int*>(&r);
        for (int i = threadIdx.x; i < int(sizeof(MoeRoutes) / 4); i += blockDim.x)
            reinterpret_cast<int*>(p.routes)[i] = src[i];
    }
    const int64_t units = int64_t(r.chunks) * groups;
    int64_t u = units * blockIdx.x / gridDim.x;
    const int64_t u1 = units * (blockIdx.x + 1) / gridDim.x;
    while (u < u1) {
        const int c = int(u / groups), g0 = int(u - int64_t(c) * groups);
        const int g1 = int(min(int64_t(groups), g0 + (u1 - u)));
        const int e = r.expert[c], cols = r.n[c];
        const int16_t* list = r.list + r.start[c];
        const int64_t row0 = int64_t(e) * 2 * p.f;
        const W4Stage st{smem_u32(x), smem_u32(xs), cols, 0};
        w4_sweep<1, KW, FOLD, W4_WHOLE, true>(
            pipe, &tm, p.in, row0 + int64_t(g0) * kMoeInRows<KW>, row0 + 2 * p.f, uint32_t(p.f), st,
            g1 - g0, 0, steps,
            [&]() {
                w4_stage_half<1, FOLD>(
                    x, xs, [&](int n) { return p.x + int64_t(list[n] / p.k) * p.d; },
                    p.pi ? p.pi + e * p.d : nullptr, 0, steps, cols, int(p.d));
                __syncthreads();
            },
            [&](int grp, int r, int n, float gate, float up) {
                if (n < cols)
                    p.h[int64_t(list[n]) * p.f + int64_t(g0 + grp) * kMoeInRows<KW> + r] =
                        gate / (1.f + expf(-gate)) * up;
            });
        u += g1 - g0;
    }
}

// part[slice][pair] = D h over a slice of the columns
template <int FOLD>
__global__ void __launch_bounds__(W4_THREADS, 1) moe_out_kernel(const __grid_constant__ CUtensorMap tm, const MoeParams p)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort;
    __shared__ MoeRoutes r;
    __shared__ int cnt[kMoeExperts], off[kMoeExperts], coff[kMoeExperts];
    __shared__ float undo[8];
    __shared__ uint32_t top[8];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int groups = int(p.d / MOE_OUT_ROWS), nsteps = int(p.f / W4_STEP);
    uint4* x = reinterpret_cast<uint4*>(smem + w4_at_x(1));
    float* xs = reinterpret_cast<float*>(smem + w4_at_x(1) + w4_x_bytes(p.slice, p.chunk, true));
    W4Pipe pipe = w4_pipe<1>(smem, &abort);
    pdl_go();
    moe_routes(p, r, cnt, off, coff);                      // again, while the first kernel ends
    bool waited = false;
    const int64_t units = int64_t(r.chunks) * p.slices * groups;
    int64_t u = units * blockIdx.x / gridDim.x;
    const int64_t u1 = units * (blockIdx.x + 1) / gridDim.x;
    while (u < u1) {
        const int cs = int(u / groups), g0 = int(u - int64_t(cs) * groups);
        const int g1 = int(min(int64_t(groups), g0 + (u1 - u)));
        const int c = cs / p.slices, sl = cs - c * p.slices;
        const int e = r.expert[c], cols = r.n[c];
        const int k0 = sl * p.slice, steps = min(p.slice, nsteps - k0);
        const int16_t* list = r.list + r.start[c];
        const int64_t row0 = int64_t(e) * p.d;
        const W4Stage st{smem_u32(x), smem_u32(xs), cols, uint32_t(steps * 256 * cols)};
        auto stage = [&]() {
            if (!waited) pdl_wait();                       // for h
            waited = true;
            w4_stage_split<1, FOLD>(
                x, xs, undo, top, [&](int n) { return p.h + int64_t(list[n]) * p.f; },
                p.po ? p.po + e * p.f : nullptr, k0 * W4_STEP, steps, cols, int(p.f), cols <= 4);
            __syncthreads();
        };
        auto done = [&](int grp, int r, int n, float v) {
            if (n < cols)
                p.part[(int64_t(sl) * p.T * p.k + list[n]) * p.d + int64_t(g0 + grp) * MOE_OUT_ROWS +
                       r] = v * undo[n];
        };
        const int64_t first = row0 + int64_t(g0) * MOE_OUT_ROWS;
        if (cols <= 4)
            w4_sweep<1, MOE_OUT_KW, FOLD, W4_BESIDE, false>(pipe, &tm, p.out, first, row0 + p.d, 0u, st,
                                                            g1 - g0, k0, steps, stage, done);
        else
            w4_sweep<1, MOE_OUT_KW, FOLD, W4_TWICE, false>(pipe, &tm, p.out, first, row0 + p.d, 0u, st,
                                                           g1 - g0, k0, steps, stage, done);
        u += g1 - g0;
    }
    if (!waited) pdl_wait();
}

// y[t] = sum over the token's experts of w (sum over the slices of part)
__global__ void __launch_bounds__(256) moe_join_kernel(const MoeParams p)
{
    pdl_wait();
    const int64_t r = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int t = blockIdx.y;
    if (r >= p.d) return;
    float y = 0.f;
    for (int j = 0; j < p.k; ++j) {
        const int pair = t * p.k + j;
        if (p.routes->id[pair] < 0) continue;
        float s = 0.f;
        for (int sl = 0; sl < p.slices; ++sl) s += p.part[(int64_t(sl) * p.T * p.k + pair) * p.d + r];
        y = fmaf(p.routes->w[pair], s, y);
    }
    p.y[t * p.d + r] = y;
}

static_assert(sizeof(MoeRoutes) + 3 * 4 * kMoeExperts + 256 <= 11 * 1024 - 256, "static shared memory");

struct MoePlan {
    int chunk, slices, slice;
    size_t smem_in, smem_out, at_h, at_part, bytes;
};

// Tokens of an expert that are staged together (up to 8, the columns of one
// product; fewer where a row of x is so long that they would not fit beside the
// ring) and slices of the second product's columns: as few as fit, or more where
// few row groups would leave CTAs idle.  A group of a slice costs about 190
// instructions a step and warp and 100 to join, and the slowest CTA counts.
MoePlan moe_plan(int64_t T, int64_t E, int k, int64_t d, int64_t f)
{
    constexpr int MOST = 68 * 1024;                        // bytes of staged activations and sums
    MoePlan m{};
    const int si = int(d / W4_STEP), so = int(f / W4_STEP);
    m.chunk = int(std::min<int64_t>(std::min<int64_t>(T, W4_COLS), (MOST / si - 128) / 256));
    const int most = std::min(so, MOST / (512 * m.chunk + 128));
    const int64_t chunks = std::max(std::min(T * k, E), ceil_div(T * k, m.chunk));
    double best = 1e300;
    const int fewest = (so + most - 1) / most;             // (slices under 2 KW steps gain nothing)
    const int top = std::max(fewest, (so + 2 * MOE_OUT_KW - 1) / (2 * MOE_OUT_KW));
    for (int s = fewest; s <= top; ++s) {
        const int steps = (so + s - 1) / s;
        const int64_t rounds = ceil_div(chunks * s * (d / MOE_OUT_ROWS), kMoeSms);
        const double cost = double(rounds) * (((steps + 2 * MOE_OUT_KW - 1) / (2 * MOE_OUT_KW)) * 2 * 190 + 100);
        if (cost < best * 0.97) { best = cost; m.slice = steps; }
    }
    m.slices = (so + m.slice - 1) / m.slice;
    m.smem_in = w4_smem(si, m.chunk, 1, 1, false);
    m.smem_out = w4_smem(m.slice, m.chunk, 1, 1, true);
    const size_t pairs = size_t(T) * k;
    m.at_h = align_up(sizeof(MoeRoutes), 256);
    m.at_part = m.at_h + align_up(pairs * f * 4, 256);
    // the most slices that a plan may have: a workspace that serves fewer tokens too
    m.bytes = m.at_part + align_up(size_t(top) * pairs * d * 4, 256);
    return m;
}

}  // namespace gptq

extern "C" size_t gptq_w4a16_moe_workspace_bytes(int64_t tokens, int64_t n_experts, int top_k,
                                                 int64_t d_model, int64_t d_ff)
{
    if (tokens <= 0 || n_experts <= 0 || top_k <= 0 || d_model <= 0 || d_ff <= 0) return 0;
    if (tokens > gptq::kMoeTokens || top_k > gptq::kMoeTopK || n_experts > gptq::kMoeExperts || d_model % 128 != 0 ||
        d_ff % 128 != 0 || d_model > gptq::kMoeMaxModel || d_ff > gptq::kMaxDim)
        return 0;
    return gptq::moe_plan(tokens, n_experts, top_k, d_model, d_ff).bytes;
}

extern "C" int gptq_w4a16_moe(const uint16_t* x, int64_t tokens, const float* logits,
                              int64_t n_experts, int top_k, int renormalize,
                              const uint32_t* qweight_in, const uint16_t* scales_in,
                              const uint8_t* qzeros_in, const int32_t* perm_in,
                              const uint32_t* qweight_out, const uint16_t* scales_out,
                              const uint8_t* qzeros_out, const int32_t* perm_out, int64_t d_model,
                              int64_t d_ff, int group_size, float* y, void* ws, size_t ws_bytes,
                              void* stream)
{
    using namespace gptq;
    if (d_model < 128 || d_model > kMoeMaxModel || d_model % 128 != 0 || d_ff < 128 || d_ff > kMaxDim ||
        d_ff % 128 != 0 || tokens < 0 || n_experts < 1 || top_k < 1)
        return GPTQ_ERR_SHAPE;
    if (tokens > kMoeTokens || n_experts > kMoeExperts || top_k > kMoeTopK || top_k > n_experts)
        return GPTQ_ERR_UNSUPPORTED;
    const int64_t gi = group_size == -1 ? d_model : group_size;
    const int64_t go = group_size == -1 ? d_ff : group_size;
    if (gi < 32 || gi % 32 != 0 || d_model % gi != 0 || d_ff % go != 0) return GPTQ_ERR_UNSUPPORTED;
    if (tokens == 0) return GPTQ_OK;
    if (!x || !logits || !qweight_in || !scales_in || !qzeros_in || !qweight_out || !scales_out ||
        !qzeros_out || !y || !ws)
        return GPTQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned(logits, 4) || !aligned16(qweight_in) || !aligned16(scales_in) ||
        !aligned16(qzeros_in) || !aligned16(perm_in) || !aligned16(qweight_out) ||
        !aligned16(scales_out) || !aligned16(qzeros_out) || !aligned16(perm_out) || !aligned16(y) ||
        !aligned16(ws))
        return GPTQ_ERR_INVALID_ARG;
    if (ws_bytes < gptq_w4a16_moe_workspace_bytes(tokens, n_experts, top_k, d_model, d_ff))
        return GPTQ_ERR_INVALID_ARG;
    const MoePlan plan = moe_plan(tokens, n_experts, top_k, d_model, d_ff);
    MoeParams p{};
    p.x = reinterpret_cast<const __half*>(x);
    p.logits = logits;
    p.pi = perm_in;
    p.po = perm_out;
    p.d = d_model; p.f = d_ff;
    p.T = (int)tokens; p.E = (int)n_experts; p.k = top_k; p.renorm = renormalize != 0;
    p.in = w4_layer(qweight_in, scales_in, qzeros_in, d_model, gi);
    p.out = w4_layer(qweight_out, scales_out, qzeros_out, d_ff, go);
    p.chunk = plan.chunk; p.slice = plan.slice; p.slices = plan.slices;
    uint8_t* w = static_cast<uint8_t*>(ws);
    p.routes = reinterpret_cast<MoeRoutes*>(w);
    p.h = reinterpret_cast<float*>(w + plan.at_h);
    p.part = reinterpret_cast<float*>(w + plan.at_part);
    p.y = y;
    cudaStream_t st = as_stream(stream);
    KernelTimer kt(kKMoe, st);
    const int sms = device_sm_count();
    auto ctas = [&](int64_t units) { return (unsigned)std::min<int64_t>(sms, units); };
    // Four column shares (64 rows of h a group, half the joins) or eight (32 rows, finer
    // rounds): by the slowest CTA's share, at the costs in moe_plan (24 tokens of 8 experts
    // of 14336: 218 us with four, 221 with eight; one token: 56.7 and 56.1)
    const int64_t pairs = tokens * top_k;
    const int64_t chunks = std::max(std::min(pairs, n_experts), ceil_div(pairs, plan.chunk));
    auto cost = [&](int kw, int rows) {
        return ceil_div(chunks * (d_ff / rows), sms) * (ceil_div(d_model / W4_STEP, kw) * 190 + 100);
    };
    const bool fine = cost(8, kMoeInRows<8>) < cost(4, kMoeInRows<4>);
    const int fi = w4_fold(gi), fo = w4_fold(go);
    auto in = fine ? (fi == 4 ? moe_in_kernel<8, 4> : fi == 2 ? moe_in_kernel<8, 2> : moe_in_kernel<8, 1>)
                   : (fi == 4 ? moe_in_kernel<4, 4> : fi == 2 ? moe_in_kernel<4, 2> : moe_in_kernel<4, 1>);
    auto out = fo == 4 ? moe_out_kernel<4> : fo == 2 ? moe_out_kernel<2> : moe_out_kernel<1>;
    static std::atomic<bool> done[15][64];
    if (!smem_opt_in(reinterpret_cast<const void*>(in), MOE_MAX_SMEM, done[5 * fine + fi]) ||
        !smem_opt_in(reinterpret_cast<const void*>(out), MOE_MAX_SMEM, done[10 + fo]))
        return GPTQ_ERR_CUDA;
    CUtensorMap ti, to;
    if (w4_tmap(&ti, qweight_in, n_experts * 2 * d_ff, d_model, 16) != GPTQ_OK ||
        w4_tmap(&to, qweight_out, n_experts * d_model, d_ff, 32) != GPTQ_OK)
        return GPTQ_ERR_CUDA;
    if (plan.smem_in > MOE_MAX_SMEM || plan.smem_out > MOE_MAX_SMEM) return GPTQ_ERR_SHAPE;
    in<<<ctas(pairs * (d_ff / (fine ? kMoeInRows<8> : kMoeInRows<4>))), W4_THREADS, plan.smem_in, st>>>(ti, p);
    // what follows reads what the kernel before it wrote: not launched without it
    if (launch_status() != GPTQ_OK ||
        launch_after(out, ctas(pairs * plan.slices * (d_model / MOE_OUT_ROWS)), W4_THREADS,
                     plan.smem_out, st, to, p) != cudaSuccess ||
        launch_after(moe_join_kernel, dim3((unsigned)ceil_div(d_model, 256), (unsigned)tokens), 256,
                     0, st, p) != cudaSuccess)
        return GPTQ_ERR_CUDA;
    count_launches(3);
    return launch_status();
}
