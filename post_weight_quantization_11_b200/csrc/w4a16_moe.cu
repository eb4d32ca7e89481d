// A whole mixture-of-experts layer of packed experts for a few tokens -- top-k
// routed experts ("INT4/INT8 量化推理" sec. 五) with weights in 4 bits and fp16
// activations (sec. 六 of the same page):
//
//   p = softmax(logits), S = top_k of it,  y = sum_S w_e D_e (silu(G_e x) * U_e x)
//
// Three kernels: the routes, h (one warp per row of an expert and token), y.
#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "tc_common.cuh"

namespace gptq {

constexpr int kMoeTokens = 64, kMoeExperts = 256, kMoeTopK = 8;

struct MoeParams {
    const __half* x;
    const float* logits;
    const uint32_t* qwi;
    const __half* sci;
    const uint8_t* qzi;
    const int32_t* pi;
    const uint32_t* qwo;
    const __half* sco;
    const uint8_t* qzo;
    const int32_t* po;
    int64_t d, f, gi, go;
    int T, E, k, renorm;
    int* ids;          // T x k, -1: none
    float* w;          // T x k
    float* h;          // T k x f
    float* y;
};

// One warp: the routes of token t into ids / w[0 .. k)
__device__ __forceinline__ void moe_route(const float* logits, int E, int k, int renorm, int* ids,
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

__global__ void __launch_bounds__(256) moe_route_kernel(const MoeParams p)
{
    for (int t = threadIdx.x >> 5; t < p.T; t += 8)
        moe_route(p.logits + int64_t(t) * p.E, p.E, p.k, p.renorm, p.ids + t * p.k, p.w + t * p.k);
}

// One warp: the product of row r of a packed layer with x (through perm)
template <typename T>
__device__ __forceinline__ float row_dot(const uint32_t* qw, const __half* sc, const uint8_t* qz,
                                         const int32_t* perm, int64_t r, int64_t d, int64_t g,
                                         const T* x)
{
    const int lane = threadIdx.x & 31;
    const int64_t G = d / g;
    float s = 0.f;
    for (int64_t k = lane; k < d; k += 32) {
        const int64_t src = perm ? perm[k] : k;
        if (src < 0 || src >= d) {
            atomicCAS(&g_device_status, 0, kErrIndex);
            continue;
        }
        const int64_t gi = k / g;
        const int c = (qw[r * (d / 8) + k / 8] >> (4 * (k % 8))) & 15;
        const int z = (qz[r * ((G + 1) / 2) + gi / 2] >> (4 * (gi & 1))) & 15;
        s += float(x[src]) * (__half2float(sc[r * G + gi]) * float(c - z));
    }
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

__global__ void __launch_bounds__(256) moe_in_simple_kernel(const MoeParams p)
{
    const int64_t r = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int pair = blockIdx.y, e = p.ids[pair];
    if (e < 0 || r >= p.f) return;
    const int64_t m = 2 * p.f, G = p.d / p.gi;
    const __half* x = p.x + int64_t(pair / p.k) * p.d;
    const int32_t* perm = p.pi ? p.pi + e * p.d : nullptr;
    const uint32_t* qw = p.qwi + e * m * (p.d / 8);
    const __half* sc = p.sci + e * m * G;
    const uint8_t* qz = p.qzi + e * m * ((G + 1) / 2);
    const float gate = row_dot(qw, sc, qz, perm, r, p.d, p.gi, x);
    const float up = row_dot(qw, sc, qz, perm, r + p.f, p.d, p.gi, x);
    if ((threadIdx.x & 31) == 0) p.h[pair * p.f + r] = gate / (1.f + expf(-gate)) * up;
}

__global__ void __launch_bounds__(256) moe_out_simple_kernel(const MoeParams p)
{
    const int64_t r = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int t = blockIdx.y;
    if (r >= p.d) return;
    const int64_t G = p.f / p.go;
    float s = 0.f;
    for (int j = 0; j < p.k; ++j) {
        const int pair = t * p.k + j, e = p.ids[pair];
        if (e < 0) continue;
        s += p.w[pair] * row_dot(p.qwo + e * p.d * (p.f / 8), p.sco + e * p.d * G,
                                 p.qzo + e * p.d * ((G + 1) / 2), p.po ? p.po + e * p.f : nullptr, r,
                                 p.f, p.go, p.h + pair * p.f);
    }
    if ((threadIdx.x & 31) == 0) p.y[t * p.d + r] = s;
}

}  // namespace gptq

extern "C" size_t gptq_w4a16_moe_workspace_bytes(int64_t tokens, int64_t n_experts, int top_k,
                                                 int64_t d_model, int64_t d_ff)
{
    if (tokens <= 0 || n_experts <= 0 || top_k <= 0 || d_model <= 0 || d_ff <= 0) return 0;
    const size_t pairs = size_t(tokens) * size_t(top_k);
    return gptq::align_up(pairs * 8, 256) + gptq::align_up(pairs * size_t(d_ff) * 4, 256);
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
    if (d_model < 128 || d_model > kMaxDim || d_model % 128 != 0 || d_ff < 128 || d_ff > kMaxDim ||
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
    const int64_t pairs = tokens * top_k;
    MoeParams p{};
    p.x = reinterpret_cast<const __half*>(x);
    p.logits = logits;
    p.qwi = qweight_in; p.sci = reinterpret_cast<const __half*>(scales_in); p.qzi = qzeros_in;
    p.pi = perm_in;
    p.qwo = qweight_out; p.sco = reinterpret_cast<const __half*>(scales_out); p.qzo = qzeros_out;
    p.po = perm_out;
    p.d = d_model; p.f = d_ff; p.gi = gi; p.go = go;
    p.T = (int)tokens; p.E = (int)n_experts; p.k = top_k; p.renorm = renormalize != 0;
    uint8_t* w = static_cast<uint8_t*>(ws);
    p.ids = reinterpret_cast<int*>(w);
    p.w = reinterpret_cast<float*>(w + pairs * 4);
    p.h = reinterpret_cast<float*>(w + align_up(size_t(pairs) * 8, 256));
    p.y = y;
    cudaStream_t st = as_stream(stream);
    KernelTimer kt(kKMoe, st);
    moe_route_kernel<<<1, 256, 0, st>>>(p);
    moe_in_simple_kernel<<<dim3((unsigned)ceil_div(d_ff, 8), (unsigned)pairs), 256, 0, st>>>(p);
    moe_out_simple_kernel<<<dim3((unsigned)ceil_div(d_model, 8), (unsigned)tokens), 256, 0, st>>>(p);
    count_launches(3);
    return launch_status();
}
