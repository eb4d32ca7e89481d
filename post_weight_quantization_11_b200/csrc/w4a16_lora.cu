// W4A16 product with low-rank adapters of many requests -- the packed product
// of "INT4/INT8 量化推理" sec. 六 plus each row's adapter:
//
//   y[b] = x[b] Q^T + scaling[a] (x[b] A_a^T) B_a^T,   a = adapter[b]
//
// Two kernels: t[b] = scaling[a] A_a x[b] (one warp per row and rank), then one
// warp per output.
#include "common.cuh"
#include "tc_common.cuh"

namespace gptq {

struct LoraParams {
    const __half* x;
    const uint32_t* qweight;
    const __half* scales;
    const uint8_t* qzeros;
    const int32_t* perm;
    const __half* a;
    const __half* b;
    const float* scaling;
    const int32_t* adapter;
    int64_t batch, m, d, g, n;
    int rank;
    float* t;
    float* y;
};

__global__ void __launch_bounds__(256) lora_shrink_simple_kernel(const LoraParams p)
{
    const int lane = threadIdx.x & 31;
    const int64_t item = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t b = item / p.rank, r = item - b * p.rank;
    if (b >= p.batch) return;
    int64_t a = p.adapter[b];
    if (a < -1 || a >= p.n) {
        if (lane == 0) atomicCAS(&g_device_status, 0, kErrIndex);
        a = -1;
    }
    float s = 0.f;
    if (a >= 0)
        for (int64_t j = lane; j < p.d; j += 32)
            s += __half2float(p.x[b * p.d + j]) * __half2float(p.a[(a * p.rank + r) * p.d + j]);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) p.t[b * p.rank + r] = a >= 0 ? s * p.scaling[a] : 0.f;
}

__global__ void __launch_bounds__(256) lora_product_simple_kernel(const LoraParams p)
{
    const int lane = threadIdx.x & 31;
    const int64_t r = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5), b = blockIdx.y;
    if (r >= p.m) return;
    const int64_t G = p.d / p.g;
    float s = 0.f;
    for (int64_t k = lane; k < p.d; k += 32) {
        const int64_t src = p.perm ? p.perm[k] : k;
        if (src < 0 || src >= p.d) {
            atomicCAS(&g_device_status, 0, kErrIndex);
            continue;
        }
        const int64_t gi = k / p.g;
        const int c = (p.qweight[r * (p.d / 8) + k / 8] >> (4 * (k % 8))) & 15;
        const int z = (p.qzeros[r * ((G + 1) / 2) + gi / 2] >> (4 * (gi & 1))) & 15;
        s += __half2float(p.x[b * p.d + src]) * (__half2float(p.scales[r * G + gi]) * float(c - z));
    }
    const int64_t a = p.adapter[b];
    if (a >= 0 && a < p.n)
        for (int k = lane; k < p.rank; k += 32)
            s += p.t[b * p.rank + k] * __half2float(p.b[(a * p.m + r) * p.rank + k]);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) p.y[b * p.m + r] = s;
}

}  // namespace gptq

extern "C" size_t gptq_w4a16_lora_workspace_bytes(int64_t batch, int64_t d_out, int64_t d_in,
                                                  int rank)
{
    if (batch <= 0 || d_out <= 0 || d_in <= 0 || rank <= 0) return 0;
    return gptq::align_up(size_t(batch) * size_t(rank) * 4, 256);
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
    if (rank < 8 || rank > 256 || rank % 8 != 0) return GPTQ_ERR_UNSUPPORTED;
    if (batch == 0) return GPTQ_OK;
    if (!x || !qweight || !scales || !qzeros || !y || !ws || !adapter ||
        (n_adapters > 0 && (!lora_a || !lora_b || !lora_scaling)))
        return GPTQ_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(qweight) || !aligned16(scales) || !aligned16(qzeros) ||
        !aligned16(y) || !aligned16(ws) || !aligned16(perm) || !aligned16(lora_a) ||
        !aligned16(lora_b) || !aligned(lora_scaling, 4) || !aligned(adapter, 4))
        return GPTQ_ERR_INVALID_ARG;
    if (ws_bytes < gptq_w4a16_lora_workspace_bytes(batch, d_out, d_in, rank))
        return GPTQ_ERR_INVALID_ARG;
    LoraParams p{};
    p.x = reinterpret_cast<const __half*>(x);
    p.qweight = qweight;
    p.scales = reinterpret_cast<const __half*>(scales);
    p.qzeros = qzeros; p.perm = perm;
    p.a = reinterpret_cast<const __half*>(lora_a);
    p.b = reinterpret_cast<const __half*>(lora_b);
    p.scaling = lora_scaling; p.adapter = adapter;
    p.batch = batch; p.m = d_out; p.d = d_in; p.g = g; p.n = n_adapters; p.rank = rank;
    p.t = static_cast<float*>(ws);
    p.y = y;
    cudaStream_t st = as_stream(stream);
    KernelTimer kt(kKLora, st);
    lora_shrink_simple_kernel<<<(unsigned)ceil_div(batch * rank, 8), 256, 0, st>>>(p);
    lora_product_simple_kernel<<<dim3((unsigned)ceil_div(d_out, 8), (unsigned)batch), 256, 0, st>>>(p);
    count_launches(2);
    return launch_status();
}
