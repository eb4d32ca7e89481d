// Attention of the last tokens of each sequence over the paged 4-bit cache that
// gptq_kv4_append fills -- "大模型量化实战（上）" (the KV cache in INT4):
//
//   out = sum_j p_j V_j,  p = softmax_j(scale q . K_j),  K_j = s_j (c_j - z_j)
//
// One CTA per (query, head): its warps walk the keys, each with a running
// maximum and sum, and join at the end.
#include <cmath>

#include "common.cuh"
#include "tc_common.cuh"

namespace gptq {

struct KvAttn {
    const __half* q;
    int64_t tokens, seqs, pages, width, window, max_q, max_len;
    int hq, hkv, g, page_shift;
    const uint32_t* kc;
    const __half2* kp;
    const uint32_t* vc;
    const __half2* vp;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* start;
    float scale;                           // times log2(e)
    __half* out;
};

template <int E>
__global__ void __launch_bounds__(128) kv4_attention_simple_kernel(const KvAttn p)
{
    constexpr int D = 32 * E, NB = D / 32;
    __shared__ float part[4][D], ml[4][2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.z, h = blockIdx.y;
    const int64_t s0 = p.start[b], s1 = p.start[b + 1], L = p.lens[b];
    if (s0 < 0 || s1 < s0 || s1 > p.tokens || s1 - s0 > p.max_q || L < 0 || L > p.max_len) {
        if (threadIdx.x == 0) atomicCAS(&g_device_status, 0, kErrIndex);
        return;
    }
    const int64_t t = s0 + blockIdx.x;
    if (t >= s1) return;
    const int64_t hi = L - (s1 - s0) + int64_t(blockIdx.x) + 1;      // keys [lo, hi)
    const int64_t lo = p.window > 0 && hi - p.window > 0 ? hi - p.window : 0;
    const int hk = h / (p.hq / p.hkv);
    const __half* q = p.q + (t * p.hq + h) * D;
    float qv[E], acc[E];
    int kd[E], vd[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int n = lane * E + e;                        // nibble of the row
        const int w = n / 8, u = n / 4;
        kd[e] = 32 * (w % NB) + 8 * (w / NB) + n % 8;
        vd[e] = 32 * (u % NB) + 4 * (u / NB) + n % 4;
        qv[e] = __half2float(q[kd[e]]);
        acc[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int64_t j = lo + warp; j < hi; j += 4) {
        const int64_t page = p.table[int64_t(b) * p.width + (j >> p.page_shift)];
        if (page < 0 || page >= p.pages) {
            if (lane == 0) atomicCAS(&g_device_status, 0, kErrIndex);
            continue;
        }
        const int64_t row = ((page * p.hkv + hk) << p.page_shift) + (j & ((1 << p.page_shift) - 1));
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int n = lane * E + e;
            const float c = float((p.kc[row * (D / 8) + n / 8] >> (4 * (n % 8))) & 15u);
            const float2 sz = __half22float2(p.kp[row * (D / p.g) + kd[e] / p.g]);
            dot += qv[e] * (sz.x * (c - sz.y));
        }
        for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        dot *= p.scale;
        const float mx = fmaxf(m, dot), al = exp2f(m - mx), pr = exp2f(dot - mx);
        m = mx;
        l = l * al + pr;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int n = lane * E + e;
            const float c = float((p.vc[row * (D / 8) + n / 8] >> (4 * (n % 8))) & 15u);
            const float2 sz = __half22float2(p.vp[row * (D / p.g) + vd[e] / p.g]);
            acc[e] = acc[e] * al + pr * (sz.x * (c - sz.y));
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) part[warp][vd[e]] = acc[e];
    if (lane == 0) { ml[warp][0] = m; ml[warp][1] = l; }
    __syncthreads();
    float top = -INFINITY;
    for (int w = 0; w < 4; ++w) top = fmaxf(top, ml[w][0]);
    float wt[4], sum = 0.f;
    for (int w = 0; w < 4; ++w) {
        wt[w] = ml[w][0] == -INFINITY ? 0.f : exp2f(ml[w][0] - top);
        sum += wt[w] * ml[w][1];
    }
    for (int d = threadIdx.x; d < D; d += 128) {
        float o = 0.f;
        for (int w = 0; w < 4; ++w) o += wt[w] * part[w][d];
        p.out[(t * p.hq + h) * D + d] = __float2half_rn(sum > 0.f ? o / sum : 0.f);
    }
}

}  // namespace gptq

extern "C" size_t gptq_kv4_attention_workspace_bytes(int64_t seqs, int q_heads, int kv_heads,
                                                     int head_dim, int64_t max_q_len,
                                                     int64_t max_seq_len)
{
    if (seqs <= 0 || q_heads <= 0 || kv_heads <= 0 || head_dim <= 0 || max_q_len <= 0 ||
        max_seq_len <= 0)
        return 0;
    return 256;
}

extern "C" int gptq_kv4_attention(const uint16_t* q, int64_t tokens, int64_t seqs, int q_heads,
                                  int kv_heads, int head_dim, const uint32_t* k_codes,
                                  const uint16_t* k_params, const uint32_t* v_codes,
                                  const uint16_t* v_params, int64_t pages, int page_size,
                                  int group_size, const int32_t* block_table, int64_t table_width,
                                  const int32_t* seq_lens, const int32_t* q_start, float scale,
                                  int64_t window, int64_t max_q_len, int64_t max_seq_len,
                                  uint16_t* out, void* ws, size_t ws_bytes, void* stream)
{
    using namespace gptq;
    if (tokens < 0 || tokens > (int64_t(1) << 24) || seqs < 0 || seqs > 65535 || kv_heads < 1 ||
        kv_heads > 1024 || q_heads < 1 || q_heads > 1024 || q_heads % kv_heads != 0)
        return GPTQ_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return GPTQ_ERR_UNSUPPORTED;
    const int g = group_size == -1 ? head_dim : group_size;
    if ((g != 32 && g != 64 && g != 128 && g != 256) || head_dim % g != 0)
        return GPTQ_ERR_UNSUPPORTED;
    if (page_size < 16 || page_size > 4096 || (page_size & (page_size - 1)))
        return GPTQ_ERR_UNSUPPORTED;
    if (!std::isfinite(scale)) return GPTQ_ERR_INVALID_ARG;
    if (pages < 1 || pages > (int64_t(1) << 31) || table_width < 0 || window < 0 || max_q_len < 0 ||
        max_seq_len < 0 || max_seq_len > (int64_t(1) << 30) ||
        max_seq_len > table_width * int64_t(page_size))
        return GPTQ_ERR_SHAPE;
    if (seqs == 0 || tokens == 0 || max_q_len == 0) return GPTQ_OK;
    if (!q || !k_codes || !k_params || !v_codes || !v_params || !seq_lens || !q_start || !out ||
        !ws || (max_seq_len > 0 && !block_table))
        return GPTQ_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_codes) || !aligned16(k_params) || !aligned16(v_codes) ||
        !aligned16(v_params) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(q_start, 4) || !aligned16(out) || !aligned16(ws))
        return GPTQ_ERR_INVALID_ARG;
    if (ws_bytes < gptq_kv4_attention_workspace_bytes(seqs, q_heads, kv_heads, head_dim, max_q_len,
                                                      max_seq_len))
        return GPTQ_ERR_INVALID_ARG;
    KvAttn p{};
    p.q = reinterpret_cast<const __half*>(q);
    p.tokens = tokens; p.seqs = seqs; p.pages = pages; p.width = table_width;
    p.window = window; p.max_q = std::min(max_q_len, tokens); p.max_len = max_seq_len;
    p.hq = q_heads; p.hkv = kv_heads; p.g = g;
    while ((1 << p.page_shift) < page_size) ++p.page_shift;
    p.kc = k_codes; p.kp = reinterpret_cast<const __half2*>(k_params);
    p.vc = v_codes; p.vp = reinterpret_cast<const __half2*>(v_params);
    p.table = block_table; p.lens = seq_lens; p.start = q_start;
    p.scale = scale * 1.4426950408889634f;
    p.out = reinterpret_cast<__half*>(out);
    cudaStream_t st = as_stream(stream);
    KernelTimer kt(kKKvAttention, st);
    const dim3 grid((unsigned)p.max_q, (unsigned)q_heads, (unsigned)seqs);
    auto run = [&](auto kern) {
        kern<<<grid, 128, 0, st>>>(p);
        count_launches();
        return launch_status();
    };
    switch (head_dim) {
        case 64: return run(kv4_attention_simple_kernel<2>);
        case 128: return run(kv4_attention_simple_kernel<4>);
        default: return run(kv4_attention_simple_kernel<8>);
    }
}
