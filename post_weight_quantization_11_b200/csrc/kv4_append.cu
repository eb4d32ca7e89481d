// Appending to a paged 4-bit key / value cache -- "大模型量化实战（上）" (the
// KV cache in INT4), with the group quantizer of the round-to-nearest baseline
// ("校准艺术" sec. 2.1) on rows that arrive token by token, and the rotary
// position rotation on the way:
//
//   (a, b) -> (a c - b s, b c + a s)        pairs of the first rot_dim elements
//   mn = min(0, min x), mx = max(0, max x)  over a group of group_size elements
//   s = fp16((mx - mn) / 15), z = clamp(rne(-mn / s)), c = clamp(rne(x / s) + z)
//
// One warp per row (a token's head of q, k or v): lane l holds the E =
// head_dim / 32 consecutive elements from E l on.  A rotation partner is in the
// same lane (interleaved) or rot_dim / 2 / E lanes away, a group is group_size
// / E lanes, and a cache word is 8 / E lanes: shuffles, no shared memory.  Every
// operation is an IEEE fp32 one with its own rounding (no contraction), so the
// codes are a function of the inputs alone.
#include "common.cuh"
#include "quant_common.cuh"
#include "tc_common.cuh"

namespace gptq {

struct KvAppend {
    const void* q;
    const void* k;
    const void* v;
    int64_t qs, ks, vs;                    // elements between tokens
    int64_t tokens;
    int hq, hkv;
    const int32_t* pos;
    const int64_t* slots;
    const float* table;
    int64_t n_pos;
    int rot, inter, g;
    int64_t pages;
    int page_shift;
    uint32_t* kc;
    __half2* kp;
    uint32_t* vc;
    __half2* vp;
    __half* q_out;
    __half* k_val;
    __half* v_val;
};

template <int N> struct alignas(N) Bytes { uint8_t b[N]; };

// E consecutive elements as fp32
template <int E> __device__ __forceinline__ void load_row(const float* p, float (&x)[E])
{
    using V = Bytes<(E * 4 < 16 ? E * 4 : 16)>;
    constexpr int PER = sizeof(V) / 4;
#pragma unroll
    for (int i = 0; i < E / PER; ++i)
        *reinterpret_cast<V*>(&x[i * PER]) = reinterpret_cast<const V*>(p)[i];
}

template <int E> __device__ __forceinline__ void load_row(const __half* p, float (&x)[E])
{
    alignas(16) __half h[E];
    *reinterpret_cast<Bytes<E * 2>*>(h) = *reinterpret_cast<const Bytes<E * 2>*>(p);
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = __half2float(h[i]);
}

template <int E> __device__ __forceinline__ void store_halves(__half* p, const float (&x)[E])
{
    alignas(16) __half h[E];
#pragma unroll
    for (int i = 0; i < E; ++i) h[i] = __float2half_rn(x[i]);
    *reinterpret_cast<Bytes<E * 2>*>(p) = *reinterpret_cast<const Bytes<E * 2>*>(h);
}

template <typename T, int E>
__global__ void __launch_bounds__(256) kv4_append_kernel(const KvAppend p)
{
    constexpr int D = 32 * E, NB = D / 32;
    constexpr uint32_t ALL = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    const int rows = p.hq + 2 * p.hkv;
    const int64_t item = int64_t(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5);
    const int64_t t = item / rows;
    if (t >= p.tokens) return;                             // whole warps
    const int r = int(item - t * rows);
    const int64_t slot = p.slots[t];
    const int32_t pos = p.rot ? p.pos[t] : 0;
    if ((slot >> p.page_shift) >= p.pages || pos < 0 || (p.rot && pos >= p.n_pos)) {
        if (lane == 0) atomicCAS(&g_device_status, 0, kErrIndex);   // nothing of the token is written
        return;
    }
    const bool is_q = r < p.hq, is_v = r >= p.hq + p.hkv;
    const int h = is_q ? r : (is_v ? r - p.hq - p.hkv : r - p.hq);
    const T* src = is_q ? static_cast<const T*>(p.q) + t * p.qs
                        : (is_v ? static_cast<const T*>(p.v) + t * p.vs
                                : static_cast<const T*>(p.k) + t * p.ks);
    float x[E];
    load_row<E>(src + int64_t(h) * D + lane * E, x);
    if (!is_v && p.rot) {
        const int half = p.rot / 2, sh = half / E;         // lanes between partners
        const float* row = p.table + int64_t(pos) * p.rot;
        const bool in = lane * E < p.rot;
        if (p.inter) {
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const int j = (lane * E + i) / 2;
                const float c = in ? row[j] : 1.f, s = in ? row[half + j] : 0.f;
                const float a = x[i], b = x[i + 1];
                if (in) {
                    x[i] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
                    x[i + 1] = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
                }
            }
        } else {
            const bool first = lane < sh;
            const int mate = in ? (first ? lane + sh : lane - sh) : lane;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float o = __shfl_sync(ALL, x[i], mate);
                const int j = (first ? lane : lane - sh) * E + i;
                const float c = in ? row[j] : 1.f, s = in ? row[half + j] : 0.f;
                if (in)
                    x[i] = first ? __fsub_rn(__fmul_rn(x[i], c), __fmul_rn(o, s))
                                 : __fadd_rn(__fmul_rn(x[i], c), __fmul_rn(o, s));
            }
        }
    }
    if (is_q) {
        store_halves<E>(p.q_out + (t * p.hq + h) * D + lane * E, x);
        return;
    }
    constexpr float BIG = 3.402823466e38f;
    float mn = 0.f, mx = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        x[i] = fminf(fmaxf(x[i], -BIG), BIG);              // NaN -> -BIG
        mn = fminf(mn, x[i]);
        mx = fmaxf(mx, x[i]);
    }
    const int lpg = p.g / E;                               // lanes per group (a power of two)
    for (int o = 1; o < lpg; o <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(ALL, mn, o));
        mx = fmaxf(mx, __shfl_xor_sync(ALL, mx, o));
    }
    const GroupQ gq = group_params(mn, mx, 15.f);
    uint32_t w = 0;
    float val[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float c = quant_code_fast(x[i], gq, 15.f);
        w |= code_byte(c) << (4 * i);
        val[i] = __fmul_rn(__fsub_rn(c, gq.z), gq.s);
    }
    __half* values = is_v ? p.v_val : p.k_val;
    if (values) store_halves<E>(values + (t * p.hkv + h) * D + lane * E, val);
    if (slot < 0) return;                                  // padding: the cache is left alone
    const int64_t page = slot >> p.page_shift, at = slot & ((1 << p.page_shift) - 1);
    const int64_t rowi = (((page * p.hkv + h) << p.page_shift) + at);
    if (lane % lpg == 0)
        (is_v ? p.vp : p.kp)[rowi * (D / p.g) + lane / lpg] =
            __halves2half2(gq.h, __float2half_rn(gq.z));
    if (is_v) {                                            // half words: elements 32 i + 4 h' ..
        uint16_t* out = reinterpret_cast<uint16_t*>(p.vc + rowi * (D / 8));
        if constexpr (E == 2) {
            w |= __shfl_xor_sync(ALL, w, 1) << 8;
            if (!(lane & 1)) out[((lane >> 1) & 7) * NB + (lane >> 4)] = uint16_t(w);
        } else if constexpr (E == 4) {
            out[(lane & 7) * NB + (lane >> 3)] = uint16_t(w);
        } else {
            out[(2 * (lane & 3)) * NB + (lane >> 2)] = uint16_t(w);
            out[(2 * (lane & 3) + 1) * NB + (lane >> 2)] = uint16_t(w >> 16);
        }
    } else {                                               // words: elements 32 i + 8 t' ..
        uint32_t* out = p.kc + rowi * (D / 8);
        if constexpr (E == 2) w |= __shfl_xor_sync(ALL, w, 1) << 8;
        if constexpr (E == 2) w |= __shfl_xor_sync(ALL, w, 2) << 16;
        if constexpr (E == 4) w |= __shfl_xor_sync(ALL, w, 1) << 16;
        if (lane % (8 / E) == 0) {
            const int word = lane * E / 8;                 // of the row, in element order
            out[(word & 3) * NB + (word >> 2)] = w;
        }
    }
}

}  // namespace gptq

extern "C" int gptq_kv4_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                               const void* v, int64_t v_stride, int dtype, int64_t tokens,
                               int q_heads, int kv_heads, int head_dim, const int32_t* positions,
                               const int64_t* slots, const float* cos_sin, int64_t n_positions,
                               int rot_dim, int interleaved, int group_size, int64_t pages,
                               int page_size, uint32_t* k_codes, uint16_t* k_params,
                               uint32_t* v_codes, uint16_t* v_params, uint16_t* q_out,
                               uint16_t* k_values, uint16_t* v_values, void* stream)
{
    using namespace gptq;
    if (dtype != GPTQ_DTYPE_F32 && dtype != GPTQ_DTYPE_F16) return GPTQ_ERR_INVALID_ARG;
    if (tokens < 0 || tokens > (int64_t(1) << 24) || kv_heads < 1 || kv_heads > 1024 ||
        (q && (q_heads < 1 || q_heads > 1024)))
        return GPTQ_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return GPTQ_ERR_UNSUPPORTED;
    const int g = group_size == -1 ? head_dim : group_size;
    if ((g != 32 && g != 64 && g != 128 && g != 256) || head_dim % g != 0)
        return GPTQ_ERR_UNSUPPORTED;
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0) return GPTQ_ERR_UNSUPPORTED;
    if (page_size < 16 || page_size > 4096 || (page_size & (page_size - 1)))
        return GPTQ_ERR_UNSUPPORTED;
    if (pages < 1 || pages > (int64_t(1) << 31) || (rot_dim > 0 && n_positions < 1))
        return GPTQ_ERR_SHAPE;
    if (tokens == 0) return GPTQ_OK;
    if (!k || !v || !slots || !k_codes || !k_params || !v_codes || !v_params)
        return GPTQ_ERR_INVALID_ARG;
    if ((q == nullptr) != (q_out == nullptr) || (k_values == nullptr) != (v_values == nullptr))
        return GPTQ_ERR_INVALID_ARG;
    if (rot_dim > 0 && (!cos_sin || !positions)) return GPTQ_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(k_codes) ||
        !aligned16(k_params) || !aligned16(v_codes) || !aligned16(v_params) ||
        !aligned16(cos_sin) || !aligned(positions, 4) || !aligned(slots, 8) || !aligned16(q_out) ||
        !aligned16(k_values) || !aligned16(v_values))
        return GPTQ_ERR_INVALID_ARG;
    const int64_t unit = dtype == GPTQ_DTYPE_F32 ? 4 : 8;  // elements in 16 bytes
    if (k_stride < int64_t(kv_heads) * head_dim || v_stride < int64_t(kv_heads) * head_dim ||
        (q && q_stride < int64_t(q_heads) * head_dim) || k_stride % unit || v_stride % unit ||
        (q && q_stride % unit))
        return GPTQ_ERR_INVALID_ARG;
    KvAppend p{};
    p.q = q; p.k = k; p.v = v;
    p.qs = q_stride; p.ks = k_stride; p.vs = v_stride;
    p.tokens = tokens;
    p.hq = q ? q_heads : 0;
    p.hkv = kv_heads;
    p.pos = positions; p.slots = slots;
    p.table = cos_sin; p.n_pos = n_positions;
    p.rot = rot_dim; p.inter = interleaved != 0; p.g = g;
    p.pages = pages;
    while ((1 << p.page_shift) < page_size) ++p.page_shift;
    p.kc = k_codes; p.kp = reinterpret_cast<__half2*>(k_params);
    p.vc = v_codes; p.vp = reinterpret_cast<__half2*>(v_params);
    p.q_out = reinterpret_cast<__half*>(q_out);
    p.k_val = reinterpret_cast<__half*>(k_values);
    p.v_val = reinterpret_cast<__half*>(v_values);
    const int64_t items = tokens * (p.hq + 2 * p.hkv), blocks = ceil_div(items, 8);
    if (blocks > 0x7fffffff) return GPTQ_ERR_SHAPE;
    cudaStream_t st = as_stream(stream);
    KernelTimer kt(kKKvAppend, st);
    auto run = [&](auto kern) {
        kern<<<(unsigned)blocks, 256, 0, st>>>(p);
        count_launches();
        return launch_status();
    };
    const bool f32 = dtype == GPTQ_DTYPE_F32;
    switch (head_dim) {
        case 64: return f32 ? run(kv4_append_kernel<float, 2>) : run(kv4_append_kernel<__half, 2>);
        case 128: return f32 ? run(kv4_append_kernel<float, 4>) : run(kv4_append_kernel<__half, 4>);
        default: return f32 ? run(kv4_append_kernel<float, 8>) : run(kv4_append_kernel<__half, 8>);
    }
}
