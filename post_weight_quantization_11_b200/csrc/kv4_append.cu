// Appending to a paged 4-bit key / value cache -- "大模型量化实战（上）" (the
// KV cache in INT4), with the group quantizer of the round-to-nearest baseline
// ("校准艺术" sec. 2.1) on rows that arrive token by token, and the rotary
// position rotation on the way:
//
//   (a, b) -> (a c - b s, b c + a s)        pairs of the first rot_dim elements
//   mn = min(0, min x), mx = max(0, max x)  over a group of group_size elements
//   s = fp16((mx - mn) fp32(1 / 15)), z = clamp(rne(-mn / s)), c = clamp(rne(x / s) + z)
//
// A row (a token's head of q, k or v) is head_dim / 8 lanes of eight consecutive
// elements: a warp has 256 / head_dim rows at a time and a few rows of one token in
// turn, whose position, cosines, sines and slot are read once; the next rows are
// loaded while some are worked on.  A rotation partner is in the same lane
// (interleaved) or rot_dim / 16 lanes away, a group is group_size / 8 lanes, and a
// cache word is a lane's: shuffles, no shared memory.  Every operation is an IEEE
// fp32 one with its own rounding (no contraction), so the codes are a function of
// the inputs alone.
// Measured (B200, 32 + 2 x 8 heads of 128, fp16, groups of 32): 26 us for 4001 tokens
// (104 MB: 4.0 TB/s, 0.61 of the measured copy rate; bound by 200 instructions a round
// of two rows, issued in 75 % of the slots, with rows loaded one round ahead; six CTAs an SM: 32,
// eight: 28, ten: 26; rows two rounds ahead, with the registers that takes: 36), 2.3 us
// for 16.
#include "common.cuh"
#include "quant_common.cuh"
#include "tc_common.cuh"

namespace gptq {

constexpr int KVA_THREADS = 128, KVA_CTAS = 9;   // a CTA's threads, CTAs an SM (56 registers)

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
    int rot, inter;
    int lanes_shift, groups_shift;         // log2 of a group's lanes, of a row's groups
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

// Eight elements as loaded
template <typename T> struct Raw8;
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p)
    {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};
template <> struct Raw8<__half> {
    uint4 a;
    __device__ __forceinline__ void load(const __half* p) { a = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        const __half2* h = reinterpret_cast<const __half2*>(&a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(h[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
};

__device__ __forceinline__ void store8(__half* p, const float (&x)[8])
{
    uint4 v;
    __half2* h = reinterpret_cast<__half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = v;
}

// group_params for 4 bits without its divisions.  The scale is the range times the
// rounded 1 / 15, as a division of fp32 tensors by 15 computes it on the GPU, so that a
// program's own fp32 quantizer gives the same bytes; it differs by one unit of the fp16
// scale from the quotient's in about 3 of 100 000 groups.  A range over 2^20 gives the
// largest scale either way.  The zero point's quotient is rounded correctly by
// div_rn_recip where it decides anything.
__device__ __forceinline__ GroupQ group_params4(float mn, float mx)
{
    constexpr float K15 = 0x1.111112p-4f;                  // RN(1 / 15)
    if (mn == mx) { mn = -1.f; mx = 1.f; }                 // all-zero group
    const float s_pre = __fmul_rn(fminf(__fsub_rn(mx, mn), 1048576.f), K15);
    unsigned short hb = __half_as_ushort(__float2half_rn(s_pre));
    hb = hb == 0 ? (unsigned short)0x0001u : hb >= 0x7c00u ? (unsigned short)0x7bffu : hb;
    GroupQ g;
    g.h = __ushort_as_half(hb);
    g.s = __half2float(g.h);
    g.r = __frcp_rn(g.s);
    g.z = fminf(fmaxf(rne_for_clamp(div_rn_recip(-mn, g.s, g.r)), 0.f), 15.f);
    return g;
}

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(KVA_THREADS, KVA_CTAS) kv4_append_kernel(const KvAppend p)
{
    constexpr int NB = D / 32, LANES = D / 8, AT_ONCE = 32 / LANES;
    constexpr uint32_t ALL = 0xffffffffu;
    const int lane = threadIdx.x & 31, l = lane % LANES;
    const int64_t t = blockIdx.x;
    const int rows = p.hq + 2 * p.hkv;
    const int step = (KVA_THREADS / 32) * AT_ONCE * gridDim.y;
    int first = (blockIdx.y * (KVA_THREADS / 32) + (threadIdx.x >> 5)) * AT_ONCE;   // of the warp's rows
    if (first >= rows) return;                             // whole warps
    const int64_t slot = p.slots[t];
    const int32_t pos = p.rot ? p.pos[t] : 0;
    const T* q = static_cast<const T*>(p.q) + t * p.qs + l * 8;
    const T* k = static_cast<const T*>(p.k) + t * p.ks + l * 8;
    const T* v = static_cast<const T*>(p.v) + t * p.vs + l * 8;
    const int sub = lane / LANES;
    auto row = [&](int i) {                                // (a row behind the last: the last)
        i = min(i, rows - 1);
        return i < p.hq ? q + i * D : i < p.hq + p.hkv ? k + (i - p.hq) * D : v + (i - p.hq - p.hkv) * D;
    };
    Raw8<T> next;
    next.load(row(first + sub));
    if ((slot >> p.page_shift) >= p.pages || pos < 0 || (p.rot && pos >= p.n_pos)) {
        if (lane == 0) atomicCAS(&g_device_status, 0, kErrIndex);   // nothing of the token is written
        return;
    }
    // the lane's cosines and sines, and the partner's lane
    const int sh = p.rot / 16;                             // lanes between partners
    const bool in = l * 8 < p.rot, low = l < sh;
    const int mate = in ? (low ? lane + sh : lane - sh) : lane;
    float c[INTER ? 4 : 8], s[INTER ? 4 : 8];
    if (in) {
        const float* tab = p.table + int64_t(pos) * p.rot + (INTER ? l * 4 : (low ? l : l - sh) * 8);
        const float* tas = tab + p.rot / 2;
#pragma unroll
        for (int i = 0; i < (INTER ? 4 : 8); i += 4) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(tab + i));
            const float4 b = __ldg(reinterpret_cast<const float4*>(tas + i));
            c[i] = a.x; c[i + 1] = a.y; c[i + 2] = a.z; c[i + 3] = a.w;
            s[i] = b.x; s[i + 1] = b.y; s[i + 2] = b.z; s[i + 3] = b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < (INTER ? 4 : 8); ++i) { c[i] = 1.f; s[i] = 0.f; }
    }
    const int64_t page = slot >> p.page_shift, at = slot & ((1 << p.page_shift) - 1);
    for (;;) {
        float x[8];
        next.get(x);
        const int now = first + sub;
        const bool live = now < rows, is_q = now < p.hq, is_v = now >= p.hq + p.hkv;
        first += step;
        if (first < rows) next.load(row(first + sub));
        if (p.rot && first - step < p.hq + p.hkv) {        // (some row of the warp is not v)
            const bool turn = in && !is_v;
            if constexpr (INTER) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float a = x[i], b = x[i + 1];
                    const float u = __fsub_rn(__fmul_rn(a, c[i / 2]), __fmul_rn(b, s[i / 2]));
                    const float w = __fadd_rn(__fmul_rn(b, c[i / 2]), __fmul_rn(a, s[i / 2]));
                    x[i] = turn ? u : a;
                    x[i + 1] = turn ? w : b;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float o = __shfl_sync(ALL, x[i], mate);
                    const float u = __fmul_rn(x[i], c[i]), w = __fmul_rn(o, s[i]);
                    const float y = low ? __fsub_rn(u, w) : __fadd_rn(u, w);
                    x[i] = turn ? y : x[i];
                }
            }
        }
        if (is_q) store8(p.q_out + (t * p.hq + now) * D + l * 8, x);
        if (first - step + AT_ONCE > p.hq) {               // some row of the warp is k or v
            const int h = now - p.hq - (is_v ? p.hkv : 0);
            constexpr float BIG = 3.402823466e38f;
            float mn = 0.f, mx = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = fminf(fmaxf(x[i], -BIG), BIG);      // NaN -> -BIG
                mn = fminf(mn, x[i]);
                mx = fmaxf(mx, x[i]);
            }
            const int lpg = 1 << p.lanes_shift;            // lanes per group
            for (int o = 1; o < lpg; o <<= 1) {
                mn = fminf(mn, __shfl_xor_sync(ALL, mn, o));
                mx = fmaxf(mx, __shfl_xor_sync(ALL, mx, o));
            }
            if (live && !is_q) {
                const GroupQ gq = group_params4(mn, mx);
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float code = quant_code_fast(x[i], gq, 15.f);
                    w |= code_byte(code) << (4 * i);
                    x[i] = __fmul_rn(__fsub_rn(code, gq.z), gq.s);
                }
                __half* values = is_v ? p.v_val : p.k_val;
                if (values) store8(values + (t * p.hkv + h) * D + l * 8, x);
                if (slot >= 0) {                           // < 0: padding, the cache is left alone
                    const int64_t rowi = ((page * p.hkv + h) << p.page_shift) + at;
                    if ((l & (lpg - 1)) == 0)
                        (is_v ? p.vp : p.kp)[(rowi << p.groups_shift) + (l >> p.lanes_shift)] =
                            __halves2half2(gq.h, __float2half_rn(gq.z));
                    const int i = l >> 2, u = l & 3;       // block of 32 elements, eighth of it
                    if (is_v) {                            // half words: elements 32 i + 4 h' ..
                        uint16_t* out = reinterpret_cast<uint16_t*>(p.vc + rowi * (D / 8));
                        out[(2 * u) * NB + i] = uint16_t(w);
                        out[(2 * u + 1) * NB + i] = uint16_t(w >> 16);
                    } else {                               // words: elements 32 i + 8 t' ..
                        p.kc[rowi * (D / 8) + u * NB + i] = w;
                    }
                }
            }
        }
        if (first >= rows) return;
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
    p.rot = rot_dim; p.inter = interleaved != 0;
    while ((8 << p.lanes_shift) < g) ++p.lanes_shift;
    while ((g << p.groups_shift) < head_dim) ++p.groups_shift;
    p.pages = pages;
    while ((1 << p.page_shift) < page_size) ++p.page_shift;
    p.kc = k_codes; p.kp = reinterpret_cast<__half2*>(k_params);
    p.vc = v_codes; p.vp = reinterpret_cast<__half2*>(v_params);
    p.q_out = reinterpret_cast<__half*>(q_out);
    p.k_val = reinterpret_cast<__half*>(k_values);
    p.v_val = reinterpret_cast<__half*>(v_values);
    // CTAs per token: all rows at once while there are few tokens, six rounds a warp beyond
    const int rows = p.hq + 2 * p.hkv, at_once = KVA_THREADS / 32 * (256 / head_dim);
    const int64_t all = ceil_div(rows, at_once);
    const int64_t split = std::max<int64_t>(
        std::min<int64_t>(all, ceil_div(int64_t(device_sm_count()) * 8, tokens)), ceil_div(all, 6));
    cudaStream_t st = as_stream(stream);
    KernelTimer kt(kKKvAppend, st);
    auto run = [&](auto inter, auto plain) {
        const dim3 grid((unsigned)tokens, (unsigned)split);
        if (p.inter) inter<<<grid, KVA_THREADS, 0, st>>>(p);
        else plain<<<grid, KVA_THREADS, 0, st>>>(p);
        count_launches();
        return launch_status();
    };
    const bool f32 = dtype == GPTQ_DTYPE_F32;
#define KVA_RUN(D)                                                                        \
    return f32 ? run(kv4_append_kernel<float, D, true>, kv4_append_kernel<float, D, false>)   \
               : run(kv4_append_kernel<__half, D, true>, kv4_append_kernel<__half, D, false>);
    switch (head_dim) {
        case 64: KVA_RUN(64)
        case 128: KVA_RUN(128)
        default: KVA_RUN(256)
    }
#undef KVA_RUN
}
