// Attention of the last tokens of each sequence over the paged 4-bit cache that
// gptq_kv4_append fills -- "大模型量化实战（上）" (the KV cache in INT4):
//
//   out = sum_j p_j V_j,  p = softmax_j(scale q . K_j),  K_j = s_j (c_j - z_j)
//
// The rows (query, head) of a sequence that share a key head are the columns of the
// products, eight to a CTA; keys and values are their row operands, read once.
//  * Work: (chunk of keys, key head and row tile, sequence).  Chunks have one size,
//    so ragged batches balance; CTAs whose chunk lies behind a sequence's end leave
//    at once.  The four warps of a CTA take tiles of 32 keys in turn, each with its
//    own running maximum, sum and output, joined at the end.  Up to eight chunks that
//    fit the GPU at once are a cluster, whose CTAs join them out of each other's
//    shared memory; otherwise a second kernel joins them, in a fixed order.
//  * A tile is contiguous in a page of 32 keys or more, its halves in one of 16: four or
//    eight bulk copies (codes and parameters of keys and values), one instruction of as
//    many lanes, KV_RING tiles ahead on one mbarrier a tile.
//  * Scores: S^T = K q^T on m16n8k16 mma.sync, keys as rows.  A code alone in a half
//    word is the fp16 subnormal c 2^-24 (low nibble) or c 2^-20 (high), one AND per
//    operand register; one packed FMA more makes it (c - z) 2^-14, exact and a normal
//    number.  (The matrix pipe aligns subnormals by their exponent field: with the codes as
//    they are and the zero point applied to the product, s (sum c q - z sum q), a channel
//    in which the query is large and the keys small cost the scores up to 17 times the fp32
//    sums' bound.  32 ragged sequences took 54 us then, two of 131000 keys 82.)
//  * out^T = V^T p: two keys' words of the same elements, merged half by half, give
//    operand registers of two keys again by one AND.  A value's scale goes into its
//    probability: u = p s, in two fp16 parts (22 bits), scaled by a power of two that
//    follows the largest s of the warp's keys (n - 9 bits fewer for a key whose s is 2^-n
//    of that one, n > 9: below the output's rounding up to n = 20); its zero point into
//    sum u (z - 8), subtracted at the end
//    from the sum over the codes c - 8.
//  * The running maximum follows the scores in steps of KV_LAZY: p = 2^(score - m) may
//    reach 2^KV_LAZY before the outputs are scaled again, which few tiles ask for.
//  * The rows of an operand are the keys kv_key(g) of its eight: the same keys are
//    then two neighbouring columns of the other product's operand, and the reads of
//    shared memory hit every bank as often (keys) or twice (values).
// Measured (B200, 32 heads on 8 of 128): 57 us for 32 ragged sequences of up to 8000 keys
// (178 MB: 3.1 TB/s), 85 us for two of 131000 in groups of 64 (2.9 TB/s), 6.5 us for one of
// 777; bound by about 810 instructions a tile and warp (240 unpack, 32 to 48 multiply),
// issued in 63 % of the cycles by four warps a scheduler, and by the uneven last round of
// chunks.
#include <cmath>

#include "common.cuh"
#include "tc_common.cuh"
#include "w4_rows.cuh"

namespace gptq {

constexpr int KV_WARPS = 4, KV_TILE = 32, KV_RING = 3;
constexpr float KV_LAZY = 7.f;
constexpr float KV_NONE = -3e38f;          // the maximum of no scores: finite, so that no difference is NaN
constexpr int KV_CLUSTER = 1024;           // most keys of a cluster's chunk
constexpr int KV_ALONE = 256;              // up to so many keys: one chunk, no second kernel
constexpr int KV_TILES = 65535;            // most key heads times row tiles of a call (grid rows)

struct KvAttn {
    const __half* q;
    int64_t tokens, seqs, pages, width, window;
    int max_q, max_len, hq, hkv, page_shift;
    const uint32_t* kc;
    const __half2* kp;
    const uint32_t* vc;
    const __half2* vp;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* start;
    float scale;                           // times log2(e)
    int chunk, splits, row_tiles, cluster; // cluster: the chunks of a row tile are one
    int grp;                               // query heads per key head
    uint32_t grp_mul;                      // ceil(2^32 / grp): r / grp = r grp_mul >> 32 for r grp < 2^32
    float* part;                           // unit x 8 rows x (D, then maximum and sum)
    __half* out;
};

// Key of row g of an operand's eight
__device__ __forceinline__ int kv_key(int g) { return (g & 1) ? 4 + ((g >> 1) ^ 1) : (g >> 1); }

// 2^x, 2 ulp, 0 for -inf and below the normal numbers
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Two codes of values, c 2^-14 / scale each -> (c - 8) 2^-14, exact: normal numbers around 0, so
// that neither the matrix pipe's alignment of subnormals nor the rounding of long sums of
// codes of one sign costs bits of their difference to the zero points
__device__ __forceinline__ uint32_t kv_center(uint32_t v, float scale)
{
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(scale),
                              __float2half2_rn(-8.f * 0x1p-14f));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Minus the zero point (the high half of a parameter word), times 2^-14, twice
__device__ __forceinline__ uint32_t kv_minus(uint32_t param)
{
    const uint32_t z = __byte_perm(param, param, 0x3232);
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&z), __float2half2_rn(-0x1p-14f));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Two codes of a key, c 2^-14 / scale each -> (c - z) 2^-14, exact
__device__ __forceinline__ uint32_t kv_sub(uint32_t v, float scale, uint32_t minus)
{
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(scale),
                              *reinterpret_cast<const __half2*>(&minus));
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ void kv_bulk(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// Query of a row, whose head is the rest (rows are at most 8 x 65535)
__device__ __forceinline__ int kv_query(const KvAttn& p, int r)
{
    return p.grp == 1 ? r : int(__umulhi(uint32_t(r), p.grp_mul));
}

// Place of row r of a sequence in q and out: elements from the sequence's first row on
__device__ __forceinline__ int64_t kv_row(const KvAttn& p, int64_t s0, int hk, int r)
{
    const int i = kv_query(p, r);
    return (s0 + i) * p.hq + hk * p.grp + (r - i * p.grp);
}

// What a row tile of a sequence sees
struct KvSpan {
    bool ok;                               // the sequence's range and length are valid
    int64_t s0;
    int n, L, rows, lo, base, hi;          // queries, keys, rows; keys [lo, hi) are seen, base: lo's tile
};

__device__ __forceinline__ KvSpan kv_span(const KvAttn& p, int b, int rt)
{
    KvSpan s;
    const int64_t s0 = p.start[b], s1 = p.start[b + 1], L = p.lens[b];
    s.ok = s0 >= 0 && s1 >= s0 && s1 <= p.tokens && s1 - s0 <= p.max_q && L >= 0 && L <= p.max_len;
    s.s0 = s0;
    s.n = int(s1 - s0);
    s.L = int(L);
    s.rows = s.n * p.grp - rt * 8;         // from the tile's first row on
    if (!s.ok || s.rows <= 0) { s.rows = s.lo = s.base = s.hi = 0; return s; }
    const int i0 = kv_query(p, rt * 8), i1 = kv_query(p, rt * 8 + min(s.rows, 8) - 1);
    s.hi = max(0, s.L - s.n + i1 + 1);
    const int64_t lo = p.window > 0 ? int64_t(s.L) - s.n + i0 + 1 - p.window : 0;
    s.lo = int(max(lo, int64_t(0)));
    s.base = s.lo & ~(KV_TILE - 1);
    return s;
}

template <int D, int G> struct KvShape {
    static constexpr int NB = D / 32, GB = NB / G;         // blocks of 32 elements, of a group
    static constexpr int CODES = KV_TILE * D / 2, PARAMS = KV_TILE * G * 4;
    static constexpr int SLOT = 2 * (CODES + PARAMS);
    static constexpr int RING = KV_WARPS * KV_RING * SLOT;
    static constexpr int JOIN = KV_WARPS * 8 * D * 4;      // in the ring's place, at the end
    static constexpr int SMEM = (RING > JOIN ? RING : JOIN) + 128;
    static constexpr int CTAS = D == 64 ? 4 : D == 128 && G < 4 ? 4 : 2;   // per SM, by registers
};

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
}

// The address of shared memory `a` in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer_addr(uint32_t a, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}

__device__ __forceinline__ float peer_f(uint32_t a)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ float4 peer_f4(uint32_t a)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

// HALF: at most four rows, whose second parts of u take the other four columns of the
// operand (16 products a tile instead of 32 for the values, each of which holds the
// scheduler up for six cycles)
template <int D, int G, bool HALF>
__global__ void __launch_bounds__(KV_WARPS * 32, KvShape<D, G>::CTAS) kv4_attention_kernel(const KvAttn p)
{
    using Sh = KvShape<D, G>;
    constexpr int NB = Sh::NB, GB = Sh::GB;
    constexpr uint32_t LO = 0x000F000Fu, HI = 0x00F000F0u, ALL = 0xffffffffu;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float poison[8];
    __shared__ float wm[KV_WARPS][8], wl[KV_WARPS][8], cm[8], cl[8];
    __shared__ __align__(8) uint64_t bars[KV_WARPS * KV_RING];
    __shared__ int abort;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int warp = __shfl_sync(ALL, threadIdx.x >> 5, 0);
    const int b = blockIdx.z, hk = blockIdx.y / p.row_tiles, rt = blockIdx.y - hk * p.row_tiles;
    const KvSpan sp = kv_span(p, b, rt);
    if (!sp.ok) {
        if (threadIdx.x == 0) atomicCAS(&g_device_status, 0, kErrIndex);
        return;
    }
    if (sp.rows <= 0) return;
    const int c0 = sp.base + int(blockIdx.x) * p.chunk, c1 = min(sp.hi, c0 + p.chunk);
    if (!p.cluster && c0 >= sp.hi && (blockIdx.x > 0 || p.splits > 1)) return;
    const int tiles = c1 > c0 ? (c1 - c0 + KV_TILE - 1) / KV_TILE : 0;

    if (lane == 0)
        for (int i = 0; i < KV_RING; ++i) mbar_init(&bars[warp * KV_RING + i], 1);
    if (threadIdx.x == 0) abort = 0;
    fence_mbar_init();
    __syncwarp();
    // producer: lanes 0 .. 7, half tile lane / 4, array lane % 4 (key codes, value codes,
    // key and value parameters); the page of the next tile is looked up a tile ahead
    const uint32_t ring = smem_u32(smem) + warp * (KV_RING * Sh::SLOT);
    const uint32_t bar0 = smem_u32(&bars[warp * KV_RING]);
    const int half = (lane >> 2) & 1, what = lane & 3;
    const bool whole = p.page_shift >= 5, copies = lane < (whole ? 4 : 8);
    const int32_t* table = p.table + int64_t(b) * p.width;
    const uint32_t keyb = what < 2 ? D / 2 : G * 4;        // bytes of a key
    const uint32_t mask = (1u << p.page_shift) - 1u;
    const uint32_t pageb = (uint32_t(p.hkv) * keyb) << p.page_shift;
    const uint8_t* from0 =
        (what == 0 ? reinterpret_cast<const uint8_t*>(p.kc)
                   : what == 1 ? reinterpret_cast<const uint8_t*>(p.vc)
                               : what == 2 ? reinterpret_cast<const uint8_t*>(p.kp)
                                           : reinterpret_cast<const uint8_t*>(p.vp)) +
        ((uint32_t(hk) * keyb) << p.page_shift);
    const uint32_t to0 = ring + (what < 2 ? what * Sh::CODES : 2 * Sh::CODES + (what - 2) * Sh::PARAMS) +
                         half * keyb * 16;
    int ptile = warp, pslot = 0, pkey = c0 + warp * KV_TILE + half * 16;
    bool stray = false;                                    // a page out of range was met
    uint32_t phase = 0;                                    // parity of the slot to read; from W4_GONE on:
                                                           // a wait gave up, the results are void
    uint32_t page = 0;
    // (pages of 16: a half tile in front of the first key that is seen takes page 0, its own
    // may be freed)
    auto look = [&]() {
        page = pkey < c1 && (whole || pkey + 16 > sp.lo) ? uint32_t(table[pkey >> p.page_shift]) : 0u;
    };
    auto issue = [&]() {
        if (ptile >= tiles) return;
        const bool bad = page >= uint32_t(p.pages);
        if (__any_sync(ALL, bad || phase >= W4_GONE)) {
            if (__any_sync(ALL, phase >= W4_GONE)) { phase |= W4_GONE; ptile = tiles; return; }
            if (bad) page = 0u;                            // page 0 in its place; its keys are masked
            if (lane == 0) atomicCAS(&g_device_status, 0, kErrIndex);
            stray = true;
        }
        const uint32_t bar = bar0 + pslot * 8;
        const bool both = c0 + ptile * KV_TILE + 16 < c1;  // halves of the tile
        if (lane == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                         "r"(both ? Sh::SLOT : Sh::SLOT / 2)
                         : "memory");
        __syncwarp();
        if (copies && pkey < c1)
            kv_bulk(to0 + pslot * Sh::SLOT, from0 + (uint64_t(page) * pageb + (uint32_t(pkey) & mask) * keyb),
                    keyb << (whole && both ? 5 : 4), bar);
        ptile += KV_WARPS;
        pkey += KV_WARPS * KV_TILE;
        pslot = pslot + 1 == KV_RING ? 0 : pslot + 1;
        look();
    };
    look();
#pragma unroll
    for (int i = 0; i < KV_RING; ++i) issue();

    // the queries' operand (row g of the tile: elements 32 i + 8 t .. of block i, in the
    // order of a word's nibbles)
    uint32_t qf[NB][4];
    {
        const int r = HALF ? g & 3 : g;
        const bool on = r < sp.rows;
        const __half* src = p.q + kv_row(p, sp.s0, hk, rt * 8 + (on ? r : 0)) * D;
        float sum = 0.f;                                   // finite where the elements are
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (on) v = *reinterpret_cast<const uint4*>(src + 32 * i + 8 * t);
            const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = __half22float2(h[e]);
                sum += f.x + f.y;
            }
            qf[i][0] = __byte_perm(v.x, v.z, 0x5410);      // elements 0, 4
            qf[i][1] = __byte_perm(v.y, v.w, 0x5410);      // 2, 6
            qf[i][2] = __byte_perm(v.x, v.z, 0x7632);      // 1, 5
            qf[i][3] = __byte_perm(v.y, v.w, 0x7632);      // 3, 7
        }
        sum += __shfl_xor_sync(ALL, sum, 1);
        sum += __shfl_xor_sync(ALL, sum, 2);
        if (warp == 0 && t == 0) poison[g] = sum * 0.f;
    }
    __syncthreads();
    // rows 2 t and 2 t + 1: the keys they see
    int lim[2], from[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int r = rt * 8 + min((2 * t + j) & (HALF ? 3 : 7), sp.rows - 1);
        lim[j] = sp.L - sp.n + kv_query(p, r) + 1;
        const int64_t lo = p.window > 0 ? int64_t(lim[j]) - p.window : 0;
        from[j] = int(max(lo, int64_t(0)));
    }
    const int all_lim = sp.L - sp.n + kv_query(p, rt * 8) + 1;    // keys [all_from, all_lim): seen by every row
    const int last = sp.L - sp.n + kv_query(p, rt * 8 + min(sp.rows, 8) - 1) + 1;
    const int all_from = p.window > 0 ? int(max(int64_t(last) - p.window, int64_t(0))) : 0;

    float m[2] = {KV_NONE, KV_NONE}, l[2] = {0.f, 0.f}, zs[G][2] = {};
    float o[NB][2][4] = {};                                // [block][nibbles 0, 2 | 1, 3]
    uint32_t top_exp = 0;                                  // biased fp16 exponent of the largest value scale
    float factor = 0x1p21f;                                // 2^(21 - top_exp): u < 2^(7 + KV_LAZY)
    const float up = p.scale * 0x1p14f;
    // what the scores of rows 2 t, 2 t + 1 begin with: 0, or NaN for a query that is not
    // finite (an infinity alone can make every score -inf, which is no key seen)
    const float start[2] = {poison[2 * t], poison[2 * t + 1]};
    int slot = 0;
    for (int tile = warp; tile < tiles; tile += KV_WARPS) {
        const int k0 = c0 + tile * KV_TILE;
        if (phase < W4_GONE && !w4_try_wait(bar0 + slot * 8, phase) &&
            !w4_wait_long(bar0 + slot * 8, phase, &abort)) {   // its copies in flight, then no more
            for (int i = 0; i < KV_RING && tile + i * KV_WARPS < tiles; ++i) {
                const bool wrap = slot + i >= KV_RING;
                w4_land(bar0 + (slot + i - (wrap ? KV_RING : 0)) * 8, phase ^ uint32_t(wrap));
            }
            phase |= W4_GONE;
        }
        const uint8_t* base = smem + warp * (KV_RING * Sh::SLOT) + slot * Sh::SLOT;
        float sc[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {                      // scores of 16 keys
            uint32_t kw[2][NB];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t* src = base + (h * 16 + i * 8 + kv_key(g)) * (D / 2) + t * (NB * 4);
                if constexpr (NB == 2) {
                    const uint2 v = *reinterpret_cast<const uint2*>(src);
                    kw[i][0] = v.x; kw[i][1] = v.y;
                } else {
#pragma unroll
                    for (int u = 0; u < NB / 4; ++u) {
                        const uint4 v = *reinterpret_cast<const uint4*>(src + u * 16);
                        kw[i][4 * u] = v.x; kw[i][4 * u + 1] = v.y;
                        kw[i][4 * u + 2] = v.z; kw[i][4 * u + 3] = v.w;
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[h][e] = start[e & 1];
#pragma unroll
            for (int k = 0; k < G; ++k) {
                float sx[2];
                uint32_t mz[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {              // scale, and minus the zero point twice
                    const uint32_t v = *reinterpret_cast<const uint32_t*>(
                        base + 2 * Sh::CODES + ((h * 16 + i * 8 + kv_key(g)) * G + k) * 4);
                    sx[i] = __half2float(__ushort_as_half((unsigned short)v)) * up;
                    mz[i] = kv_minus(v);
                }
                float dot[4];
#pragma unroll
                for (int i = 0; i < GB; ++i) {
                    const uint32_t a = kw[0][k * GB + i], c = kw[1][k * GB + i];
                    const uint32_t a8 = a >> 8, c8 = c >> 8;
                    const uint32_t (&f)[4] = qf[k * GB + i];
                    const uint32_t l0 = kv_sub(a & LO, 1024.f, mz[0]), l1 = kv_sub(c & LO, 1024.f, mz[1]);
                    const uint32_t l2 = kv_sub(a8 & LO, 1024.f, mz[0]), l3 = kv_sub(c8 & LO, 1024.f, mz[1]);
                    const uint32_t h0 = kv_sub(a & HI, 64.f, mz[0]), h1 = kv_sub(c & HI, 64.f, mz[1]);
                    const uint32_t h2 = kv_sub(a8 & HI, 64.f, mz[0]), h3 = kv_sub(c8 & HI, 64.f, mz[1]);
                    if (i == 0) mma_16816_first(dot, l0, l1, l2, l3, f[0], f[1]);
                    else mma_16816(dot, l0, l1, l2, l3, f[0], f[1]);
                    mma_16816(dot, h0, h1, h2, h3, f[2], f[3]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 v = fma2(make_float2(sx[i], sx[i]), make_float2(dot[2 * i], dot[2 * i + 1]),
                                          make_float2(sc[h][2 * i], sc[h][2 * i + 1]));
                    sc[h][2 * i] = v.x;
                    sc[h][2 * i + 1] = v.y;
                }
            }
        }
        const bool edge = k0 < all_from || k0 + KV_TILE > all_lim || stray;
        uint32_t there = 3u;                               // halves with a valid page
        if (edge) {                                        // some keys are not seen by some row
            if (stray)
                for (int h = 0; h < 2; ++h) {
                    const int key = k0 + h * 16;
                    if (key < c1 && (whole || key + 16 > sp.lo) &&
                        uint32_t(table[key >> p.page_shift]) >= uint32_t(p.pages))
                        there &= ~(1u << h);
                }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = k0 + h * 16 + (e >> 1) * 8 + kv_key(g);
                    if (key >= lim[e & 1] || key < from[e & 1] || !((there >> h) & 1u))
                        sc[h][e] = -INFINITY;
                }
        }
        // scales and zero points of the lane's four values
        uint32_t vz[2][2][G], big = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < G; ++k)
                    vz[h][i][k] = *reinterpret_cast<const uint32_t*>(
                        base + 2 * Sh::CODES + Sh::PARAMS +
                        ((h * 16 + i * 8 + kv_key(g)) * G + k) * 4);
        if (edge) {                                        // keys that no row sees: whatever the slot holds
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int key = k0 + h * 16 + i * 8 + kv_key(g);
                    if (key < sp.lo || key >= c1 || !((there >> h) & 1u))
#pragma unroll
                        for (int k = 0; k < G; ++k) vz[h][i][k] = 0u;
                }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < G; ++k) big = max(big, vz[h][i][k] & 0x7fffu);
        float mx[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            mx[j] = fmaxf(fmaxf(sc[0][j], sc[0][2 + j]), fmaxf(sc[1][j], sc[1][2 + j]));
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) mx[j] = fmaxf(mx[j], __shfl_xor_sync(ALL, mx[j], s));
        }
        big = __reduce_max_sync(ALL, big) >> 10;
        if (__any_sync(ALL, mx[0] > m[0] + KV_LAZY || mx[1] > m[1] + KV_LAZY) || big > top_exp) {
            float down = 1.f;                              // of the outputs, for a larger value scale
            if (big > top_exp) {
                down = __uint_as_float((127u - (big - top_exp)) << 23);
                top_exp = big;
                factor = __uint_as_float((127u + 21u - big) << 23);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float mn = fmaxf(m[j], mx[j]);
                const float al = ex2(m[j] - mn), ad = al * down;
                m[j] = mn;
                l[j] *= al;
#pragma unroll
                for (int k = 0; k < G; ++k) zs[k][j] *= ad;
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        o[i][x][j] *= ad;
                        o[i][x][2 + j] *= ad;
                    }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sc[h][e] = ex2(sc[h][e] - m[e & 1]);
                l[e & 1] += sc[h][e];
            }
#pragma unroll
        for (int h = 0; h < 2; ++h) {                      // out += V^T u of 16 keys
            uint32_t vw[4][(NB + 1) / 2];                  // keys 2 t, 2 t + 1, and 8 on
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t* src = base + Sh::CODES +
                                     (h * 16 + (i >> 1) * 8 + kv_key(2 * t + (i & 1))) * (D / 2) +
                                     g * (NB * 2);
                if constexpr (NB == 2) {
                    vw[i][0] = *reinterpret_cast<const uint32_t*>(src);
                } else if constexpr (NB == 4) {
                    const uint2 v = *reinterpret_cast<const uint2*>(src);
                    vw[i][0] = v.x; vw[i][1] = v.y;
                } else {
                    const uint4 v = *reinterpret_cast<const uint4*>(src);
                    vw[i][0] = v.x; vw[i][1] = v.y; vw[i][2] = v.z; vw[i][3] = v.w;
                }
            }
#pragma unroll
            for (int k = 0; k < G; ++k) {
                uint32_t bh[2], bl[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 sz = __half22float2(*reinterpret_cast<const __half2*>(&vz[h][i][k]));
                    const float s = sz.x * factor, z = sz.y - 8.f;
                    const float u0 = sc[h][2 * i] * s, u1 = sc[h][2 * i + 1] * s;
                    zs[k][0] = fmaf(u0, z, zs[k][0]);
                    zs[k][1] = fmaf(u1, z, zs[k][1]);
                    const __half2 uh = __floats2half2_rn(u0, u1);
                    const float2 f = __half22float2(uh);
                    const __half2 ul = __floats2half2_rn(u0 - f.x, u1 - f.y);
                    const uint32_t wh = *reinterpret_cast<const uint32_t*>(&uh);
                    const uint32_t wl = *reinterpret_cast<const uint32_t*>(&ul);
                    bh[i] = movmatrix(HALF && t >= 2 ? wl : wh);
                    if (!HALF) bl[i] = movmatrix(wl);
                }
#pragma unroll
                for (int i = k * GB; i < (k + 1) * GB; ++i) {
                    const uint32_t pick = (i & 1) ? 0x7632 : 0x5410;
                    const uint32_t a = __byte_perm(vw[0][i / 2], vw[1][i / 2], pick);
                    const uint32_t c = __byte_perm(vw[2][i / 2], vw[3][i / 2], pick);
                    const uint32_t a8 = a >> 8, c8 = c >> 8;
                    const uint32_t n0 = kv_center(a & LO, 1024.f), n1 = kv_center(a8 & LO, 1024.f);
                    const uint32_t n2 = kv_center(c & LO, 1024.f), n3 = kv_center(c8 & LO, 1024.f);
                    const uint32_t h0 = kv_center(a & HI, 64.f), h1 = kv_center(a8 & HI, 64.f);
                    const uint32_t h2 = kv_center(c & HI, 64.f), h3 = kv_center(c8 & HI, 64.f);
                    mma_16816(o[i][0], n0, n1, n2, n3, bh[0], bh[1]);
                    mma_16816(o[i][1], h0, h1, h2, h3, bh[0], bh[1]);
                    if (!HALF) {
                        mma_16816(o[i][0], n0, n1, n2, n3, bl[0], bl[1]);
                        mma_16816(o[i][1], h0, h1, h2, h3, bl[0], bl[1]);
                    }
                }
            }
        }
        if (++slot == KV_RING) { slot = 0; phase ^= 1u; }
        __syncwarp();                                      // every lane has read the slot
        issue();
    }
    // sums over the keys of all lanes, then the warp's result in its own units
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) {
            l[j] += __shfl_xor_sync(ALL, l[j], s);
#pragma unroll
            for (int k = 0; k < G; ++k) zs[k][j] += __shfl_xor_sync(ALL, zs[k][j], s);
        }
    if (HALF)
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[i][e >> 2][e & 3] += __shfl_xor_sync(ALL, o[i][e >> 2][e & 3], 2);
    __syncthreads();                                       // every warp is done with its ring
    const float undo = 1.f / factor;
    float* mine = reinterpret_cast<float*>(smem) + warp * (8 * D);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (HALF && t >= 2) break;
        if (g == 0) { wm[warp][2 * t + j] = m[j]; wl[warp][2 * t + j] = l[j]; }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const float z = zs[i / GB][j];
            *reinterpret_cast<float4*>(mine + (2 * t + j) * D + 32 * i + 4 * g) = make_float4(
                fmaf(o[i][0][j], 0x1p14f, -z) * undo, fmaf(o[i][1][j], 0x1p14f, -z) * undo,
                fmaf(o[i][0][2 + j], 0x1p14f, -z) * undo, fmaf(o[i][1][2 + j], 0x1p14f, -z) * undo);
        }
    }
    __syncthreads();
    const int rows = min(sp.rows, 8);
    const int64_t unit = (int64_t(b) * gridDim.y + blockIdx.y) * p.splits + blockIdx.x;
    float* dst = p.part + unit * (8 * (D + 2));
    if (threadIdx.x < rows) {                              // the warps' weights in row r
        const int r = threadIdx.x;
        float top = KV_NONE, sum = 0.f, c[KV_WARPS];
#pragma unroll
        for (int w = 0; w < KV_WARPS; ++w) top = fmaxf(top, wm[w][r]);
#pragma unroll
        for (int w = 0; w < KV_WARPS; ++w) {               // (a warp without keys: its sums are 0)
            c[w] = ex2(wm[w][r] - top);
            sum = fmaf(c[w], wl[w][r], sum);
        }
        if (p.cluster) { cm[r] = top; cl[r] = sum; }
        else if (p.splits > 1) { dst[8 * D + r] = top; dst[8 * D + 8 + r] = sum; }
        // (sum 0: no key is seen; NaN, from a query that is not finite, goes on to the row)
        const float scale = p.splits > 1 ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int w = 0; w < KV_WARPS; ++w) wm[w][r] = c[w] * scale;
    }
    __syncthreads();
    auto put = [&](int r, int d, float4 v) {
        alignas(8) const __half2 h[2] = {__floats2half2_rn(v.x, v.y), __floats2half2_rn(v.z, v.w)};
        *reinterpret_cast<uint2*>(p.out + kv_row(p, sp.s0, hk, rt * 8 + r) * D + d) =
            *reinterpret_cast<const uint2*>(h);
    };
    for (int e = threadIdx.x * 4; e < rows * D; e += KV_WARPS * 32 * 4) {
        const int r = e / D, d = e - r * D;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < KV_WARPS; ++w) {
            const float c = wm[w][r];
            const float4 u = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) +
                                                              w * (8 * D) + e);
            v.x = fmaf(c, u.x, v.x); v.y = fmaf(c, u.y, v.y);
            v.z = fmaf(c, u.z, v.z); v.w = fmaf(c, u.w, v.w);
        }
        if (p.cluster) *reinterpret_cast<float4*>(reinterpret_cast<float*>(smem) + e) = v;
        else if (p.splits == 1) put(r, d, v);
        else *reinterpret_cast<float4*>(dst + e) = v;
    }
    if (p.cluster) {                               // each CTA joins its share of the elements
        cluster_sync();
        const uint32_t am = smem_u32(cm), al = smem_u32(cl), ao = smem_u32(smem);
        for (int e = (blockIdx.x * (KV_WARPS * 32) + threadIdx.x) * 4; e < rows * D;
             e += p.splits * (KV_WARPS * 32 * 4)) {
            const int r = e / D;
            float top = KV_NONE, sum = 0.f;
            for (int s = 0; s < p.splits; ++s) top = fmaxf(top, peer_f(peer_addr(am + r * 4, s)));
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int s = 0; s < p.splits; ++s) {
                const float c = ex2(peer_f(peer_addr(am + r * 4, s)) - top);
                sum = fmaf(c, peer_f(peer_addr(al + r * 4, s)), sum);
                const float4 u = peer_f4(peer_addr(ao + e * 4, s));
                v.x = fmaf(c, u.x, v.x); v.y = fmaf(c, u.y, v.y);
                v.z = fmaf(c, u.z, v.z); v.w = fmaf(c, u.w, v.w);
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            put(r, e - r * D, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
        }
        cluster_sync();                                    // the others have read this CTA's memory
    }
}

// out = the chunks' results joined: one warp per row
template <int D> __global__ void __launch_bounds__(256) kv4_join_kernel(const KvAttn p)
{
    constexpr int E = D / 32;
    pdl_wait();
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int b = blockIdx.y, hk = blockIdx.x / p.row_tiles, rt = blockIdx.x - hk * p.row_tiles;
    const KvSpan sp = kv_span(p, b, rt);
    if (!sp.ok || r >= sp.rows) return;
    const int n = sp.hi > sp.base ? (sp.hi - sp.base + p.chunk - 1) / p.chunk : 0;
    const float* part = p.part + (int64_t(b) * gridDim.x + blockIdx.x) * p.splits * (8 * (D + 2));
    float top = KV_NONE, sum = 0.f, v[E] = {};
    for (int s = lane; s < n; s += 32) top = fmaxf(top, part[int64_t(s) * (8 * (D + 2)) + 8 * D + r]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll 4
    for (int s = 0; s < n; ++s) {
        const float* src = part + int64_t(s) * (8 * (D + 2));
        const float c = ex2(src[8 * D + r] - top);         // (a chunk that this row does not see: 0s)
        sum = fmaf(c, src[8 * D + 8 + r], sum);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = fmaf(c, src[r * D + e * 32 + lane], v[e]);
    }
    __half* dst = p.out + kv_row(p, sp.s0, hk, rt * 8 + r) * D;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e * 32 + lane] = __float2half_rn(sum == 0.f ? 0.f : v[e] / sum);
}

// Keys per chunk: a multiple of a CTA's round of tiles, and as few chunks as give each
// SM eight CTAs (two rounds of four) when every sequence has the bound's length; twelve
// from 8 sequences on, whose lengths may differ (us at six, eight, twelve, sixteen and
// twenty-four: 12 ragged ones of up to 8000: 27, 29, 30, 30, 34; 16: 33, 36, 35, 35, 37;
// 32: 59, 62, 57, 57, 59; 8 of 40000: 64, 63, 62, 63, 67; two of 131000: 88, 85, 98 with
// sixteen, 111 with twenty-four; 6 of 40000: 54, 53, then 55 and 60)
struct KvPlan { int chunk, splits; int64_t row_tiles; bool cluster; size_t bytes; };

KvPlan kv_plan(int64_t seqs, int hq, int hkv, int D, int64_t max_q, int64_t max_len, int64_t window)
{
    KvPlan k{};
    k.row_tiles = std::min<int64_t>((max_q * (hq / hkv) + 7) / 8, KV_TILES / hkv + 1);
    int64_t span = max_len;
    if (window > 0) span = std::min(span, window + max_q + 2 * KV_TILE);
    span = std::max<int64_t>(span, 1);
    constexpr int ROUND = KV_WARPS * KV_TILE;
    const int64_t units = seqs * hkv * k.row_tiles;
    const int64_t aim = 148 * (seqs < 8 ? 8 : 12);
    auto rounded = [&](int64_t keys) {
        return std::max<int64_t>(ROUND, (keys + ROUND - 1) / ROUND * ROUND);
    };
    // clusters of two to eight chunks where all of them fit the GPU at once (four CTAs an
    // SM; heads of 256, with two, may take two rounds) with at most KV_CLUSTER keys each: one
    // sequence of 777 keys in one launch
    const int64_t most = std::min<int64_t>(8, 148 * 4 / std::max<int64_t>(units, 1));
    int64_t chunk = rounded((units * span + aim - 1) / aim);
    if (span <= KV_ALONE) {
        chunk = std::max(chunk, rounded(span));
    } else if (most >= 2 && rounded((span + most - 1) / most) <= KV_CLUSTER) {
        chunk = rounded((span + most - 1) / most);
        k.cluster = true;
    } else {
        chunk = std::max(chunk, rounded((span + 4095) / 4096));
    }
    k.chunk = int(std::min<int64_t>(chunk, int64_t(1) << 30));
    k.splits = int((span + k.chunk - 1) / k.chunk);
    k.cluster = k.cluster && k.splits > 1;
    // None where the chunks are joined in a cluster or there is one: so is every smaller
    // call then.  Otherwise units splits < units + aim by the choice of chunk, and one chunk
    // from units = aim on; this bound grows with every argument, so a workspace for the
    // bounds serves every smaller call.
    if (k.cluster || span <= KV_ALONE) return k;
    const int64_t parts = std::min(units * ((max_len + ROUND - 1) / ROUND + 1),
                                   std::min<int64_t>(units, 148 * 12) + 148 * 12);
    k.bytes = align_up(size_t(parts) * 8 * (D + 2) * 4, 256);
    return k;
}

}  // namespace gptq

extern "C" size_t gptq_kv4_attention_workspace_bytes(int64_t seqs, int q_heads, int kv_heads,
                                                     int head_dim, int64_t max_q_len,
                                                     int64_t max_seq_len)
{
    if (seqs <= 0 || q_heads <= 0 || kv_heads <= 0 || head_dim <= 0 || max_q_len <= 0 ||
        max_seq_len < 0)
        return 0;
    if (seqs > 65535 || q_heads > 1024 || kv_heads > 1024 || q_heads % kv_heads != 0 || head_dim > 256 ||
        max_q_len > (int64_t(1) << 24) || max_seq_len > (int64_t(1) << 30))
        return 0;
    return gptq::kv_plan(seqs, q_heads, kv_heads, head_dim, max_q_len, max_seq_len, 0).bytes;
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
        (max_seq_len > 0 && !block_table))
        return GPTQ_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_codes) || !aligned16(k_params) || !aligned16(v_codes) ||
        !aligned16(v_params) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(q_start, 4) || !aligned16(out) || !aligned16(ws))
        return GPTQ_ERR_INVALID_ARG;
    if (max_q_len > (int64_t(1) << 24)) return GPTQ_ERR_SHAPE;
    // no query reaches back further than max_seq_len keys (and a caller's "no limit" may be
    // the largest number there is: sums with it would wrap)
    if (window >= max_seq_len) window = 0;
    if (ws_bytes < gptq_kv4_attention_workspace_bytes(seqs, q_heads, kv_heads, head_dim, max_q_len,
                                                      max_seq_len))
        return GPTQ_ERR_INVALID_ARG;
    const int64_t max_q = std::min(max_q_len, tokens);
    const KvPlan plan = kv_plan(seqs, q_heads, kv_heads, head_dim, max_q, max_seq_len, window);
    if (plan.bytes > ws_bytes || (plan.bytes && !ws)) return GPTQ_ERR_INVALID_ARG;
    if (kv_heads * plan.row_tiles > KV_TILES) return GPTQ_ERR_SHAPE;
    KvAttn p{};
    p.q = reinterpret_cast<const __half*>(q);
    p.tokens = tokens; p.seqs = seqs; p.pages = pages; p.width = table_width;
    p.window = window; p.max_q = (int)max_q; p.max_len = (int)max_seq_len;
    p.hq = q_heads; p.hkv = kv_heads;
    p.grp = q_heads / kv_heads;
    p.grp_mul = uint32_t(((uint64_t(1) << 32) + p.grp - 1) / p.grp);
    while ((1 << p.page_shift) < page_size) ++p.page_shift;
    p.kc = k_codes; p.kp = reinterpret_cast<const __half2*>(k_params);
    p.vc = v_codes; p.vp = reinterpret_cast<const __half2*>(v_params);
    p.table = block_table; p.lens = seq_lens; p.start = q_start;
    p.scale = scale * 1.4426950408889634f;
    p.cluster = plan.cluster;
    p.chunk = plan.chunk; p.splits = plan.splits; p.row_tiles = (int)plan.row_tiles;
    p.part = static_cast<float*>(ws);
    p.out = reinterpret_cast<__half*>(out);
    cudaStream_t st = as_stream(stream);
    KernelTimer kt(kKKvAttention, st);
    const dim3 grid((unsigned)p.splits, (unsigned)(kv_heads * p.row_tiles), (unsigned)seqs);
    const bool few = max_q * p.grp <= 4;
    auto run = [&](auto kern, auto kern4, auto join, int smem, std::atomic<bool> (&done)[2][64]) -> int {
        if (few) kern = kern4;
        if (!smem_opt_in(reinterpret_cast<const void*>(kern), smem, done[few])) return GPTQ_ERR_CUDA;
        if (plan.cluster) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = grid;
            cfg.blockDim = KV_WARPS * 32;
            cfg.dynamicSmemBytes = smem;
            cfg.stream = st;
            cudaLaunchAttribute at{};
            at.id = cudaLaunchAttributeClusterDimension;
            at.val.clusterDim.x = grid.x;
            at.val.clusterDim.y = at.val.clusterDim.z = 1;
            cfg.attrs = &at;
            cfg.numAttrs = 1;
            if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return GPTQ_ERR_CUDA;
            count_launches();
            return launch_status();
        }
        kern<<<grid, KV_WARPS * 32, smem, st>>>(p);
        if (launch_status() != GPTQ_OK) return GPTQ_ERR_CUDA;
        count_launches();
        if (p.splits > 1) {
            if (launch_after(join, dim3((unsigned)(kv_heads * p.row_tiles), (unsigned)seqs), 256, 0,
                             st, p) != cudaSuccess)
                return GPTQ_ERR_CUDA;
            count_launches();
        }
        return launch_status();
    };
#define KV_RUN(D, G)                                                                            \
    if (head_dim == D && g * G == D) {                                                          \
        static std::atomic<bool> done[2][64];                                                   \
        return run(kv4_attention_kernel<D, G, false>, kv4_attention_kernel<D, G, true>,         \
                   kv4_join_kernel<D>, KvShape<D, G>::SMEM, done);                              \
    }
    KV_RUN(64, 1) KV_RUN(64, 2)
    KV_RUN(128, 1) KV_RUN(128, 2) KV_RUN(128, 4)
    KV_RUN(256, 1) KV_RUN(256, 2) KV_RUN(256, 4) KV_RUN(256, 8)
#undef KV_RUN
    return GPTQ_ERR_UNSUPPORTED;
}
