// The tcgen05 W4A16 product (w4a16_tc.cu) for other kernels of the library.
#pragma once

#include "common.cuh"
#include "tc_common.cuh"

namespace gptq {

struct WqPlan {
    bool small;                          // batch tiles of up to 32
    int ntile, n_rt, n_nt;               // columns of a batch tile; row and batch tiles
    int chunk, chunks_per_split, ksplit; // columns per accumulation; splits of K
};

WqPlan wq_plan(int64_t batch, int64_t m, int64_t d, int64_t gsz, int sms);

// y = xp Q^T for activations xp in the order of wq_gathered.  split_stride == 0: the
// splits meet in y by atomic adds; else split i writes y + i split_stride.
int wq_run(const WqPlan& plan, const __half* xp, int64_t batch, const uint32_t* qweight,
           const __half* scales, const uint8_t* qzeros, int64_t m, int64_t d, int64_t gsz, float* y,
           int64_t split_stride, cudaStream_t st);

// Element i of the reordered activations (see gather_cols_kernel)
__device__ __forceinline__ __half wq_gathered(const __half* __restrict__ x,
                                              const int32_t* __restrict__ perm, int64_t i, int64_t d)
{
    const int64_t b = i / d, k = i - b * d;
    const int e = int(k & 7);
    const int64_t ks = (k & ~int64_t(7)) + ((e & 1) ? 4 + (e >> 1) : (e >> 1));
    const int32_t pk = perm ? perm[ks] : int32_t(ks);
    if (pk >= 0 && pk < d) return x[b * d + pk];
    atomicCAS(&g_device_status, 0, kErrIndex);       // not followed: zero and record
    return __ushort_as_half(0);
}

}  // namespace gptq
