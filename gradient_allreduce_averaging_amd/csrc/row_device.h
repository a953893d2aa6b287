// Device-side building blocks of the kernels over rows of tokens (norm.hip,
// distill.hip): the operands' addresses, wave and block reductions.  Not part
// of the ABI.
#pragma once

#include "device.h"

namespace ddp_detail {

// One matrix operand of every rank; null addresses where it is absent.
struct RowPtrs {
    char *p[DDP_MAX_RANKS];
    int64_t pitch;   // bytes from row to row
};

struct VecPtrs {
    char *p[DDP_MAX_RANKS];
};

inline void set_rows(RowPtrs *d, const ddp_rows_t *m, int32_t n, int esz)
{
    d->pitch = m ? m->stride * esz : 0;
    for (int r = 0; r < n; ++r) d->p[r] = m ? static_cast<char *>(m->rank[r]) : nullptr;
}

inline void set_vecs(VecPtrs *d, const void *const *v, int32_t n)
{
    for (int r = 0; r < n; ++r)
        d->p[r] = v ? static_cast<char *>(const_cast<void *>(v[r])) : nullptr;
}

constexpr int kWave = 64;

struct OpSum {
    static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
// The larger of two non-negative floats by their bits, so that a NaN (sign
// cleared) beats every number.
struct OpMaxAbs {
    static __device__ __forceinline__ float of(float a, float b)
    {
        return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
    }
};
struct OpMax {
    static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); }
};

// Every lane gets the whole wave's value; the tree is the same for each lane,
// and the operations commute, so all lanes hold the same bits.
template <class Op>
__device__ __forceinline__ float wave_all(float x)
{
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) x = Op::of(x, __shfl_xor(x, d, kWave));
    return x;
}

// Every thread of a block of `waves` waves gets the block's value.  `lds`
// holds `waves` floats; the first barrier lets an earlier use of it end.
template <class Op>
__device__ __forceinline__ float block_all(float x, float *lds, int waves)
{
    x = wave_all<Op>(x);
    if (waves == 1) return x;
    __syncthreads();
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = x;
    __syncthreads();
    float y = lds[0];
    for (int w = 1; w < waves; ++w) y = Op::of(y, lds[w]);
    return y;
}

__device__ __forceinline__ float load_as(const char *p, int64_t i, int dt)
{
    return dt == kF32 ? ld_elem<float>(p, i) : widen_bf16(ld_elem<uint16_t>(p, i));
}

}  // namespace ddp_detail
