// Root-mean-square norm of a residual sum, and its backward
// (ddp_rms_norm, ddp_rms_norm_grad).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "host.h"
#include "row_device.h"
#include "rows.h"

using namespace ddp_detail;

namespace {

constexpr int kI8 = 2;
constexpr int kE4M3 = 3;

constexpr int kNormThreads = 256;

struct NormArgs {
    RowPtrs x, res, sum, y;
    VecPtrs scale;
    int64_t rows[DDP_MAX_RANKS];
    const char *weight;
    int64_t width;
    int wdt;
    float eps;
};

// s of element j: the residual added in f32 and rounded to the dtype.
template <int DT, bool RES>
__device__ __forceinline__ float sum_elem(const char *x, const char *res, int64_t j)
{
    float s = load_elem<DT>(x, j);
    if (RES) {
        s = s + load_elem<DT>(res, j);
        if (DT == kBF16) s = widen_bf16(bf16_rne(s));
    }
    return s;
}

// One value in 8 bits: q within [-top, top] but for its rounding (a NaN row
// has codes of no meaning).
template <int YT>
__device__ __forceinline__ uint8_t code_of(float q)
{
    if (YT == kI8) {
        q = fminf(fmaxf(rintf(q), -127.0f), 127.0f);
        return (uint8_t)(int8_t)(int)q;
    }
    q = fminf(fmaxf(q, -448.0f), 448.0f);
    return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false) & 0xff);
}

// scale = most / top and the factor of the codes, top / most.  For a row so
// small that top / most would overflow, both products go through an exact
// power of two: code = (y * up) * inv.
struct Quant {
    float scale, up, inv;
};
template <int YT>
__device__ __forceinline__ Quant quant_of(float most)
{
    const float top = YT == kI8 ? 127.0f : 448.0f;
    Quant q;
    q.scale = most / top;
    q.up = most < 0x1p-100f ? 0x1p100f : 1.0f;
    q.inv = most == 0.0f ? 0.0f : top / (most * q.up);
    return q;
}

template <int DT, int YT, bool RES>
__global__ void __launch_bounds__(kNormThreads) norm_rows(NormArgs a)
{
    __shared__ float lds[kNormThreads / kWave];
    constexpr int waves = kNormThreads / kWave;
    const int r = blockIdx.y;
    const int64_t W = a.width;
    for (int64_t row = blockIdx.x; row < a.rows[r]; row += gridDim.x) {
        const char *x = a.x.p[r] + row * a.x.pitch;
        const char *res = RES ? a.res.p[r] + row * a.res.pitch : nullptr;
        char *sum = a.sum.p[r] ? a.sum.p[r] + row * a.sum.pitch : nullptr;
        char *y = a.y.p[r] + row * a.y.pitch;
        float ss = 0.0f;
        for (int64_t j = threadIdx.x; j < W; j += kNormThreads) {
            const float s = sum_elem<DT, RES>(x, res, j);
            if (sum) store_elem<DT>(sum, j, s);
            ss += s * s;
        }
        ss = block_all<OpSum>(ss, lds, waves);
        const float rho = 1.0f / sqrtf(ss / (float)W + a.eps);
        // sum_out may be x or the residual, so s is read back where it was stored
        auto y_at = [&](int64_t j) {
            const float s = sum ? load_elem<DT>(sum, j) : sum_elem<DT, RES>(x, res, j);
            return s * rho * (a.weight ? load_as(a.weight, j, a.wdt) : 1.0f);
        };
        if constexpr (YT == kI8 || YT == kE4M3) {
            float most = 0.0f;
            for (int64_t j = threadIdx.x; j < W; j += kNormThreads)
                most = OpMaxAbs::of(most, fabsf(y_at(j)));
            most = block_all<OpMaxAbs>(most, lds, waves);
            const Quant q = quant_of<YT>(most);
            if (threadIdx.x == 0) st_elem<float>(a.scale.p[r], row, q.scale);
            for (int64_t j = threadIdx.x; j < W; j += kNormThreads)
                st_elem<uint8_t>(y, j, code_of<YT>(y_at(j) * q.up * q.inv));
        } else {
            for (int64_t j = threadIdx.x; j < W; j += kNormThreads) store_elem<YT>(y, j, y_at(j));
        }
    }
}

// ---------------------------------------------------------------- backward

struct NormGradArgs {
    RowPtrs s, dy, dsum, dx;
    int64_t rows[DDP_MAX_RANKS];
    const char *weight;
    float *part;        // [n_ranks][blocks][width] partial weight gradients, or null
    int64_t width;
    int wdt;
    float eps;
};

template <int DT, int YT>
__global__ void __launch_bounds__(kNormThreads) norm_grad_rows(NormGradArgs a)
{
    __shared__ float lds[kNormThreads / kWave];
    constexpr int waves = kNormThreads / kWave;
    const int r = blockIdx.y;
    const int64_t W = a.width;
    float *part = a.part ? a.part + ((int64_t)r * gridDim.x + blockIdx.x) * W : nullptr;
    if (part)
        for (int64_t j = threadIdx.x; j < W; j += kNormThreads) part[j] = 0.0f;
    for (int64_t row = blockIdx.x; row < a.rows[r]; row += gridDim.x) {
        const char *s = a.s.p[r] + row * a.s.pitch;
        const char *dy = a.dy.p[r] + row * a.dy.pitch;
        const char *ds = a.dsum.p[r] ? a.dsum.p[r] + row * a.dsum.pitch : nullptr;
        char *dx = a.dx.p[r] + row * a.dx.pitch;
        float ss = 0.0f, gs = 0.0f;
        for (int64_t j = threadIdx.x; j < W; j += kNormThreads) {
            const float v = load_elem<DT>(s, j);
            const float g = load_elem<YT>(dy, j) * (a.weight ? load_as(a.weight, j, a.wdt) : 1.0f);
            ss += v * v;
            gs += g * v;
        }
        ss = block_all<OpSum>(ss, lds, waves);
        gs = block_all<OpSum>(gs, lds, waves);
        const float rho = 1.0f / sqrtf(ss / (float)W + a.eps);
        const float c = rho * rho * (gs / (float)W);
        for (int64_t j = threadIdx.x; j < W; j += kNormThreads) {
            const float v = load_elem<DT>(s, j), d = load_elem<YT>(dy, j);
            const float g = d * (a.weight ? load_as(a.weight, j, a.wdt) : 1.0f);
            float o = rho * (g - v * c);
            if (ds) o = load_elem<DT>(ds, j) + o;
            store_elem<DT>(dx, j, o);
            if (part) part[j] += d * v * rho;
        }
    }
}

struct DwArgs {
    VecPtrs dw;
    int64_t width;
    int64_t parts;
    const float *part;
    int dt, accumulate;
};

__global__ void __launch_bounds__(kNormThreads) norm_grad_weight(DwArgs a, int64_t first_block)
{
    const int r = blockIdx.y;
    const int64_t j = (first_block + blockIdx.x) * kNormThreads + threadIdx.x;
    if (j >= a.width) return;
    const float *p = a.part + (int64_t)r * a.parts * a.width + j;
    float t = 0.0f;
    for (int64_t b = 0; b < a.parts; ++b) t += p[b * a.width];
    char *dw = a.dw.p[r];
    if (a.dt == kF32)
        store_elem<kF32>(dw, j, a.accumulate ? load_elem<kF32>(dw, j) + t : t);
    else
        store_elem<kBF16>(dw, j, a.accumulate ? load_elem<kBF16>(dw, j) + t : t);
}

// Blocks of each rank in the backward, each with its own partial weight
// gradient.
int64_t grad_blocks(int64_t most, int32_t n_ranks)
{
    return std::max<int64_t>(1, std::min<int64_t>(most, std::max(1, 512 / n_ranks)));
}

int dtype_bytes(int dt) { return dt == DDP_F32 ? 4 : dt == DDP_BF16 ? 2 : 1; }
bool eight(int dt) { return dt == DDP_I8 || dt == DDP_E4M3; }

bool eps_ok(float eps) { return eps >= 0.0f && std::isfinite(eps); }

template <int DT, int YT>
void launch_norm(const NormArgs &a, bool res, dim3 g, hipStream_t st)
{
    if (res)
        norm_rows<DT, YT, true><<<g, kNormThreads, 0, st>>>(a);
    else
        norm_rows<DT, YT, false><<<g, kNormThreads, 0, st>>>(a);
}

constexpr int64_t kMostGridRows = 1 << 16;   // rows of a grid; blocks step through the rest

}  // namespace

extern "C" {

ddp_status_t ddp_rms_norm(const int64_t *rows, int32_t n_ranks, int64_t width, const ddp_rows_t *x,
                          const ddp_rows_t *residual, ddp_dtype_t dtype, const void *weight,
                          ddp_dtype_t weight_dtype, float eps, const ddp_rows_t *sum_out,
                          const ddp_rows_t *y, ddp_dtype_t y_dtype, float *const *scale, void *stream)
{
    int64_t total, most;
    ddp_status_t st = check_shape(rows, n_ranks, width, &total, &most);
    if (st != DDP_OK) return st;
    if (!dtype_ok(dtype) || (weight && !dtype_ok(weight_dtype)) || !eps_ok(eps) ||
        !(dtype_ok(y_dtype) || eight(y_dtype)))
        return DDP_ERR_INVALID_ARG;
    if (!eight(y_dtype) && !pair_ok(dtype, y_dtype)) return DDP_ERR_UNSUPPORTED;
    if (!eight(y_dtype) && scale) return DDP_ERR_INVALID_ARG;
    if (total == 0) return DDP_OK;
    if (!x || !x->rank || !y || !y->rank || (residual && !residual->rank) ||
        (sum_out && !sum_out->rank) || (eight(y_dtype) && !scale))
        return DDP_ERR_INVALID_ARG;
    const int esz = dtype_size(dtype), ysz = dtype_bytes(y_dtype);
    Operand op[kMaxOperands];
    int n = 0;
    op[n++] = rows_operand(x, rows, width, esz, false, true);
    op[n++] = rows_operand(y, rows, width, ysz, true, false);
    if (residual) op[n++] = rows_operand(residual, rows, width, esz, false, true);
    if (sum_out) op[n++] = rows_operand(sum_out, rows, width, esz, true, false);
    if (weight) op[n++] = span_operand(weight, width, dtype_size(weight_dtype), false);
    if (scale)
        op[n++] = vector_operand(reinterpret_cast<const void *const *>(scale), rows, 1, 4, true);
    if ((st = check_operands(op, n, n_ranks)) != DDP_OK) return st;
    NormArgs a;
    std::memset(&a, 0, sizeof(a));
    set_rows(&a.x, x, n_ranks, esz);
    set_rows(&a.res, residual, n_ranks, esz);
    set_rows(&a.sum, sum_out, n_ranks, esz);
    set_rows(&a.y, y, n_ranks, ysz);
    set_vecs(&a.scale, reinterpret_cast<const void *const *>(scale), n_ranks);
    std::memcpy(a.rows, rows, sizeof(int64_t) * (size_t)n_ranks);
    a.weight = static_cast<const char *>(weight);
    a.wdt = weight_dtype;
    a.width = width;
    a.eps = eps;
    const dim3 g((unsigned)std::min(most, kMostGridRows), (unsigned)n_ranks);
    hipStream_t hs = static_cast<hipStream_t>(stream);
    const bool res = residual != nullptr;
    if (dtype == DDP_F32) {
        if (y_dtype == DDP_F32) launch_norm<kF32, kF32>(a, res, g, hs);
        else if (y_dtype == DDP_BF16) launch_norm<kF32, kBF16>(a, res, g, hs);
        else if (y_dtype == DDP_I8) launch_norm<kF32, kI8>(a, res, g, hs);
        else launch_norm<kF32, kE4M3>(a, res, g, hs);
    } else {
        if (y_dtype == DDP_BF16) launch_norm<kBF16, kBF16>(a, res, g, hs);
        else if (y_dtype == DDP_I8) launch_norm<kBF16, kI8>(a, res, g, hs);
        else launch_norm<kBF16, kE4M3>(a, res, g, hs);
    }
    return launched("norm kernel launch");
}

int64_t ddp_rms_norm_grad_workspace(const int64_t *rows, int32_t n_ranks, int64_t width)
{
    int64_t total, most;
    if (check_shape(rows, n_ranks, width, &total, &most) != DDP_OK) return -1;
    return (int64_t)sizeof(float) * n_ranks * grad_blocks(most, n_ranks) * width;
}

ddp_status_t ddp_rms_norm_grad(const int64_t *rows, int32_t n_ranks, int64_t width,
                               const ddp_rows_t *s, ddp_dtype_t dtype, const void *weight,
                               ddp_dtype_t weight_dtype, float eps, const ddp_rows_t *dy,
                               ddp_dtype_t dy_dtype, const ddp_rows_t *dsum, const ddp_rows_t *dx,
                               void *const *dweight, ddp_dtype_t dweight_dtype, int32_t accumulate,
                               void *workspace, int64_t workspace_bytes, void *stream)
{
    int64_t total, most;
    ddp_status_t st = check_shape(rows, n_ranks, width, &total, &most);
    if (st != DDP_OK) return st;
    if (!dtype_ok(dtype) || (weight && !dtype_ok(weight_dtype)) || !dtype_ok(dy_dtype) ||
        (dweight && !dtype_ok(dweight_dtype)) || !eps_ok(eps))
        return DDP_ERR_INVALID_ARG;
    if (!pair_ok(dtype, dy_dtype)) return DDP_ERR_UNSUPPORTED;
    if (total == 0 && !dweight) return DDP_OK;
    if (total > 0 && (!s || !s->rank || !dy || !dy->rank || !dx || !dx->rank ||
                      (dsum && !dsum->rank)))
        return DDP_ERR_INVALID_ARG;
    const int esz = dtype_size(dtype), ysz = dtype_size(dy_dtype);
    const int64_t blocks = grad_blocks(most, n_ranks);
    const int64_t need = ddp_rms_norm_grad_workspace(rows, n_ranks, width);
    if (dweight) {
        if (!workspace || !aligned(workspace, 16)) return DDP_ERR_INVALID_ARG;
        if (workspace_bytes < need) return DDP_ERR_CAPACITY;
    }
    Operand op[kMaxOperands];
    int n = 0;
    if (total > 0) {
        op[n++] = rows_operand(s, rows, width, esz, false, true);
        op[n++] = rows_operand(dy, rows, width, ysz, false, true);
        if (dsum) op[n++] = rows_operand(dsum, rows, width, esz, false, true);
        op[n++] = rows_operand(dx, rows, width, esz, true, false);
        if (weight) op[n++] = span_operand(weight, width, dtype_size(weight_dtype), false);
    }
    if (dweight) {
        op[n++] = vector_operand(dweight, nullptr, width, dtype_size(dweight_dtype), true);
        op[n++] = span_operand(workspace, need, 1, true);
    }
    if ((st = check_operands(op, n, n_ranks)) != DDP_OK) return st;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    NormGradArgs a;
    std::memset(&a, 0, sizeof(a));
    set_rows(&a.s, total > 0 ? s : nullptr, n_ranks, esz);
    set_rows(&a.dy, total > 0 ? dy : nullptr, n_ranks, ysz);
    set_rows(&a.dsum, total > 0 ? dsum : nullptr, n_ranks, esz);
    set_rows(&a.dx, total > 0 ? dx : nullptr, n_ranks, esz);
    std::memcpy(a.rows, rows, sizeof(int64_t) * (size_t)n_ranks);
    a.weight = static_cast<const char *>(weight);
    a.wdt = weight_dtype;
    a.part = dweight ? static_cast<float *>(workspace) : nullptr;
    a.width = width;
    a.eps = eps;
    const dim3 g((unsigned)blocks, (unsigned)n_ranks);
    if (dtype == DDP_BF16)
        norm_grad_rows<kBF16, kBF16><<<g, kNormThreads, 0, hs>>>(a);
    else if (dy_dtype == DDP_F32)
        norm_grad_rows<kF32, kF32><<<g, kNormThreads, 0, hs>>>(a);
    else
        norm_grad_rows<kF32, kBF16><<<g, kNormThreads, 0, hs>>>(a);
    if ((st = launched("norm gradient kernel launch")) != DDP_OK || !dweight) return st;
    DwArgs w;
    std::memset(&w, 0, sizeof(w));
    set_vecs(&w.dw, dweight, n_ranks);
    w.width = width;
    w.parts = blocks;
    w.part = a.part;
    w.dt = dweight_dtype;
    w.accumulate = accumulate != 0;
    return launch_split((width + kNormThreads - 1) / kNormThreads, kNormThreads,
                        "weight gradient kernel launch", [&](int64_t b0, unsigned nb) {
                            norm_grad_weight<<<dim3(nb, (unsigned)n_ranks), kNormThreads, 0, hs>>>(w, b0);
                        });
}

}  // extern "C"
