// Distillation from a teacher's top logits, forward and backward
// (ddp_distill_loss, ddp_distill_grad).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "host.h"
#include "row_device.h"
#include "rows.h"

using namespace ddp_detail;

namespace {

constexpr int kDistillThreads = 256;

struct DistillArgs {
    RowPtrs z, teacher, index, dz;
    VecPtrs weight, row_loss;
    int64_t rows[DDP_MAX_RANKS];
    int64_t first[DDP_MAX_RANKS];   // tokens of the ranks before
    int64_t vocab;
    int32_t n_ranks, top;
    int tdt, index_bytes;
    float tau, scale;               // scale: grad_scale * n_ranks * tau
    float *den;                     // D
    float *w;                       // [tokens] the weight of each live token, 0 for others
    float *loss_of;                 // [tokens] row_loss
    float *loss;
};

// The vocabulary index of a token's entry k, or -1 where the entry is not
// live, and its logit.
__device__ __forceinline__ int64_t entry_of(const DistillArgs &a, int r, int64_t row, int k, float *t)
{
    const char *ip = a.index.p[r] + row * a.index.pitch;
    const int64_t j = a.index_bytes == 4 ? (int64_t)ld_elem<int32_t>(ip, k) : ld_elem<int64_t>(ip, k);
    if (j < 0 || j >= a.vocab) return -1;
    *t = load_as(a.teacher.p[r] + row * a.teacher.pitch, k, a.tdt);
    return *t == -INFINITY ? -1 : j;
}

__device__ __forceinline__ float weight_of(const DistillArgs &a, int r, int64_t row)
{
    if (!a.weight.p[r]) return 1.0f;
    const float w = ld_elem<float>(a.weight.p[r], row);
    return w > 0.0f ? w : 0.0f;
}

// w of every token (one thread each): 0 unless the token is live.
__global__ void __launch_bounds__(kDistillThreads) distill_weights(DistillArgs a)
{
    const int r = blockIdx.y;
    for (int64_t row = (int64_t)blockIdx.x * kDistillThreads + threadIdx.x; row < a.rows[r];
         row += (int64_t)gridDim.x * kDistillThreads) {
        float w = weight_of(a, r, row);
        if (w > 0.0f) {
            bool live = false;
            float t;
            for (int k = 0; k < a.top && !live; ++k) live = entry_of(a, r, row, k, &t) >= 0;
            if (!live) w = 0.0f;
        }
        a.w[a.first[r] + row] = w;
    }
}

// den = sum of w; with the losses of the tokens also loss = sum of w * row_loss / den.
__global__ void __launch_bounds__(kDistillThreads) distill_total(DistillArgs a, int64_t tokens,
                                                                 int with_loss)
{
    __shared__ float lds[kDistillThreads / kWave];
    float d = 0.0f, l = 0.0f;
    for (int64_t i = threadIdx.x; i < tokens; i += kDistillThreads) {
        const float w = a.w[i];
        d += w;
        if (with_loss && w > 0.0f) l += w * a.loss_of[i];
    }
    d = block_all<OpSum>(d, lds, kDistillThreads / kWave);
    l = block_all<OpSum>(l, lds, kDistillThreads / kWave);
    if (threadIdx.x == 0) {
        if (with_loss) *a.loss = d > 0.0f ? l / d : 0.0f;
        *a.den = d;
    }
}

template <int DT, bool GRAD>
__global__ void __launch_bounds__(kDistillThreads) distill_rows(DistillArgs a)
{
    __shared__ float lds[kDistillThreads / kWave];
    __shared__ float prob[DDP_MAX_TOP], zsel[DDP_MAX_TOP];
    __shared__ int64_t at[DDP_MAX_TOP];
    constexpr int waves = kDistillThreads / kWave;
    const int r = blockIdx.y, tid = threadIdx.x;
    const int64_t V = a.vocab;
    const float inv_tau = 1.0f / a.tau;
    for (int64_t row = blockIdx.x; row < a.rows[r]; row += gridDim.x) {
        const char *z = a.z.p[r] + row * a.z.pitch;
        char *dz = GRAD ? a.dz.p[r] + row * a.dz.pitch : nullptr;
        const int64_t token = a.first[r] + row;
        const float w = a.w[token];
        if (!(w > 0.0f)) {
            if (tid == 0) {
                a.loss_of[token] = 0.0f;
                if (a.row_loss.p[r]) st_elem<float>(a.row_loss.p[r], row, 0.0f);
            }
            if (GRAD)
                for (int64_t j = tid; j < V; j += kDistillThreads) store_elem<DT>(dz, j, 0.0f);
            continue;
        }
        float m = -INFINITY;
        for (int64_t j = tid; j < V; j += kDistillThreads) m = fmaxf(m, load_elem<DT>(z, j));
        m = block_all<OpMax>(m, lds, waves);
        float sum = 0.0f;
        for (int64_t j = tid; j < V; j += kDistillThreads)
            sum += expf((load_elem<DT>(z, j) - m) * inv_tau);
        sum = block_all<OpSum>(sum, lds, waves);
        // the teacher
        float tm = -INFINITY;
        __syncthreads();
        for (int k = tid; k < a.top; k += kDistillThreads) {
            float t = 0.0f;
            const int64_t j = entry_of(a, r, row, k, &t);
            at[k] = j;
            prob[k] = t;
            if (j >= 0) {
                tm = fmaxf(tm, t);
                zsel[k] = load_elem<DT>(z, j);
            }
        }
        tm = block_all<OpMax>(tm, lds, waves);
        float mass = 0.0f;
        for (int k = tid; k < a.top; k += kDistillThreads)
            if (at[k] >= 0) mass += expf((prob[k] - tm) * inv_tau);
        mass = block_all<OpSum>(mass, lds, waves);
        const float lmass = logf(mass), lsum = logf(sum);
        float kl = 0.0f;
        for (int k = tid; k < a.top; k += kDistillThreads) {
            if (at[k] < 0) continue;
            const float lp = (prob[k] - tm) * inv_tau - lmass;
            const float p = expf((prob[k] - tm) * inv_tau) / mass;
            if (p > 0.0f) kl += p * (lp - ((zsel[k] - m) * inv_tau - lsum));
            prob[k] = p;
        }
        kl = block_all<OpSum>(kl, lds, waves);
        const float loss = a.tau * a.tau * kl;
        if (tid == 0) {
            a.loss_of[token] = loss;
            if (a.row_loss.p[r]) st_elem<float>(a.row_loss.p[r], row, loss);
        }
        if (!GRAD) continue;
        const float c = a.scale * (w / *a.den), inv_sum = 1.0f / sum;
        for (int64_t j = tid; j < V; j += kDistillThreads)
            store_elem<DT>(dz, j, c * (expf((load_elem<DT>(z, j) - m) * inv_tau) * inv_sum));
        __syncthreads();   // the entries' places are written again below
        for (int k = tid; k < a.top; k += kDistillThreads) {
            if (at[k] < 0) continue;
            float p = 0.0f;
            for (int i = 0; i < a.top; ++i)
                if (at[i] == at[k]) p += prob[i];
            store_elem<DT>(dz, at[k], c * (expf((zsel[k] - m) * inv_tau) * inv_sum - p));
        }
        __syncthreads();   // prob, zsel and at are used again
    }
}

int64_t distill_bytes(int64_t total) { return 16 + (2 * total * 4 + 15) / 16 * 16; }

constexpr int64_t kMostGridRows = 1 << 16;

ddp_status_t run_distill(bool grad, const int64_t *rows, int32_t n_ranks, int64_t vocab,
                         const ddp_rows_t *logits, int dtype, int32_t top, const ddp_rows_t *teacher,
                         int teacher_dtype, const ddp_rows_t *index, int32_t index_bytes,
                         const float *const *token_weight, float temperature, float grad_scale,
                         const ddp_rows_t *dlogits, float *loss, float *const *row_loss,
                         void *workspace, int64_t workspace_bytes, void *stream)
{
    int64_t total, most;
    ddp_status_t st = check_shape(rows, n_ranks, vocab, &total, &most);
    if (st != DDP_OK) return st;
    if (!dtype_ok(dtype) || !dtype_ok(teacher_dtype) || top < 1 ||
        (index_bytes != 4 && index_bytes != 8) || !(temperature > 0.0f) ||
        !std::isfinite(temperature) || !loss)
        return DDP_ERR_INVALID_ARG;
    if (top > DDP_MAX_TOP) return DDP_ERR_UNSUPPORTED;
    if (total > 0 && (!logits || !logits->rank || !teacher || !teacher->rank || !index ||
                      !index->rank || (grad && (!dlogits || !dlogits->rank))))
        return DDP_ERR_INVALID_ARG;
    const int64_t need = distill_bytes(total);
    if (!workspace || !aligned(workspace, 16)) return DDP_ERR_INVALID_ARG;
    if (workspace_bytes < need) return DDP_ERR_CAPACITY;
    const int esz = dtype_size(dtype), tsz = dtype_size(teacher_dtype);
    Operand op[kMaxOperands];
    int n = 0;
    if (total > 0) {
        op[n++] = rows_operand(logits, rows, vocab, esz, false, true);
        op[n++] = rows_operand(teacher, rows, top, tsz, false, false);
        op[n++] = rows_operand(index, rows, top, index_bytes, false, false);
        if (grad) op[n++] = rows_operand(dlogits, rows, vocab, esz, true, false);
        if (token_weight)
            op[n++] = vector_operand(reinterpret_cast<const void *const *>(token_weight), rows, 1, 4,
                                     false);
        if (row_loss)
            op[n++] = vector_operand(reinterpret_cast<const void *const *>(row_loss), rows, 1, 4, true);
    }
    op[n++] = span_operand(loss, 1, 4, true);
    op[n++] = span_operand(workspace, need, 1, true);
    if ((st = check_operands(op, n, n_ranks)) != DDP_OK) return st;
    DistillArgs a;
    std::memset(&a, 0, sizeof(a));
    if (total > 0) {
        set_rows(&a.z, logits, n_ranks, esz);
        set_rows(&a.teacher, teacher, n_ranks, tsz);
        set_rows(&a.index, index, n_ranks, index_bytes);
        set_rows(&a.dz, grad ? dlogits : nullptr, n_ranks, esz);
        set_vecs(&a.weight, reinterpret_cast<const void *const *>(token_weight), n_ranks);
        set_vecs(&a.row_loss, reinterpret_cast<const void *const *>(row_loss), n_ranks);
    }
    std::memcpy(a.rows, rows, sizeof(int64_t) * (size_t)n_ranks);
    for (int r = 1; r < n_ranks; ++r) a.first[r] = a.first[r - 1] + rows[r - 1];
    a.vocab = vocab;
    a.n_ranks = n_ranks;
    a.top = top;
    a.tdt = teacher_dtype;
    a.index_bytes = index_bytes;
    a.tau = temperature;
    a.scale = grad_scale * (float)n_ranks * temperature;
    a.den = static_cast<float *>(workspace);
    a.w = a.den + 4;
    a.loss_of = a.w + total;
    a.loss = loss;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    if (total > 0) {
        const int64_t wb = std::min<int64_t>((most + kDistillThreads - 1) / kDistillThreads, 256);
        distill_weights<<<dim3((unsigned)wb, (unsigned)n_ranks), kDistillThreads, 0, hs>>>(a);
        if ((st = launched("distillation weight kernel launch")) != DDP_OK) return st;
        if (grad) {
            distill_total<<<1, kDistillThreads, 0, hs>>>(a, total, 0);
            if ((st = launched("distillation total kernel launch")) != DDP_OK) return st;
        }
        const dim3 g((unsigned)std::min(most, kMostGridRows), (unsigned)n_ranks);
        if (dtype == DDP_F32) {
            if (grad) distill_rows<kF32, true><<<g, kDistillThreads, 0, hs>>>(a);
            else distill_rows<kF32, false><<<g, kDistillThreads, 0, hs>>>(a);
        } else {
            if (grad) distill_rows<kBF16, true><<<g, kDistillThreads, 0, hs>>>(a);
            else distill_rows<kBF16, false><<<g, kDistillThreads, 0, hs>>>(a);
        }
        if ((st = launched("distillation kernel launch")) != DDP_OK) return st;
    }
    distill_total<<<1, kDistillThreads, 0, hs>>>(a, total, 1);
    return launched("distillation total kernel launch");
}

}  // namespace

extern "C" {

int64_t ddp_distill_workspace(const int64_t *rows, int32_t n_ranks, int64_t vocab)
{
    int64_t total, most;
    if (check_shape(rows, n_ranks, vocab, &total, &most) != DDP_OK) return -1;
    return distill_bytes(total);
}

ddp_status_t ddp_distill_loss(const int64_t *rows, int32_t n_ranks, int64_t vocab,
                              const ddp_rows_t *logits, ddp_dtype_t dtype, int32_t top,
                              const ddp_rows_t *teacher, ddp_dtype_t teacher_dtype,
                              const ddp_rows_t *index, int32_t index_bytes,
                              const float *const *token_weight, float temperature, float *loss,
                              float *const *row_loss, void *workspace, int64_t workspace_bytes,
                              void *stream)
{
    return run_distill(false, rows, n_ranks, vocab, logits, dtype, top, teacher, teacher_dtype, index,
                       index_bytes, token_weight, temperature, 1.0f, nullptr, loss, row_loss,
                       workspace, workspace_bytes, stream);
}

ddp_status_t ddp_distill_grad(const int64_t *rows, int32_t n_ranks, int64_t vocab,
                              const ddp_rows_t *logits, ddp_dtype_t dtype, int32_t top,
                              const ddp_rows_t *teacher, ddp_dtype_t teacher_dtype,
                              const ddp_rows_t *index, int32_t index_bytes,
                              const float *const *token_weight, float temperature,
                              float grad_scale, const ddp_rows_t *dlogits, float *loss,
                              float *const *row_loss, void *workspace, int64_t workspace_bytes,
                              void *stream)
{
    return run_distill(true, rows, n_ranks, vocab, logits, dtype, top, teacher, teacher_dtype, index,
                       index_bytes, token_weight, temperature, grad_scale, dlogits, loss, row_loss,
                       workspace, workspace_bytes, stream);
}

}  // extern "C"
