// train_api.cu -- the C ABI's entries for scoring, the losses and the LM heads in
// 8 and 4 bits (declared in include/sampler.h): argument checks and launches.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "handle.h"
#include "launch.h"
#include "sampler.h"

using dst::DeviceGuard;

namespace {

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

bool known(int dtype) { return dtype == SAMPLER_DTYPE_F32 || dtype == SAMPLER_DTYPE_BF16; }

size_t bytes_of(int dtype) { return dtype == SAMPLER_DTYPE_BF16 ? 2 : 4; }

cudaStream_t cuda_stream(sampler_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// need_tokens: the call cannot do without them (others: where out_logprob is asked for).
int check_rows(sampler_t h, const sampler_rows_t* a, bool need_tokens = true)
{
    if (!h || !a) return SAMPLER_ERR_NULL_ARG;
    if (a->n_rows < 0 || a->vocab < 1 || a->row_stride < a->vocab) return SAMPLER_ERR_BAD_SHAPE;
    if (!known(a->dtype)) return SAMPLER_ERR_BAD_DTYPE;
    if (a->n_rows > h->max_rows || a->n_rows > INT_MAX || a->vocab > h->max_vocab) return SAMPLER_ERR_TOO_LARGE;
    if (a->n_rows == 0) return SAMPLER_OK;
    if (!a->logits || (!a->tokens && (need_tokens || a->out_logprob))) return SAMPLER_ERR_NULL_ARG;
    const size_t es = bytes_of(a->dtype);
    if (!aligned(a->logits, es) || !aligned(a->tokens, 4) || !aligned(a->temperature, 4) || !aligned(a->weight, 4) ||
        !aligned(a->out_logprob, 4) || !aligned(a->out_entropy, 4) || !aligned(a->out_status, 4))
        return SAMPLER_ERR_BAD_SHAPE;
    if (a->out_grad && (a->grad_stride < a->vocab || !aligned(a->out_grad, es))) return SAMPLER_ERR_BAD_SHAPE;
    // in place is one value for one value
    if (a->out_grad == a->logits && a->grad_stride != a->row_stride) return SAMPLER_ERR_BAD_SHAPE;
    return SAMPLER_OK;
}

// The single loss of a call over no rows or no pairs.
int write_zero(float* out, cudaStream_t stream)
{
    return cudaMemsetAsync(out, 0, sizeof(float), stream) == cudaSuccess ? SAMPLER_OK : SAMPLER_ERR_CUDA;
}

int check_scaled(const sampler_scaled_head_t* g)
{
    if (!g || !g->hidden || !g->hidden_scale || !g->weight || !g->weight_scale) return SAMPLER_ERR_NULL_ARG;
    const int64_t K = g->hidden_dim;
    if (K < 1 || K > INT_MAX - 127) return SAMPLER_ERR_BAD_SHAPE;
    const int64_t groups = (K + 127) / 128;
    if (g->hidden_stride < K || g->weight_stride < K || g->hidden_stride % 16 != 0 || g->weight_stride % 16 != 0 ||
        g->hidden_scale_stride < groups || g->weight_scale_stride < groups || !aligned(g->hidden, 16) ||
        !aligned(g->weight, 16) || !aligned(g->hidden_scale, 4) || !aligned(g->weight_scale, 4))
        return SAMPLER_ERR_BAD_SHAPE;
    return SAMPLER_OK;
}

int launch_scaled(sampler_t h, const sampler_scaled_head_t* g, void* logits, int dtype, int64_t ldl, int64_t rows,
                  int64_t vocab, cudaStream_t stream)
{
    return dst::scaled_head_launch(*g, logits, dtype, ldl, rows, vocab, h->num_sms, h->wait_ns,
                                   h->stats + SAMPLER_STAT_LM_HEAD_TIMEOUTS, &h->head_grants, stream);
}

constexpr int64_t kMicroMaxCols = 1 << 24;

bool micro_block(int block) { return block == 16 || block == 32; }

int check_micro_head(const sampler_micro_head_t* g)
{
    if (!g || !g->hidden || !g->hidden_scale || !g->weight || !g->weight_scale) return SAMPLER_ERR_NULL_ARG;
    if (!micro_block(g->block)) return SAMPLER_ERR_BAD_VALUE;
    const int64_t bytes = (g->hidden_dim + 1) / 2;
    if (g->hidden_dim < 1 || g->hidden_dim > kMicroMaxCols || g->hidden_stride < bytes || g->weight_stride < bytes ||
        g->hidden_stride % 16 != 0 || g->weight_stride % 16 != 0 || !aligned(g->hidden, 16) || !aligned(g->weight, 16) ||
        !aligned(g->hidden_scale, 16) || !aligned(g->weight_scale, 16) || !aligned(g->hidden_row_scale, 4) ||
        !aligned(g->weight_row_scale, 4))
        return SAMPLER_ERR_BAD_SHAPE;
    return SAMPLER_OK;
}

int launch_micro(sampler_t h, const sampler_micro_head_t* g, void* logits, int dtype, int64_t ldl, int64_t rows,
                 int64_t vocab, cudaStream_t stream)
{
    return dst::micro_head_launch(*g, logits, dtype, ldl, rows, vocab, h->num_sms, h->wait_ns,
                                  h->stats + SAMPLER_STAT_LM_HEAD_TIMEOUTS, &h->micro_grants, stream);
}

}  // namespace

extern "C" {

int sampler_score(sampler_t h, const sampler_rows_t* rows, sampler_stream_t stream)
{
    const int rc = check_rows(h, rows);
    if (rc != SAMPLER_OK) return rc;
    if (rows->out_grad) return SAMPLER_ERR_UNSUPPORTED;
    if (rows->n_rows == 0) return SAMPLER_OK;
    DeviceGuard guard;
    if (cudaSetDevice(h->device) != cudaSuccess) return SAMPLER_ERR_CUDA;
    dst::LossParams p;
    std::memset(&p, 0, sizeof p);
    p.rows = *rows;
    p.mode = dst::kModeScore;
    p.ws = h->row_ws;
    p.wait_ns = h->wait_ns;
    return dst::rows_launch(p, h->num_sms, &h->row_occ, cuda_stream(stream));
}

int sampler_score_grad(sampler_t h, const sampler_rows_t* rows, const float* grad_logprob, const float* grad_entropy,
                       sampler_stream_t stream)
{
    const int rc = check_rows(h, rows);
    if (rc != SAMPLER_OK) return rc;
    if (rows->n_rows == 0) return SAMPLER_OK;
    if (!rows->out_grad || !grad_logprob) return SAMPLER_ERR_NULL_ARG;
    if (!aligned(grad_logprob, 4) || !aligned(grad_entropy, 4)) return SAMPLER_ERR_BAD_SHAPE;
    DeviceGuard guard;
    if (cudaSetDevice(h->device) != cudaSuccess) return SAMPLER_ERR_CUDA;
    dst::LossParams p;
    std::memset(&p, 0, sizeof p);
    p.rows = *rows;
    p.mode = dst::kModeScoreGrad;
    p.grad_logprob = grad_logprob;
    p.grad_entropy = grad_entropy;
    p.ws = h->row_ws;
    p.wait_ns = h->wait_ns;
    return dst::rows_launch(p, h->num_sms, &h->row_occ, cuda_stream(stream));
}

int sampler_policy_loss(sampler_t h, const sampler_rows_t* rows, const sampler_policy_t* q, sampler_stream_t stream)
{
    const int rc = check_rows(h, rows);
    if (rc != SAMPLER_OK) return rc;
    if (rows->n_rows > h->row_ws.rows) return SAMPLER_ERR_TOO_LARGE;
    if (!q || !q->out_loss) return SAMPLER_ERR_NULL_ARG;
    if (!(q->clip_low >= 0.f && q->clip_low <= 1.f) || !(q->clip_high >= 0.f) || !std::isfinite(q->clip_high) ||
        !std::isfinite(q->kl_coef) || !std::isfinite(q->entropy_coef) || !std::isfinite(q->grad_scale))
        return SAMPLER_ERR_BAD_VALUE;
    if (!q->ref_logprob && (q->kl_coef != 0.f || q->out_kl)) return SAMPLER_ERR_NULL_ARG;
    if (rows->n_rows > 0 && (!q->old_logprob || !q->advantage)) return SAMPLER_ERR_NULL_ARG;
    if (!aligned(q->old_logprob, 4) || !aligned(q->advantage, 4) || !aligned(q->ref_logprob, 4) ||
        !aligned(q->grad_scale_dev, 4) || !aligned(q->out_loss, 4) || !aligned(q->out_ratio, 4) ||
        !aligned(q->out_kl, 4))
        return SAMPLER_ERR_BAD_SHAPE;
    DeviceGuard guard;
    if (cudaSetDevice(h->device) != cudaSuccess) return SAMPLER_ERR_CUDA;
    if (rows->n_rows == 0) return write_zero(q->out_loss, cuda_stream(stream));
    dst::LossParams p;
    std::memset(&p, 0, sizeof p);
    p.rows = *rows;
    p.mode = dst::kModePolicy;
    p.policy = *q;
    p.ws = h->row_ws;
    p.wait_ns = h->wait_ns;
    return dst::rows_launch(p, h->num_sms, &h->row_occ, cuda_stream(stream));
}

int sampler_preference_loss(sampler_t h, const sampler_rows_t* rows, const sampler_preference_t* q,
                            sampler_stream_t stream)
{
    int rc = check_rows(h, rows);
    if (rc != SAMPLER_OK) return rc;
    if (rows->n_rows > h->row_ws.rows) return SAMPLER_ERR_TOO_LARGE;
    if (!q || !q->out_loss) return SAMPLER_ERR_NULL_ARG;
    if (rows->out_entropy) return SAMPLER_ERR_UNSUPPORTED;
    if (q->n_pairs < 0) return SAMPLER_ERR_BAD_SHAPE;
    if (q->n_pairs > h->row_ws.rows) return SAMPLER_ERR_TOO_LARGE;
    if (!std::isfinite(q->beta) || !std::isfinite(q->margin) || !std::isfinite(q->grad_scale) ||
        !(q->label_smoothing >= 0.f && q->label_smoothing <= 1.f))
        return SAMPLER_ERR_BAD_VALUE;
    if (q->n_pairs > 0 && !q->seq_offsets) return SAMPLER_ERR_NULL_ARG;
    if (!aligned(q->seq_offsets, 4) || !aligned(q->ref_logprob, 4) || !aligned(q->grad_scale_dev, 4) ||
        !aligned(q->out_loss, 4) || !aligned(q->out_reward, 4))
        return SAMPLER_ERR_BAD_SHAPE;
    DeviceGuard guard;
    if (cudaSetDevice(h->device) != cudaSuccess) return SAMPLER_ERR_CUDA;
    cudaStream_t s = cuda_stream(stream);
    if (rows->n_rows > 0) {
        dst::LossParams p;
        std::memset(&p, 0, sizeof p);
        p.rows = *rows;
        p.mode = dst::kModePairs;
        p.ws = h->row_ws;
        p.wait_ns = h->wait_ns;
        rc = dst::rows_launch(p, h->num_sms, &h->row_occ, s);
        if (rc != SAMPLER_OK) return rc;
    }
    rc = q->n_pairs > 0 ? dst::pairs_launch(*rows, *q, h->row_ws, s) : write_zero(q->out_loss, s);
    if (rc != SAMPLER_OK || !rows->out_grad || rows->n_rows == 0) return rc;
    return dst::pairs_grad_launch(*rows, h->row_ws, q->n_pairs > 0, s);
}

int sampler_score_top(sampler_t h, const sampler_rows_t* rows, const sampler_top_t* top, sampler_stream_t stream)
{
    const int rc = check_rows(h, rows, false);
    if (rc != SAMPLER_OK) return rc;
    if (!top) return SAMPLER_ERR_NULL_ARG;
    if (rows->out_grad) return SAMPLER_ERR_UNSUPPORTED;
    if (top->top_n < 1 || top->top_n > SAMPLER_MAX_ALTERNATIVES) return SAMPLER_ERR_BAD_VALUE;
    if (rows->n_rows == 0) return SAMPLER_OK;
    if (!top->out_top_ids || !top->out_top_logprobs) return SAMPLER_ERR_NULL_ARG;
    if (!aligned(top->out_top_ids, 4) || !aligned(top->out_top_logprobs, 4) || !aligned(top->out_rest_logprob, 4))
        return SAMPLER_ERR_BAD_SHAPE;
    DeviceGuard guard;
    if (cudaSetDevice(h->device) != cudaSuccess) return SAMPLER_ERR_CUDA;
    dst::TopParams p;
    std::memset(&p, 0, sizeof p);
    p.rows = *rows;
    p.top = *top;
    p.ws = h->top_ws;
    p.wait_ns = h->wait_ns;
    return dst::top_launch(p, h->num_sms, &h->top_grants, cuda_stream(stream));
}

int sampler_distill_loss(sampler_t h, const sampler_rows_t* rows, const sampler_distill_t* q, sampler_stream_t stream)
{
    const int rc = check_rows(h, rows, false);
    if (rc != SAMPLER_OK) return rc;
    if (rows->n_rows > h->row_ws.rows) return SAMPLER_ERR_TOO_LARGE;
    if (!q || !q->out_loss) return SAMPLER_ERR_NULL_ARG;
    if (rows->out_entropy) return SAMPLER_ERR_UNSUPPORTED;
    if (q->top_n < 1 || q->top_n > SAMPLER_MAX_ALTERNATIVES || !(q->token_coef >= 0.f) || !std::isfinite(q->token_coef) ||
        !std::isfinite(q->grad_scale))
        return SAMPLER_ERR_BAD_VALUE;
    if (rows->n_rows > 0 && (!q->teacher_ids || !q->teacher_logprobs || (q->token_coef != 0.f && !rows->tokens)))
        return SAMPLER_ERR_NULL_ARG;
    if (!aligned(q->teacher_ids, 4) || !aligned(q->teacher_logprobs, 4) || !aligned(q->teacher_rest, 4) ||
        !aligned(q->grad_scale_dev, 4) || !aligned(q->out_loss, 4) || !aligned(q->out_kl, 4))
        return SAMPLER_ERR_BAD_SHAPE;
    DeviceGuard guard;
    if (cudaSetDevice(h->device) != cudaSuccess) return SAMPLER_ERR_CUDA;
    if (rows->n_rows == 0) return write_zero(q->out_loss, cuda_stream(stream));
    dst::DistillParams p;
    std::memset(&p, 0, sizeof p);
    p.rows = *rows;
    p.distill = *q;
    p.ws = h->row_ws;
    p.wait_ns = h->wait_ns;
    return dst::distill_launch(p, h->num_sms, &h->distill_occ, cuda_stream(stream));
}

int sampler_quantize_blocks(sampler_t h, const sampler_quantize_t* q, sampler_stream_t stream)
{
    if (!h || !q) return SAMPLER_ERR_NULL_ARG;
    if (q->block_rows != 1 && q->block_rows != 128) return SAMPLER_ERR_BAD_VALUE;
    if (q->rows < 0 || q->rows > INT_MAX - 127 || q->cols < 1 || q->cols > INT_MAX - 127 || q->src_stride < q->cols ||
        q->values_stride < q->cols || q->scale_stride < (q->cols + 127) / 128)
        return SAMPLER_ERR_BAD_SHAPE;
    if (!known(q->dtype)) return SAMPLER_ERR_BAD_DTYPE;
    if (q->rows == 0) return SAMPLER_OK;
    if (!q->src || !q->values || !q->scales) return SAMPLER_ERR_NULL_ARG;
    if (!aligned(q->src, bytes_of(q->dtype)) || !aligned(q->scales, 4)) return SAMPLER_ERR_BAD_SHAPE;
    DeviceGuard guard;
    if (cudaSetDevice(h->device) != cudaSuccess) return SAMPLER_ERR_CUDA;
    return dst::quantize_launch(*q, h->num_sms, cuda_stream(stream));
}

int sampler_lm_head_scaled(sampler_t h, const sampler_scaled_head_t* lm, void* logits, int32_t dtype, int64_t ldl,
                           int64_t rows, int64_t vocab, sampler_stream_t stream)
{
    if (!h || !lm) return SAMPLER_ERR_NULL_ARG;
    if (!known(dtype)) return SAMPLER_ERR_BAD_DTYPE;
    if (rows < 0 || vocab < 1 || ldl < vocab || !aligned(logits, bytes_of(dtype))) return SAMPLER_ERR_BAD_SHAPE;
    if (rows > INT_MAX - 255 || vocab > h->max_vocab) return SAMPLER_ERR_TOO_LARGE;
    if (rows == 0) return SAMPLER_OK;
    if (!logits) return SAMPLER_ERR_NULL_ARG;
    const int rc = check_scaled(lm);
    if (rc != SAMPLER_OK) return rc;
    DeviceGuard guard;
    if (cudaSetDevice(h->device) != cudaSuccess) return SAMPLER_ERR_CUDA;
    return launch_scaled(h, lm, logits, dtype, ldl, rows, vocab, cuda_stream(stream));
}

int sampler_lm_head_scaled_sample(sampler_t h, const sampler_scaled_head_t* lm, const sampler_args_t* a,
                                  const sampler_ext_t* ext, sampler_stream_t stream)
{
    if (!h || !a || !lm) return SAMPLER_ERR_NULL_ARG;
    // the sampler's own checks, before anything is enqueued
    int rc = dst::sample_check(h, a, ext);
    if (rc != SAMPLER_OK || a->n_rows == 0) return rc;
    rc = check_scaled(lm);
    if (rc != SAMPLER_OK) return rc;
    const int64_t rows = a->n_logit_rows > 0 ? a->n_logit_rows : a->n_rows;
    if (rows > INT_MAX - 255) return SAMPLER_ERR_TOO_LARGE;
    if (!aligned(a->logits, bytes_of(a->dtype))) return SAMPLER_ERR_BAD_SHAPE;
    DeviceGuard guard;
    if (cudaSetDevice(h->device) != cudaSuccess) return SAMPLER_ERR_CUDA;
    rc = launch_scaled(h, lm, const_cast<void*>(a->logits), a->dtype, a->row_stride, rows, a->vocab,
                       cuda_stream(stream));
    if (rc != SAMPLER_OK) return rc;
    return dst::sample_launch(h, a, ext, true, cuda_stream(stream));
}

int64_t sampler_micro_scale_bytes(int64_t rows, int64_t cols, int32_t block)
{
    if (!micro_block(block) || rows < 0 || rows > INT_MAX - 127 || cols < 1 || cols > kMicroMaxCols) return -1;
    return (rows + 127) / 128 * (((cols + block - 1) / block + 3) / 4) * 512;
}

int sampler_quantize_micro(sampler_t h, const sampler_micro_t* q, sampler_stream_t stream)
{
    if (!h || !q) return SAMPLER_ERR_NULL_ARG;
    if (!micro_block(q->block)) return SAMPLER_ERR_BAD_VALUE;
    if (sampler_micro_scale_bytes(q->rows, q->cols, q->block) < 0 || q->src_stride < q->cols ||
        q->values_stride < (q->cols + 1) / 2)
        return SAMPLER_ERR_BAD_SHAPE;
    if (!known(q->dtype)) return SAMPLER_ERR_BAD_DTYPE;
    if (q->rows == 0) return SAMPLER_OK;
    if (!q->src || !q->values || !q->scales || !q->row_scale) return SAMPLER_ERR_NULL_ARG;
    if (!aligned(q->src, bytes_of(q->dtype)) || !aligned(q->scales, 16) || !aligned(q->row_scale, 4))
        return SAMPLER_ERR_BAD_SHAPE;
    DeviceGuard guard;
    if (cudaSetDevice(h->device) != cudaSuccess) return SAMPLER_ERR_CUDA;
    return dst::micro_quantize_launch(*q, h->num_sms, cuda_stream(stream));
}

int sampler_micro_rows(sampler_t h, const sampler_micro_rows_t* q, sampler_stream_t stream)
{
    if (!h || !q) return SAMPLER_ERR_NULL_ARG;
    if (!micro_block(q->block)) return SAMPLER_ERR_BAD_VALUE;
    if (sampler_micro_scale_bytes(q->rows, q->cols, q->block) < 0 || q->values_stride < (q->cols + 1) / 2 || q->n < 0 ||
        q->n > INT_MAX || q->out_stride < q->cols || (!q->ids && q->n > q->rows))
        return SAMPLER_ERR_BAD_SHAPE;
    if (!known(q->dtype)) return SAMPLER_ERR_BAD_DTYPE;
    if (q->n == 0) return SAMPLER_OK;
    if (!q->out || (q->rows > 0 && (!q->values || !q->scales))) return SAMPLER_ERR_NULL_ARG;
    if (!aligned(q->out, bytes_of(q->dtype)) || !aligned(q->scales, 16) || !aligned(q->row_scale, 4) || !aligned(q->ids, 4))
        return SAMPLER_ERR_BAD_SHAPE;
    DeviceGuard guard;
    if (cudaSetDevice(h->device) != cudaSuccess) return SAMPLER_ERR_CUDA;
    return dst::micro_rows_launch(*q, cuda_stream(stream));
}

int sampler_lm_head_micro(sampler_t h, const sampler_micro_head_t* lm, void* logits, int32_t dtype, int64_t ldl,
                          int64_t rows, int64_t vocab, sampler_stream_t stream)
{
    if (!h || !lm) return SAMPLER_ERR_NULL_ARG;
    if (!known(dtype)) return SAMPLER_ERR_BAD_DTYPE;
    if (rows < 0 || vocab < 1 || ldl < vocab || !aligned(logits, bytes_of(dtype))) return SAMPLER_ERR_BAD_SHAPE;
    if (rows > INT_MAX - 255 || vocab > h->max_vocab) return SAMPLER_ERR_TOO_LARGE;
    if (rows == 0) return SAMPLER_OK;
    if (!logits) return SAMPLER_ERR_NULL_ARG;
    const int rc = check_micro_head(lm);
    if (rc != SAMPLER_OK) return rc;
    DeviceGuard guard;
    if (cudaSetDevice(h->device) != cudaSuccess) return SAMPLER_ERR_CUDA;
    return launch_micro(h, lm, logits, dtype, ldl, rows, vocab, cuda_stream(stream));
}

int sampler_lm_head_micro_sample(sampler_t h, const sampler_micro_head_t* lm, const sampler_args_t* a,
                                 const sampler_ext_t* ext, sampler_stream_t stream)
{
    if (!h || !a || !lm) return SAMPLER_ERR_NULL_ARG;
    // the sampler's own checks, before anything is enqueued
    int rc = dst::sample_check(h, a, ext);
    if (rc != SAMPLER_OK || a->n_rows == 0) return rc;
    rc = check_micro_head(lm);
    if (rc != SAMPLER_OK) return rc;
    const int64_t rows = a->n_logit_rows > 0 ? a->n_logit_rows : a->n_rows;
    if (rows > INT_MAX - 255) return SAMPLER_ERR_TOO_LARGE;
    if (!aligned(a->logits, bytes_of(a->dtype))) return SAMPLER_ERR_BAD_SHAPE;
    DeviceGuard guard;
    if (cudaSetDevice(h->device) != cudaSuccess) return SAMPLER_ERR_CUDA;
    rc = launch_micro(h, lm, const_cast<void*>(a->logits), a->dtype, a->row_stride, rows, a->vocab, cuda_stream(stream));
    if (rc != SAMPLER_OK) return rc;
    return dst::sample_launch(h, a, ext, true, cuda_stream(stream));
}

}  // extern "C"
