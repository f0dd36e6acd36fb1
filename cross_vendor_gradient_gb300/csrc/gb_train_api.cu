// C entry points of the training-step operators (include/gb.h): argument
// checks, the tables of the many-tensor calls, launches.
#include <cmath>

#include "gb_internal.cuh"
#include "gb_rows.cuh"
#include "gb_train.cuh"

using namespace gbrt;

namespace {

gb_status check_train_dtype(gb_ctx *c, int d) {
    if (d != GB_F32 && d != GB_BF16 && d != GB_F16) return set_msg(c, GB_ERR_UNSUPPORTED_DTYPE, "dtype %d", d);
    return GB_OK;
}

gb_status check_align(gb_ctx *c, const void *p, size_t a, const char *name, int t = -1) {
    if (!p) return t < 0 ? set_msg(c, GB_ERR_INVALID_ARG, "%s is NULL", name)
                         : set_msg(c, GB_ERR_INVALID_ARG, "%s[%d] is NULL", name, t);
    if (((uintptr_t)p & (a - 1)) != 0)
        return t < 0 ? set_msg(c, GB_ERR_MISALIGNED, "%s not %zu-byte aligned", name, a)
                     : set_msg(c, GB_ERR_MISALIGNED, "%s[%d] not %zu-byte aligned", name, t, a);
    return GB_OK;
}

// Warp tiles of all tensors; they are counted in 32 bits.
gb_status check_tensors(gb_ctx *c, int n_tensors, const size_t *numel, uint64_t *elems) {
    *elems = 0;
    if (n_tensors < 0) return set_msg(c, GB_ERR_INVALID_ARG, "n_tensors = %d", n_tensors);
    if (n_tensors > 0 && !numel) return set_msg(c, GB_ERR_INVALID_ARG, "numel is NULL");
    for (int t = 0; t < n_tensors; ++t) {
        GB_TRY(check_n(c, numel[t]));
        *elems += numel[t];
        if (*elems > kMaxElems) return set_msg(c, GB_ERR_INVALID_ARG, "%d tensors hold too many elements", n_tensors);
    }
    return GB_OK;
}

// A call's use of the context's workspace: a ticket counter, zero between
// calls, and partial sums.
struct Work {
    unsigned long long capture = 0;  // id of the capture that the stream is in; 0: none
    uint32_t *ticket = nullptr;
    unsigned char *partials = nullptr;
};

// A call outside of captures is ordered after the previous call that used
// staging.  Captured calls have partial sums of their own, since their graph
// may run next to later calls; those of one capture are ordered after each
// other, also on parallel branches.  Each captured call has a ticket of its
// own: two graphs that ran at the same time, against the rule, would spoil
// each other's sums, but leave no count behind.
gb_status begin_work(gb_ctx *c, cudaStream_t s, Work *w) {
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    cudaError_t e = cudaStreamGetCaptureInfo(s, &st, &id);
    if (e == cudaErrorStreamCaptureImplicit) {  // nothing has been enqueued: the context stays sound
        cudaGetLastError();
        return set_msg(c, GB_ERR_INVALID_ARG, "the legacy stream, while a stream that synchronizes with it is being captured");
    }
    if (e != cudaSuccess) return fail(c, GB_ERR_CUDA, "cudaStreamGetCaptureInfo", e);
    if (st == cudaStreamCaptureStatusInvalidated) return set_msg(c, GB_ERR_INVALID_ARG, "the stream's capture has been invalidated");
    w->capture = st == cudaStreamCaptureStatusNone ? 0 : id;
    if (!c->work_ready) {
        if (w->capture) return set_msg(c, GB_ERR_INVALID_ARG, "the first call that needs the workspace is being captured");
        GB_TRY(grow_device(c, &c->d_work, &c->d_work_bytes, gb::kWorkHead + 2 * 4 * gb::kWorkFloats));
        if ((e = cudaEventCreateWithFlags(&c->work_done, cudaEventDisableTiming)) != cudaSuccess)
            return fail(c, GB_ERR_CUDA, "cudaEventCreate", e);
        // complete before any stream's call: graphs run on streams that are not known here
        if ((e = cudaMemsetAsync(c->d_work, 0, gb::kWorkHead, c->sg)) != cudaSuccess || (e = cudaStreamSynchronize(c->sg)) != cudaSuccess)
            return fail(c, GB_ERR_CUDA, "clearing the workspace", e);
        c->work_ready = true;
    }
    w->ticket = (uint32_t *)c->d_work;
    w->partials = c->d_work + gb::kWorkHead;
    if (!w->capture) return begin(c, s);
    w->ticket += 1 + c->work_tickets++ % (gb::kWorkHead / sizeof(uint32_t) - 1);
    w->partials += 4 * gb::kWorkFloats;
    if (c->work_capture == w->capture && c->work_stream != s) GB_TRY(wait_on(c, s, c->work_done));
    return GB_OK;
}
gb_status end_work(gb_ctx *c, cudaStream_t s, const Work &w) {
    if (!w.capture) return end(c, s);
    GB_TRY(record(c, c->work_done, s));
    c->work_capture = w.capture;
    c->work_stream = s;
    return GB_OK;
}

// Whether [a, a + na) and [b, b + nb) overlap without starting together.
bool cross(const void *a, size_t na, const void *b, size_t nb) {
    if (!a || !b || a == b) return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}
bool overlap(const void *a, size_t na, const void *b, size_t nb) { return a && (a == b || cross(a, na, b, nb)); }

// The launches of a norm, N tensors each.
template <int N>
gb_status norm_launches(gb_ctx *c, const Work &w, int n_tensors, const void *const *grads, const size_t *numel, gb_dtype dtype,
                        float max_norm, float *out, cudaStream_t s) {
    gb::NormArgs<N> a;
    a.ticket = w.ticket;
    a.partials = (double *)w.partials;
    a.out = out;
    a.max_norm = max_norm;
    uint32_t used = 0;
    int t = 0;
    do {
        a.n_tensors = 0;
        a.tiles = 0;
        for (; t < n_tensors && a.n_tensors < N; ++t) {
            if (!numel[t]) continue;
            a.grad[a.n_tensors] = grads[t];
            a.numel[a.n_tensors] = numel[t];
            a.shift[a.n_tensors] = (unsigned char)gb::vector_shift(grads[t], elem_bytes(dtype));
            a.tiles += (uint32_t)gb::tiles_of(numel[t], a.shift[a.n_tensors], gb::kNormTile);
            a.tile_end[a.n_tensors++] = a.tiles;
        }
        a.last = t == n_tensors;
        a.first_partial = used;
        const uint32_t blocks = gb::grad_norm_blocks(a.tiles);
        GB_TRY(check_launch(c, gb::launch_grad_norm(a, dtype, blocks, s), "gradient norm"));
        used += blocks;
    } while (t < n_tensors);
    return GB_OK;
}

// The launches of an AdamW step, N tensors each.
template <int N>
gb_status adamw_launches(gb_ctx *c, int n_tensors, float *const *params, const void *const *grads, void *const *exp_avg,
                         void *const *exp_avg_sq, void *const *copies, const size_t *numel, uint64_t elems, gb_dtype grad_dtype,
                         gb_codec state_codec, int block, const gb_adamw *cfg, const float *grad_scale, cudaStream_t s) {
    const size_t eb = elem_bytes(grad_dtype);
    gb::AdamwArgs<N> a;
    a.beta1 = (float)cfg->beta1;
    a.gain1 = (float)(1.0 - cfg->beta1);
    a.beta2 = (float)cfg->beta2;
    a.gain2 = (float)(1.0 - cfg->beta2);
    a.keep = (float)(1.0 - cfg->lr * cfg->weight_decay);
    a.rate = (float)(cfg->lr / (1.0 - std::pow(cfg->beta1, (double)cfg->step)));
    a.unroot = (float)(1.0 / std::sqrt(1.0 - std::pow(cfg->beta2, (double)cfg->step)));
    a.eps = cfg->eps > 0x1p-63 ? (float)cfg->eps : 0x1p-63f;
    a.grad_scale = grad_scale;
    uint32_t key = gb::mix32((uint32_t)cfg->seed + 0x9E3779B9u);
    key = gb::mix32(key ^ (uint32_t)(cfg->seed >> 32));
    key = gb::mix32(key ^ (uint32_t)cfg->step);
    key = gb::mix32(key ^ (uint32_t)(cfg->step >> 32));
    a.span = state_codec == GB_CODEC_NONE ? 1 : gb::adamw_span(elems);
    const uint32_t piece = gb::kTile * a.span;
    int t = 0;
    while (t < n_tensors) {
        a.n_tensors = 0;
        a.spans = 0;
        for (; t < n_tensors && a.n_tensors < N; ++t) {
            if (!numel[t]) continue;
            const int k = a.n_tensors++;
            a.key[k] = gb::mix32(key ^ (uint32_t)t);
            a.param[k] = params[t];
            a.grad[k] = grads[t];
            a.m[k] = exp_avg[t];
            a.v[k] = exp_avg_sq[t];
            a.copy[k] = copies ? copies[t] : nullptr;
            a.numel[k] = numel[t];
            // the arrays share a vector boundary: tiles start there, in float32 states anywhere, with 8-bit
            // states (whose blocks and random numbers count from element 0) at element 0
            const uint32_t shift = gb::vector_shift(params[t], 4);
            bool alike = gb::vector_shift(grads[t], eb) == shift && (!copies || gb::vector_shift(copies[t], eb) == shift);
            if (state_codec == GB_CODEC_NONE)
                alike = alike && gb::vector_shift(exp_avg[t], 4) == shift && gb::vector_shift(exp_avg_sq[t], 4) == shift;
            else
                alike = alike && shift == 0;
            a.layout[k] = alike ? (unsigned short)shift : gb::kScattered;
            a.spans += (uint32_t)gb::tiles_of(numel[t], alike ? shift : 0, piece);
            a.span_end[k] = a.spans;
        }
        if (a.n_tensors == 0) break;
        GB_TRY(check_launch(c, gb::launch_adamw(a, grad_dtype, state_codec == GB_CODEC_NONE ? 0 : block,
                                                copies != nullptr, s), "AdamW step"));
    }
    return GB_OK;
}

}  // namespace

extern "C" {

gb_status gb_grad_norm(gb_ctx *c, int n_tensors, const void *const *grads, const size_t *numel, gb_dtype dtype,
                       float max_norm, float *out, gb_stream stream) {
    GB_TRY(check_ctx(c));
    GB_TRY(check_train_dtype(c, dtype));
    uint64_t elems = 0;
    GB_TRY(check_tensors(c, n_tensors, numel, &elems));
    if (n_tensors > 0 && !grads) return set_msg(c, GB_ERR_INVALID_ARG, "grads is NULL");
    for (int t = 0; t < n_tensors; ++t)
        if (numel[t]) GB_TRY(check_align(c, grads[t], elem_bytes(dtype), "grads", t));
    if ((size_t)n_tensors / gb::kNormTensors + 1 > 4 * gb::kWorkFloats / sizeof(double) / gb::kNormPartials)
        return set_msg(c, GB_ERR_TOO_LARGE, "%d tensors: the workspace holds partial sums of fewer", n_tensors);
    if (std::isnan(max_norm)) return set_msg(c, GB_ERR_INVALID_ARG, "max_norm is not a number");
    GB_TRY(check_align(c, out, 4, "out"));
    GB_TRY(bind(c));
    cudaStream_t s = (cudaStream_t)stream;
    Work w;
    GB_TRY(begin_work(c, s, &w));
    int filled = 0;
    for (int t = 0; t < n_tensors; ++t) filled += numel[t] != 0;
    GB_TRY(filled <= gb::kFewTensors ? norm_launches<gb::kFewTensors>(c, w, n_tensors, grads, numel, dtype, max_norm, out, s)
                                     : norm_launches<gb::kNormTensors>(c, w, n_tensors, grads, numel, dtype, max_norm, out, s));
    return end_work(c, s, w);
}

gb_status gb_adamw_step(gb_ctx *c, int n_tensors, float *const *params, const void *const *grads,
                        void *const *exp_avg, void *const *exp_avg_sq, void *const *copies, const size_t *numel,
                        gb_dtype grad_dtype, gb_codec state_codec, int block, const gb_adamw *cfg,
                        const float *grad_scale, gb_stream stream) {
    GB_TRY(check_ctx(c));
    GB_TRY(check_train_dtype(c, grad_dtype));
    if (state_codec != GB_CODEC_NONE && state_codec != GB_CODEC_E4M3)
        return set_msg(c, GB_ERR_UNSUPPORTED_CODEC, "states are float32 (GB_CODEC_NONE) or GB_CODEC_E4M3");
    GB_TRY(check_codec(c, state_codec, block));
    if (copies && grad_dtype == GB_F32)
        return set_msg(c, GB_ERR_UNSUPPORTED_DTYPE, "copies have the gradients' type, which must be of 16 bits");
    if (!cfg) return set_msg(c, GB_ERR_INVALID_ARG, "cfg is NULL");
    if (!std::isfinite(cfg->lr) || !std::isfinite(cfg->weight_decay) || !(cfg->beta1 >= 0 && cfg->beta1 < 1) ||
        !(cfg->beta2 >= 0 && cfg->beta2 < 1) || !(cfg->eps >= 0 && std::isfinite(cfg->eps)) || cfg->step < 1)
        return set_msg(c, GB_ERR_INVALID_ARG, "lr %g betas %g %g eps %g weight decay %g step %llu", cfg->lr, cfg->beta1,
                       cfg->beta2, cfg->eps, cfg->weight_decay, (unsigned long long)cfg->step);
    uint64_t elems = 0;
    GB_TRY(check_tensors(c, n_tensors, numel, &elems));
    if (n_tensors > 0 && (!params || !grads || !exp_avg || !exp_avg_sq))
        return set_msg(c, GB_ERR_INVALID_ARG, "an array of tensors is NULL");
    const size_t eb = elem_bytes(grad_dtype), sb = state_codec == GB_CODEC_NONE ? 4 : 32;
    for (int t = 0; t < n_tensors; ++t) {
        if (!numel[t]) continue;
        GB_TRY(check_align(c, params[t], 4, "params", t));
        GB_TRY(check_align(c, grads[t], eb, "grads", t));
        GB_TRY(check_align(c, exp_avg[t], sb, "exp_avg", t));
        GB_TRY(check_align(c, exp_avg_sq[t], sb, "exp_avg_sq", t));
        if (copies) GB_TRY(check_align(c, copies[t], eb, "copies", t));
    }
    if (grad_scale) GB_TRY(check_align(c, grad_scale, 4, "grad_scale"));
    if (elems == 0) return GB_OK;
    GB_TRY(bind(c));

    int filled = 0;
    for (int t = 0; t < n_tensors; ++t) filled += numel[t] != 0;
    cudaStream_t s = (cudaStream_t)stream;
    return filled <= gb::kFewTensors
               ? adamw_launches<gb::kFewTensors>(c, n_tensors, params, grads, exp_avg, exp_avg_sq, copies, numel, elems, grad_dtype,
                                                 state_codec, block, cfg, grad_scale, s)
               : adamw_launches<gb::kAdamwTensors>(c, n_tensors, params, grads, exp_avg, exp_avg_sq, copies, numel, elems, grad_dtype,
                                                   state_codec, block, cfg, grad_scale, s);
}

size_t gb_rms_norm_payload_bytes(gb_codec codec, int block, size_t rows, size_t cols) {
    if (!codec_ok(codec, block) || !is_fp8(codec)) return 0;
    if (cols && rows > kMaxElems / cols) return 0;
    return round_up(rows * cols, 16) + 4 * rows * ((cols + block - 1) / block);
}

gb_status gb_rms_norm(gb_ctx *c, const void *x, const void *residual, const void *weight, size_t rows, size_t cols,
                      gb_dtype dtype, float eps, gb_codec codec, int block, void *sum_out, void *out, float *rstd,
                      gb_stream stream) {
    GB_TRY(check_ctx(c));
    GB_TRY(check_train_dtype(c, dtype));
    if (codec == GB_CODEC_BF16) return set_msg(c, GB_ERR_UNSUPPORTED_CODEC, "the output has the rows' type or 8 bits");
    GB_TRY(check_codec(c, codec, block));
    if (cols && rows > kMaxElems / cols) return set_msg(c, GB_ERR_INVALID_ARG, "%zu x %zu too large", rows, cols);
    if (cols > UINT32_MAX / 2) return set_msg(c, GB_ERR_INVALID_ARG, "cols = %zu too large", cols);
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return set_msg(c, GB_ERR_INVALID_ARG, "eps = %g", (double)eps);
    if (rows == 0 || cols == 0) return GB_OK;
    const size_t n = rows * cols, eb = elem_bytes(dtype);
    GB_TRY(check_align(c, x, 16, "x"));
    if (residual) GB_TRY(check_align(c, residual, 16, "residual"));
    GB_TRY(check_align(c, weight, eb, "weight"));
    if (sum_out && !residual) return set_msg(c, GB_ERR_INVALID_ARG, "sum_out without a residual");
    if (sum_out) GB_TRY(check_align(c, sum_out, 16, "sum_out"));
    GB_TRY(check_align(c, out, codec == GB_CODEC_NONE ? 16 : 32, "out"));
    if (rstd) GB_TRY(check_align(c, rstd, 16, "rstd"));
    const size_t ob = codec == GB_CODEC_NONE ? n * eb : gb_rms_norm_payload_bytes(codec, block, rows, cols);
    // an output of the rows' type may be x or residual itself; nothing else may overlap
    const bool fp8 = codec != GB_CODEC_NONE;
    if (overlap(out, ob, sum_out, n * eb) || overlap(out, ob, weight, cols * eb) || overlap(sum_out, n * eb, weight, cols * eb) ||
        overlap(rstd, 4 * rows, x, n * eb) || (residual && overlap(rstd, 4 * rows, residual, n * eb)) ||
        overlap(rstd, 4 * rows, weight, cols * eb) || overlap(rstd, 4 * rows, out, ob) ||
        (sum_out && overlap(rstd, 4 * rows, sum_out, n * eb)) || cross(sum_out, n * eb, x, n * eb) ||
        cross(sum_out, n * eb, residual, n * eb) || cross(out, ob, x, n * eb) || cross(out, ob, residual, n * eb) ||
        (fp8 && (out == x || out == residual)))
        return set_msg(c, GB_ERR_INVALID_ARG, "buffers overlap");
    GB_TRY(bind(c));
    gb::RmsArgs a;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.sum = sum_out;
    a.out = out;
    a.rstd = rstd;
    a.rows = rows;
    a.whole_rows = gb::whole_rows(rows, (uint32_t)cols);
    a.cols = (uint32_t)cols;
    a.eps = eps;
    a.inv_cols = 1.0f / (float)cols;
    a.scales_off = round_up(n, 16);
    return check_launch(c, gb::launch_rms_norm(a, dtype, codec, block, (cudaStream_t)stream), "RMS norm");
}

gb_status gb_rms_norm_backward(gb_ctx *c, const void *dy, const void *h, const void *weight, const float *rstd,
                               const void *dsum, size_t rows, size_t cols, gb_dtype dtype, void *dx, void *dweight,
                               gb_stream stream) {
    GB_TRY(check_ctx(c));
    GB_TRY(check_train_dtype(c, dtype));
    if (cols && rows > kMaxElems / cols) return set_msg(c, GB_ERR_INVALID_ARG, "%zu x %zu too large", rows, cols);
    if (cols > gb::kWorkFloats) return set_msg(c, GB_ERR_TOO_LARGE, "cols = %zu beyond the workspace", cols);
    if (cols == 0) return GB_OK;
    const size_t n = rows * cols, eb = elem_bytes(dtype);
    if (rows) {
        GB_TRY(check_align(c, dy, 16, "dy"));
        GB_TRY(check_align(c, h, 16, "h"));
        GB_TRY(check_align(c, weight, eb, "weight"));
        GB_TRY(check_align(c, rstd, 16, "rstd"));
        if (dsum) GB_TRY(check_align(c, dsum, 16, "dsum"));
        GB_TRY(check_align(c, dx, 16, "dx"));
    }
    GB_TRY(check_align(c, dweight, eb, "dweight"));
    // dx may be dy, h or dsum itself; nothing else may overlap
    if (rows && (cross(dx, n * eb, dy, n * eb) || cross(dx, n * eb, h, n * eb) || cross(dx, n * eb, dsum, n * eb) ||
                 overlap(dx, n * eb, weight, cols * eb) || overlap(dx, n * eb, rstd, 4 * rows) ||
                 overlap(dx, n * eb, dweight, cols * eb) || overlap(dweight, cols * eb, dy, n * eb) ||
                 overlap(dweight, cols * eb, h, n * eb) || overlap(dweight, cols * eb, weight, cols * eb) ||
                 overlap(dweight, cols * eb, rstd, 4 * rows) || (dsum && overlap(dweight, cols * eb, dsum, n * eb))))
        return set_msg(c, GB_ERR_INVALID_ARG, "buffers overlap");
    GB_TRY(bind(c));
    cudaStream_t s = (cudaStream_t)stream;
    Work work;
    GB_TRY(begin_work(c, s, &work));
    gb::RmsGradArgs a;
    a.dy = dy;
    a.h = h;
    a.weight = weight;
    a.dsum = dsum;
    a.rstd = rstd;
    a.dx = dx;
    a.dweight = dweight;
    a.partials = (float *)work.partials;
    a.rows = rows;
    a.whole_rows = gb::whole_rows(rows, (uint32_t)cols);
    a.cols = (uint32_t)cols;
    a.inv_cols = 1.0f / (float)cols;
    GB_TRY(check_launch(c, gb::launch_rms_norm_backward(a, dtype, s), "RMS norm gradient"));
    return end_work(c, s, work);
}

}  // extern "C"
