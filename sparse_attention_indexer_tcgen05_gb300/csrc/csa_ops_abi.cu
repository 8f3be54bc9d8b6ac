// csa_ops_abi.cu -- the entry points around the step (projections, rotary positions, AdamW): argument checks and
// dispatch.  Everything is checked on the host before anything is enqueued; no device memory is allocated and the
// stream is never synchronised.
#include "csa_internal.cuh"

#include <math.h>
#include <stdlib.h>

using namespace csa;

namespace {

#define CSA_TRY(x)                   \
    do {                             \
        csa_status _s = (x);         \
        if (_s != CSA_OK) return _s; \
    } while (0)

#define CSA_CUDA(x)                                            \
    do {                                                       \
        const cudaError_t csa_e_ = (x);                        \
        if (csa_e_ != cudaSuccess) return cuda_failed(csa_e_); \
    } while (0)

// A tensor argument: must be non-null and 16-byte aligned whenever it holds at least one element.
csa_status need(const void *ptr, long long elems)
{
    if (elems <= 0) return CSA_OK;
    if (ptr == nullptr) return CSA_ERR_INVALID_ARG;
    return ((uintptr_t)ptr & 15) == 0 ? CSA_OK : CSA_ERR_ALIGNMENT;
}
csa_status need_opt(const void *ptr) { return ptr == nullptr ? CSA_OK : need(ptr, 1); }
// An optional device scalar
csa_status need_scalar(const void *ptr, size_t size)
{
    return ((uintptr_t)ptr & (size - 1)) == 0 ? CSA_OK : CSA_ERR_ALIGNMENT;
}

inline bool value_dtype(int d) { return d == CSA_F32 || d == CSA_BF16; }

// ------------------------------------------------------------------ projections

// Fills in the defaults of the strides.
csa_status check_linear(const csa_linear_params *p, csa_linear_params *q)
{
    if (p == nullptr) return CSA_ERR_INVALID_ARG;
    *q = *p;
    if (!value_dtype(p->dtype) || !value_dtype(p->out_dtype)) return CSA_ERR_INVALID_ARG;
    if (p->activation < CSA_ACT_NONE || p->activation > CSA_ACT_GELU_TANH) return CSA_ERR_INVALID_ARG;
    if (p->in_features < 1 || p->out_features < 1 || p->rows < 0 || !isfinite(p->alpha)) return CSA_ERR_INVALID_ARG;
    if (q->x_stride == 0) q->x_stride = p->in_features;
    if (q->residual_stride == 0) q->residual_stride = p->out_features;
    if (q->dy_stride == 0) q->dy_stride = p->out_features;
    if (q->x_stride < p->in_features || q->residual_stride < p->out_features || q->dy_stride < p->out_features)
        return CSA_ERR_INVALID_ARG;
    if (p->out_dtype != p->dtype && p->out_dtype != CSA_F32) return CSA_ERR_UNSUPPORTED;
    // rows and features are TMA coordinates and 32-bit loop counters, which run a step of at most 32768 beyond them;
    // strides are TMA byte strides (below 2^40)
    constexpr int most = 0x7fff0000;
    if (p->rows > most || p->in_features > most || p->out_features > most) return CSA_ERR_UNSUPPORTED;
    const long long far = 1LL << 36;
    if (q->x_stride > far || q->residual_stride > far || q->dy_stride > far) return CSA_ERR_UNSUPPORTED;
    return CSA_OK;
}

// An output that is another argument's buffer would be written while others still read it.
bool shares(const void *out, const void *const *others, int n)
{
    if (out == nullptr) return false;
    for (int i = 0; i < n; i++)
        if (others[i] == out) return true;
    return false;
}

// ------------------------------------------------------------------ rotary positions

csa_status check_rope(const csa_rope_params *p, csa_rope_params *q)
{
    if (p == nullptr) return CSA_ERR_INVALID_ARG;
    *q = *p;
    if (!value_dtype(p->dtype) || p->heads < 1 || p->head_dim < 1 || p->rows < 0) return CSA_ERR_INVALID_ARG;
    if (p->rot_offset < 0 || p->rot_dim < 0 || (p->rot_dim & 1) != 0) return CSA_ERR_INVALID_ARG;
    if ((long long)p->rot_offset + p->rot_dim > p->head_dim) return CSA_ERR_INVALID_ARG;
    if ((p->interleaved & ~1) || (p->inverse & ~1) || (p->positions_64 & ~1)) return CSA_ERR_INVALID_ARG;
    if (p->axes < 1 || p->axes > CSA_ROPE_MAX_AXES) return CSA_ERR_INVALID_ARG;
    long long sum = 0;
    for (int i = 0; i < p->axes; i++) {
        if (p->sections[i] < 0) return CSA_ERR_INVALID_ARG;
        sum += p->sections[i];
    }
    if (sum != p->rot_dim / 2) return CSA_ERR_INVALID_ARG;
    if (q->x_head_stride == 0) q->x_head_stride = p->head_dim;
    if (q->out_head_stride == 0) q->out_head_stride = p->head_dim;
    if (q->x_head_stride < p->head_dim || q->out_head_stride < p->head_dim) return CSA_ERR_INVALID_ARG;
    const long long far = 1LL << 40;
    if (p->rows > far || q->x_head_stride > far / p->heads || q->out_head_stride > far / p->heads) return CSA_ERR_UNSUPPORTED;
    if (q->x_row_stride == 0) q->x_row_stride = p->heads * q->x_head_stride;
    if (q->out_row_stride == 0) q->out_row_stride = p->heads * q->out_head_stride;
    if (q->x_row_stride < p->head_dim || q->out_row_stride < p->head_dim) return CSA_ERR_INVALID_ARG;
    if (q->x_row_stride > far || q->out_row_stride > far) return CSA_ERR_UNSUPPORTED;
    // no two vectors of out share an element: a row's heads lie within the row stride, or (heads outermost) a head's
    // rows within the head stride.  2^40 * 2^40 would pass 64 bits: compare by division
    const bool rows_outer = q->out_row_stride - p->head_dim >= (p->heads - 1) * q->out_head_stride;
    const bool heads_outer = p->rows <= 1 || (q->out_head_stride - p->head_dim) / q->out_row_stride >= p->rows - 1;
    if (!rows_outer && !heads_outer) return CSA_ERR_INVALID_ARG;
    if (p->rot_dim > 1024 || p->head_dim > (1 << 18) || (p->rows > 0 && (q->x_row_stride > (1LL << 60) / p->rows || q->out_row_stride > (1LL << 60) / p->rows)))
        return CSA_ERR_UNSUPPORTED;
    return CSA_OK;
}

// ------------------------------------------------------------------ AdamW

// The written buffers of all tensors, by their first byte: a buffer named twice would be updated by two CTAs at once.
struct Seen {
    uintptr_t *slot;
    size_t mask;
    explicit Seen(size_t n) : slot(nullptr), mask(0)
    {
        size_t cap = 64;
        while (cap < 2 * n) cap *= 2;
        slot = static_cast<uintptr_t *>(calloc(cap, sizeof(uintptr_t)));
        mask = cap - 1;
    }
    ~Seen() { free(slot); }
    bool twice(const void *p)
    {
        if (p == nullptr) return false;
        const uintptr_t a = (uintptr_t)p;
        for (size_t i = (a >> 4) * 0x9e3779b97f4a7c15ull >> 20;; i++) {
            uintptr_t &s = slot[i & mask];
            if (s == a) return true;
            if (s == 0) {
                s = a;
                return false;
            }
        }
    }
};

csa_status check_adamw(const csa_adamw_params *p, const csa_adamw_tensor *t, int32_t count)
{
    if (p == nullptr || count < 0 || (count > 0 && t == nullptr)) return CSA_ERR_INVALID_ARG;
    if (!isfinite(p->lr) || !isfinite(p->eps) || !isfinite(p->weight_decay) || p->eps < 0) return CSA_ERR_INVALID_ARG;
    if (!(p->beta1 >= 0 && p->beta1 < 1) || !(p->beta2 >= 0 && p->beta2 < 1)) return CSA_ERR_INVALID_ARG;
    if (p->step_dev == nullptr && p->step < 1) return CSA_ERR_INVALID_ARG;
    if (p->stochastic & ~1) return CSA_ERR_INVALID_ARG;
    CSA_TRY(need_scalar(p->lr_dev, 4));
    CSA_TRY(need_scalar(p->step_dev, 8));
    CSA_TRY(need_scalar(p->grad_scale, 4));
    CSA_TRY(need_scalar(p->found_inf, 4));
    Seen seen((size_t)count * 6);
    if (seen.slot == nullptr) return CSA_ERR_UNSUPPORTED;  // no host memory for the check
    for (int i = 0; i < count; i++) {
        const csa_adamw_tensor &e = t[i];
        if (e.numel < 0 || !value_dtype(e.param_dtype) || !value_dtype(e.grad_dtype)) return CSA_ERR_INVALID_ARG;
        if (e.state_dtype != CSA_STATE_F32 && e.state_dtype != CSA_STATE_E4M3) return CSA_ERR_INVALID_ARG;
        if (e.numel > (1LL << 40)) return CSA_ERR_UNSUPPORTED;
        if (e.numel == 0) continue;
        CSA_TRY(need(e.param, e.numel));
        CSA_TRY(need(e.grad, e.numel));
        CSA_TRY(need_opt(e.master));
        CSA_TRY(need(e.m, e.numel));
        CSA_TRY(need(e.v, e.numel));
        bool twice = seen.twice(e.param) || seen.twice(e.master) || seen.twice(e.m) || seen.twice(e.v);
        if (e.state_dtype == CSA_STATE_E4M3) {
            // scales are views into a larger buffer more often than not: 4-byte alignment is enough
            if (e.m_scale == nullptr || e.v_scale == nullptr) return CSA_ERR_INVALID_ARG;
            CSA_TRY(need_scalar(e.m_scale, 4));
            CSA_TRY(need_scalar(e.v_scale, 4));
            twice = twice || seen.twice(e.m_scale) || seen.twice(e.v_scale);
        }
        if (twice) return CSA_ERR_INVALID_ARG;
    }
    return CSA_OK;
}

}  // namespace

extern "C" {

size_t csa_linear_fwd_workspace_size(const csa_linear_params *p)
{
    csa_linear_params q;
    return check_linear(p, &q) == CSA_OK ? linear_fwd_workspace(q) : 0;
}

size_t csa_linear_bwd_workspace_size(const csa_linear_params *p)
{
    csa_linear_params q;
    return check_linear(p, &q) == CSA_OK ? linear_bwd_workspace(q) : 0;
}

csa_status csa_linear_fwd(const csa_linear_params *p, const void *x, const void *weight, const float *bias,
                          const void *residual, void *y, void *preact, void *workspace, size_t workspace_bytes,
                          void *stream)
{
    CSA_TRY(injected_fault());
    csa_linear_params q;
    CSA_TRY(check_linear(p, &q));
    CSA_TRY(need(x, q.rows));
    CSA_TRY(need(weight, 1));
    CSA_TRY(need_opt(bias));
    CSA_TRY(need_opt(residual));
    CSA_TRY(need(y, q.rows));
    CSA_TRY(need_opt(preact));
    const size_t ws = linear_fwd_workspace(q);
    if (workspace_bytes < ws || (ws > 0 && workspace == nullptr)) return CSA_ERR_WORKSPACE;
    CSA_TRY(need_opt(workspace));
    if (q.rows == 0) return CSA_OK;
    if (residual == y && q.residual_stride != q.out_features && q.rows > 1) return CSA_ERR_INVALID_ARG;
    const void *inputs[] = {x, weight, bias, preact, residual};
    if (shares(y, inputs, 4)) return CSA_ERR_INVALID_ARG;
    inputs[3] = y;
    if (shares(preact, inputs, 5)) return CSA_ERR_INVALID_ARG;
    CSA_CUDA(launch_linear_fwd(q, x, weight, bias, residual, y, preact, workspace, static_cast<cudaStream_t>(stream)));
    return CSA_OK;
}

csa_status csa_linear_bwd(const csa_linear_params *p, const void *dy, const void *x, const void *weight,
                          const void *preact, void *dx, void *dw, float *db, void *workspace, size_t workspace_bytes,
                          void *stream)
{
    CSA_TRY(injected_fault());
    csa_linear_params q;
    CSA_TRY(check_linear(p, &q));
    CSA_TRY(need(dy, q.rows));
    if (dw != nullptr) CSA_TRY(need(x, q.rows));
    if (dx != nullptr) CSA_TRY(need(weight, 1));
    if (q.activation != CSA_ACT_NONE) CSA_TRY(need(preact, q.rows));
    CSA_TRY(need_opt(dx));
    CSA_TRY(need_opt(dw));
    CSA_TRY(need_opt(db));
    const size_t ws = linear_bwd_workspace(q);
    if (workspace_bytes < ws || (ws > 0 && workspace == nullptr)) return CSA_ERR_WORKSPACE;
    CSA_TRY(need_opt(workspace));
    const void *inputs[] = {q.rows > 0 ? dy : nullptr, dw != nullptr ? x : nullptr, dx != nullptr ? weight : nullptr,
                            q.activation != CSA_ACT_NONE ? preact : nullptr, dx, dw};
    if (shares(dx, inputs, 4) || shares(dw, inputs, 5) || shares(db, inputs, 6)) return CSA_ERR_INVALID_ARG;
    CSA_CUDA(launch_linear_bwd(q, dy, x, weight, preact, dx, dw, db, workspace, static_cast<cudaStream_t>(stream)));
    return CSA_OK;
}

csa_status csa_rope(const csa_rope_params *p, const void *x, const void *positions, const double *inv_freq, void *out,
                    void *stream)
{
    CSA_TRY(injected_fault());
    csa_rope_params q;
    CSA_TRY(check_rope(p, &q));
    CSA_TRY(need(x, q.rows));
    CSA_TRY(need(out, q.rows));
    if (q.rot_dim > 0 && q.rows > 0) {
        if (positions == nullptr || inv_freq == nullptr) return CSA_ERR_INVALID_ARG;
        CSA_TRY(need_scalar(positions, q.positions_64 ? 8 : 4));
        CSA_TRY(need_scalar(inv_freq, 8));
    }
    if (x == out && (q.x_row_stride != q.out_row_stride || q.x_head_stride != q.out_head_stride)) return CSA_ERR_INVALID_ARG;
    if (q.rows == 0) return CSA_OK;
    CSA_CUDA(launch_rope(q, x, positions, inv_freq, out, static_cast<cudaStream_t>(stream)));
    return CSA_OK;
}

csa_status csa_adamw(const csa_adamw_params *p, const csa_adamw_tensor *tensors, int32_t count, void *stream)
{
    CSA_TRY(injected_fault());
    CSA_TRY(check_adamw(p, tensors, count));
    CSA_CUDA(launch_adamw(*p, tensors, count, static_cast<cudaStream_t>(stream)));
    return CSA_OK;
}

}  // extern "C"
