// C-ABI entry points of the operators beside the LSTM (include/lstm.h,
// "Operators beside the LSTM"): argument checks on the host, then the
// kernels' launchers under the library's kernel timing.
#include <float.h>
#include <math.h>

#include <mutex>
#include <vector>

#include "../../include/lstm.h"
#include "lstm_ops.h"

namespace lstm {
namespace {

// SMs of the current device (0 if it cannot be asked), looked up once each.
int num_sms() {
    static std::mutex mu;
    static std::vector<int> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lk(mu);
    if ((int)cache.size() <= dev) cache.resize(dev + 1, 0);
    if (!cache[dev] && cudaDeviceGetAttribute(&cache[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        cache[dev] = 0;
    return cache[dev];
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
// A required pointer to elements of `a` bytes.
bool given(const void* p, size_t a) { return p && aligned(p, a); }
bool finite_ge0(double x) { return isfinite(x) && x >= 0.0; }
// The kernel's own values: it takes them rounded to float32.
bool float_ge0(double x) { return x >= 0.0 && x <= (double)FLT_MAX; }

bool valid(const lstm_adamw_desc* d) {
    return d && d->num_tensors >= 0 && (d->grad_dtype == LSTM_F32 || d->grad_dtype == LSTM_BF16) &&
           (d->state_bits == 8 || d->state_bits == 32) && finite_ge0(d->lr) && d->beta1 >= 0.0 && d->beta1 < 1.0 &&
           d->beta2 >= 0.0 && d->beta2 < 1.0 && finite_ge0(d->weight_decay) &&
           // the largest step size and decay the kernel forms; an infinite one times a zero moment is NaN
           float_ge0(d->lr / (1.0 - d->beta1)) && float_ge0(d->lr * d->weight_decay) &&
           // what a zero second moment leaves under the quotient: its reciprocal has to be a number, not 0
           d->eps >= (double)FLT_MIN && d->eps <= 0x1p126;
}

bool valid(const lstm_norm_desc* d) {
    return d && d->rows >= 0 && d->cols >= 1 && (d->dtype == LSTM_F32 || d->dtype == LSTM_BF16) &&
           isfinite(d->eps) && d->eps >= 0.0f;
}
// (columns are counted in 32 bits, a block's stride past the last one included)
bool supported(const lstm_norm_desc* d) { return d->cols <= 1 << 30; }

bool valid(const lstm_attention_desc* d) {
    if (!d || d->batch < 0 || d->seq_len < 0 || d->heads < 1 || d->key_size < 1 || d->value_size < 1) return false;
    if (d->batch_first != 0 && d->batch_first != 1) return false;
    if ((d->dtype != LSTM_F32 && d->dtype != LSTM_BF16) || !isfinite(d->scale)) return false;
    const long long wk = (long long)d->heads * d->key_size, wv = (long long)d->heads * d->value_size;
    // one work item per (row, head) of a product; 2^31 of them is more than a GPU holds
    if ((long long)d->batch * d->heads > (1ll << 28)) return false;
    return (d->ld_q == 0 || d->ld_q >= wk) && (d->ld_k == 0 || d->ld_k >= wk) && (d->ld_v == 0 || d->ld_v >= wv);
}
// (steps are counted in 32 bits, a chunk or a segment past the last one
// included, and so is a head's place in its row)
bool supported(const lstm_attention_desc* d) {
    return d->key_size <= kLinMaxDim && d->value_size <= kLinMaxDim && d->seq_len <= 1 << 30 &&
           (long long)d->heads * (d->key_size > d->value_size ? d->key_size : d->value_size) <= 1ll << 30;
}

DType dtype_of(lstm_dtype t) { return t == LSTM_F32 ? DType::F32 : DType::BF16; }

// Fields that every product of a description shares.
LinArgs lin_args(const lstm_attention_desc* d, const int* lengths, const float* log_decay, int njobs, void* ws) {
    LinArgs a{};
    a.B = d->batch; a.T = d->seq_len; a.H = d->heads; a.batch_first = d->batch_first;
    a.dt = dtype_of(d->dtype);
    a.lengths = lengths; a.log_decay = log_decay;
    a.njobs = njobs;
    // the status word, as in every workspace, then the segments' states
    a.status = static_cast<int*>(ws);
    a.buf = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
    a.timeout_ns = wait_limit_ns();
    lin_skip(&a.skip_block, &a.skip_chunk);
    a.num_sms = num_sms();
    return a;
}

size_t lin_ws(const lstm_attention_desc* d, int njobs) {
    const int sms = num_sms();
    int n = 1;
    for (int tc = 0; tc < 2; ++tc) {   // which kernel runs depends on the pointers too
        int len = 0;
        const int k = lin_segments(d->batch, d->seq_len, d->heads, njobs, sms > 0 ? sms : 148, tc != 0, &len);
        n = k > n ? k : n;
    }
    return n <= 1 ? 0 : (size_t)njobs * d->batch * d->heads * n * d->key_size * d->value_size * 4;
}

struct Lds { long long q, k, v, o; };
Lds lds_of(const lstm_attention_desc* d) {
    const long long wk = (long long)d->heads * d->key_size, wv = (long long)d->heads * d->value_size;
    return {d->ld_q ? d->ld_q : wk, d->ld_k ? d->ld_k : wk, d->ld_v ? d->ld_v : wv, wv};
}

}  // namespace
}  // namespace lstm

using namespace lstm;

extern "C" {

lstm_status lstm_adamw_step(const lstm_adamw_desc* desc, const long long* numel, float* const* param,
                            void* const* param_bf16, const void* const* grad, void* const* m, void* const* v,
                            float* const* m_scale, float* const* v_scale, long long* step,
                            const float* scalars, cudaStream_t stream) {
    if (!valid(desc) || !given(step, 8) || !aligned(scalars, 4)) return LSTM_ERR_INVALID_ARG;
    const int N = desc->num_tensors;
    const bool eight = desc->state_bits == 8;
    if (N > 0 && (!numel || !param || !grad || !m || !v || (eight && (!m_scale || !v_scale))))
        return LSTM_ERR_INVALID_ARG;
    const size_t ge = desc->grad_dtype == LSTM_F32 ? 4 : 2, se = eight ? 1 : 4;
    for (int i = 0; i < N; ++i) {
        if (numel[i] < 0) return LSTM_ERR_INVALID_ARG;
        if (numel[i] == 0) continue;
        if (!given(param[i], 4) || !given(grad[i], ge) || !given(m[i], se) || !given(v[i], se))
            return LSTM_ERR_INVALID_ARG;
        if (eight && (!given(m_scale[i], 4) || !given(v_scale[i], 4))) return LSTM_ERR_INVALID_ARG;
        if (param_bf16 && !aligned(param_bf16[i], 2)) return LSTM_ERR_INVALID_ARG;
    }
    AdamwArgs a{};
    a.bits = desc->state_bits;
    a.gdt = dtype_of(desc->grad_dtype);
    a.lr = desc->lr; a.beta1 = desc->beta1; a.beta2 = desc->beta2; a.eps = desc->eps;
    a.weight_decay = desc->weight_decay; a.seed = desc->seed;
    a.step = step; a.scalars = scalars;
    a.num_sms = num_sms();
    if (a.num_sms <= 0) return LSTM_ERR_CUDA;
    for (int first = 0; first == 0 || first < N; first += kAdamwTensors) {
        AdamwTensor t[kAdamwTensors];
        a.count = N - first < kAdamwTensors ? N - first : kAdamwTensors;
        a.first = first;
        a.advance = first + a.count == N;
        for (int i = 0; i < a.count; ++i) {
            const int j = first + i;
            t[i] = {param[j], param_bf16 ? param_bf16[j] : nullptr, grad[j], m[j], v[j],
                    eight ? m_scale[j] : nullptr, eight ? v_scale[j] : nullptr, numel[j]};
        }
        a.t = t;
        if (timed_op(OP_ADAMW, stream, launch_adamw, &a) != cudaSuccess) return LSTM_ERR_CUDA;
    }
    return LSTM_OK;
}

lstm_status lstm_adamw_read_state(const lstm_adamw_desc* desc, const long long* numel, void* const* m,
                                  void* const* v, float* const* m_scale, float* const* v_scale,
                                  float* const* m_out, float* const* v_out, cudaStream_t stream) {
    if (!valid(desc) || desc->state_bits != 8) return LSTM_ERR_INVALID_ARG;
    const int N = desc->num_tensors;
    if (N > 0 && (!numel || !m || !v || !m_scale || !v_scale || !m_out || !v_out)) return LSTM_ERR_INVALID_ARG;
    for (int i = 0; i < N; ++i) {
        if (numel[i] < 0) return LSTM_ERR_INVALID_ARG;
        if (numel[i] == 0) continue;
        if (!m[i] || !v[i] || !given(m_scale[i], 4) || !given(v_scale[i], 4) || !given(m_out[i], 4) ||
            !given(v_out[i], 4))
            return LSTM_ERR_INVALID_ARG;
    }
    AdamwReadArgs a{};
    a.num_sms = num_sms();
    if (a.num_sms <= 0) return LSTM_ERR_CUDA;
    for (int first = 0; first < N; first += kAdamwTensors) {
        AdamwTensor t[kAdamwTensors];
        a.count = N - first < kAdamwTensors ? N - first : kAdamwTensors;
        for (int i = 0; i < a.count; ++i) {
            const int j = first + i;
            t[i] = {nullptr, nullptr, nullptr, m[j], v[j], m_scale[j], v_scale[j], numel[j]};
        }
        a.t = t;
        a.m_out = m_out + first;
        a.v_out = v_out + first;
        if (timed_op(OP_ADAMW, stream, launch_adamw_read, &a) != cudaSuccess) return LSTM_ERR_CUDA;
    }
    return LSTM_OK;
}

size_t lstm_layer_norm_workspace_size(const lstm_norm_desc* desc) {
    if (!valid(desc) || !supported(desc)) return 0;
    // the partition of the largest device this library runs on serves where no device is at hand
    const int sms = num_sms();
    const size_t n = (size_t)norm_partials(desc->rows, desc->cols, sms > 0 ? sms : 148);
    return ((n > 0 ? n : 1) * 2 * (size_t)desc->cols * 4 + 255) / 256 * 256;
}

lstm_status lstm_layer_norm_forward(const lstm_norm_desc* desc, const void* x, const void* weight,
                                    const void* bias, void* y, float* mean, float* rstd, cudaStream_t stream) {
    if (!valid(desc)) return LSTM_ERR_INVALID_ARG;
    if (!supported(desc)) return LSTM_ERR_UNSUPPORTED;
    const size_t e = desc->dtype == LSTM_F32 ? 4 : 2;
    if (!aligned(weight, e) || !aligned(bias, e) || !aligned(mean, 4) || !aligned(rstd, 4))
        return LSTM_ERR_INVALID_ARG;
    if (desc->rows > 0 && (!given(x, e) || !given(y, e))) return LSTM_ERR_INVALID_ARG;
    if (desc->rows == 0) return LSTM_OK;
    NormFwdArgs a{};
    a.rows = desc->rows; a.cols = desc->cols; a.dt = dtype_of(desc->dtype); a.eps = desc->eps;
    a.x = x; a.w = weight; a.b = bias; a.y = y; a.mean = mean; a.rstd = rstd;
    a.num_sms = num_sms();
    if (a.num_sms <= 0) return LSTM_ERR_CUDA;
    return timed_op(OP_NORM_FWD, stream, launch_norm_fwd, &a) == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

lstm_status lstm_layer_norm_backward(const lstm_norm_desc* desc, const void* grad_y, const void* x,
                                     const void* weight, const float* mean, const float* rstd, void* dx,
                                     float* dweight, float* dbias, void* workspace, size_t ws_bytes,
                                     cudaStream_t stream) {
    if (!valid(desc)) return LSTM_ERR_INVALID_ARG;
    if (!supported(desc)) return LSTM_ERR_UNSUPPORTED;
    const size_t e = desc->dtype == LSTM_F32 ? 4 : 2;
    if (!aligned(weight, e) || !aligned(dx, e) || !aligned(dweight, 4) || !aligned(dbias, 4))
        return LSTM_ERR_INVALID_ARG;
    if (desc->rows > 0 && (!given(grad_y, e) || !given(x, e) || !given(mean, 4) || !given(rstd, 4)))
        return LSTM_ERR_INVALID_ARG;
    if (dweight || dbias) {
        if (!given(workspace, 256)) return LSTM_ERR_INVALID_ARG;
        if (ws_bytes < lstm_layer_norm_workspace_size(desc)) return LSTM_ERR_WORKSPACE;
    }
    if (!dx && !dweight && !dbias) return LSTM_OK;
    NormBwdArgs a{};
    a.rows = desc->rows; a.cols = desc->cols; a.dt = dtype_of(desc->dtype);
    a.gy = grad_y; a.x = x; a.w = weight; a.mean = mean; a.rstd = rstd;
    a.dx = dx; a.dw = dweight; a.db = dbias; a.part = static_cast<float*>(workspace);
    a.num_sms = num_sms();
    if (a.num_sms <= 0) return LSTM_ERR_CUDA;
    return timed_op(OP_NORM_BWD, stream, launch_norm_bwd, &a) == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

size_t lstm_linear_attention_workspace_size(const lstm_attention_desc* desc) {
    if (!valid(desc) || !supported(desc)) return 0;
    const size_t f = lin_ws(desc, 1), b = lin_ws(desc, 3), m = f > b ? f : b;
    return (m + 255) / 256 * 256 + 256;
}

lstm_status lstm_linear_attention_forward(const lstm_attention_desc* desc, const int* lengths, const void* q,
                                          const void* k, const void* v, const float* log_decay, const float* s0,
                                          void* out, float* s_n, void* workspace, size_t ws_bytes,
                                          cudaStream_t stream) {
    if (!valid(desc)) return LSTM_ERR_INVALID_ARG;
    if (!supported(desc)) return LSTM_ERR_UNSUPPORTED;
    const size_t e = desc->dtype == LSTM_F32 ? 4 : 2;
    if (!given(log_decay, 4) || !aligned(lengths, 4) || !aligned(s0, 4) || !aligned(s_n, 4))
        return LSTM_ERR_INVALID_ARG;
    if (desc->batch > 0 && desc->seq_len > 0 && (!given(q, e) || !given(k, e) || !given(v, e) || !given(out, e)))
        return LSTM_ERR_INVALID_ARG;
    if (!given(workspace, 256)) return LSTM_ERR_INVALID_ARG;
    if (ws_bytes < lstm_linear_attention_workspace_size(desc)) return LSTM_ERR_WORKSPACE;
    if (desc->batch == 0) return LSTM_OK;
    if (num_sms() <= 0) return LSTM_ERR_CUDA;
    LinArgs a = lin_args(desc, lengths, log_decay, 1, workspace);
    const Lds ld = lds_of(desc);
    a.job[0] = {q, ld.q, k, ld.k, v, ld.v, out, ld.o, desc->key_size, desc->value_size, 0, 1.0f, desc->scale,
                s0, 0, s_n};
    return timed_op(OP_ATT_FWD, stream, launch_lin, &a) == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

lstm_status lstm_linear_attention_backward(const lstm_attention_desc* desc, const int* lengths, const void* q,
                                           const void* k, const void* v, const float* log_decay, const float* s0,
                                           const void* grad_out, const float* grad_sn, void* dq, void* dk,
                                           void* dv, float* ds0, void* workspace, size_t ws_bytes,
                                           cudaStream_t stream) {
    if (!valid(desc)) return LSTM_ERR_INVALID_ARG;
    if (!supported(desc)) return LSTM_ERR_UNSUPPORTED;
    const size_t e = desc->dtype == LSTM_F32 ? 4 : 2;
    if (!given(log_decay, 4) || !aligned(lengths, 4) || !aligned(s0, 4) || !aligned(grad_sn, 4) || !aligned(ds0, 4))
        return LSTM_ERR_INVALID_ARG;
    if (desc->batch > 0 && desc->seq_len > 0 &&
        (!given(q, e) || !given(k, e) || !given(v, e) || !given(grad_out, e) || !given(dq, e) || !given(dk, e) ||
         !given(dv, e)))
        return LSTM_ERR_INVALID_ARG;
    if (!given(workspace, 256)) return LSTM_ERR_INVALID_ARG;
    if (ws_bytes < lstm_linear_attention_workspace_size(desc)) return LSTM_ERR_WORKSPACE;
    if (desc->batch == 0) return LSTM_OK;
    if (num_sms() <= 0) return LSTM_ERR_CUDA;
    LinArgs a = lin_args(desc, lengths, log_decay, 3, workspace);
    const Lds ld = lds_of(desc);
    const int dk_ = desc->key_size, dv_ = desc->value_size;
    const float s = desc->scale;
    // dq_i = s (sum_{j <= i} g^(i-j) (do_i . v_j) k_j + g^(i+1) do_i S0^T)
    a.job[0] = {grad_out, ld.o, v, ld.v, k, ld.k, dq, ld.q, dv_, dk_, 0, 1.0f, s, s0, 1, nullptr};
    // dk_j = sum_{i >= j} s g^(i-j) (v_j . do_i) q_i + g^(n-1-j) v_j dS_n^T
    a.job[1] = {v, ld.v, grad_out, ld.o, q, ld.q, dk, ld.k, dv_, dk_, 1, s, 1.0f, grad_sn, 1, nullptr};
    // dv_j = sum_{i >= j} s g^(i-j) (k_j . q_i) do_i + g^(n-1-j) k_j dS_n; its last state is ds0
    a.job[2] = {k, ld.k, q, ld.q, grad_out, ld.o, dv, ld.v, dk_, dv_, 1, s, 1.0f, grad_sn, 0, ds0};
    return timed_op(OP_ATT_BWD, stream, launch_lin, &a) == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

lstm_status lstm_linear_attention_step(const lstm_attention_desc* desc, const int* lengths, const void* q,
                                       const void* k, const void* v, const float* log_decay, float* state,
                                       void* out, cudaStream_t stream) {
    if (!valid(desc) || desc->seq_len != 1) return LSTM_ERR_INVALID_ARG;
    if (!supported(desc)) return LSTM_ERR_UNSUPPORTED;
    const size_t e = desc->dtype == LSTM_F32 ? 4 : 2;
    if (!given(log_decay, 4) || !aligned(lengths, 4)) return LSTM_ERR_INVALID_ARG;
    if (desc->batch == 0) return LSTM_OK;
    if (!given(q, e) || !given(k, e) || !given(v, e) || !given(out, e) || !given(state, 4))
        return LSTM_ERR_INVALID_ARG;
    const Lds ld = lds_of(desc);
    LinStepArgs a{};
    a.B = desc->batch; a.H = desc->heads; a.dk = desc->key_size; a.dv = desc->value_size;
    a.dt = dtype_of(desc->dtype); a.scale = desc->scale; a.lengths = lengths;
    a.q = q; a.k = k; a.v = v; a.ldq = ld.q; a.ldk = ld.k; a.ldv = ld.v;
    a.log_decay = log_decay; a.state = state; a.out = out;
    return timed_op(OP_ATT_STEP, stream, launch_lin_step, &a) == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

}  // extern "C"
