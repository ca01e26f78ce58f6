// Internal interface between the entry points of the operators beside the
// LSTM (lstm_ops_abi.cu) and their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "lstm_internal.h"

namespace lstm {

// Timing kinds of these operators; names in lstm_abi.cu, same order.
enum OpKind { OP_ADAMW = 0, OP_NORM_FWD, OP_NORM_BWD, kOpKinds };

// Runs launch(args, s, &launches) bracketed by the library's kernel timing.
cudaError_t timed_op(OpKind kind, cudaStream_t s, cudaError_t (*launch)(const void*, cudaStream_t, int*),
                     const void* args);

// ---------------------------------------------------------------- AdamW
// Elements that share one scale of the 8-bit moments.
constexpr int kAdamwBlock = 256;
// Tensors one launch takes (its table travels in the kernel's parameters).
constexpr int kAdamwTensors = 64;

struct AdamwTensor {
    float* p;
    void* copy;          // bf16 copy of p, or null
    const void* g;
    void* m;
    void* v;
    float* ms;           // 8-bit states: scales, one per kAdamwBlock elements
    float* vs;
    long long n;
};

struct AdamwArgs {
    int count;           // tensors in t
    int first;           // index of t[0] among the call's tensors
    int bits;            // 32 or 8
    DType gdt;
    double lr, beta1, beta2, eps, weight_decay;
    uint64_t seed;
    long long* step;     // device: steps taken before this one
    const float* scalars;   // device {learning-rate factor, gradient factor} or null
    int advance;         // 1: *step += 1 once the update has run
    int num_sms;
    const AdamwTensor* t;   // host
};
cudaError_t launch_adamw(const void* args, cudaStream_t s, int* nlaunch);

struct AdamwReadArgs {
    int count;
    float* const* m_out;    // host arrays
    float* const* v_out;
    int num_sms;
    const AdamwTensor* t;
};
cudaError_t launch_adamw_read(const void* args, cudaStream_t s, int* nlaunch);

// ---------------------------------------------------------------- layer norm
struct NormFwdArgs {
    long long rows;
    int cols;
    DType dt;
    float eps;
    const void* x; const void* w; const void* b;   // w, b: [cols] or null
    void* y;
    float* mean; float* rstd;                      // [rows] or null
    int num_sms;
};
cudaError_t launch_norm_fwd(const void* args, cudaStream_t s, int* nlaunch);

struct NormBwdArgs {
    long long rows;
    int cols;
    DType dt;
    const void* gy; const void* x; const void* w;
    const float* mean; const float* rstd;
    void* dx; float* dw; float* db;                // each may be null
    float* part;                                   // [norm_partials][2][cols]
    int num_sms;
};
// Row groups whose sums of dw and db are kept apart before they are added.
int norm_partials(long long rows, int cols, int num_sms);
cudaError_t launch_norm_bwd(const void* args, cudaStream_t s, int* nlaunch);

}  // namespace lstm
