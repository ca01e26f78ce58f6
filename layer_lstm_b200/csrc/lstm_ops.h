// Internal interface between the entry points of the operators beside the
// LSTM (lstm_ops_abi.cu) and their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "lstm_internal.h"

namespace lstm {

// Timing kinds of these operators; names in lstm_abi.cu, same order.
enum OpKind { OP_ADAMW = 0, OP_NORM_FWD, OP_NORM_BWD, OP_ATT_FWD, OP_ATT_BWD, OP_ATT_STEP, kOpKinds };

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

// ---------------------------------------------------------------- linear attention
// One product of the recurrence, for every (batch row, head):
//   out_i = oscale (sum_{j <= i} bscale g^(i-j) (a_i . b_j) c_j + g^(i+e) a_i X0)
// over the row's n valid steps, taken forwards (e = 1) or, with `reverse`,
// backwards (e = 0), and the state after them
//   X = g^n X0 + sum_j bscale g^(n-e-j) b_j^T c_j.
// The forward is one such product; the backward is three (its gradients with
// respect to q, k and v) on permuted operands.
struct LinJob {
    const void* a; long long lda;   // rows of da (a, b) and dc (c, o) elements per head, ld between time rows
    const void* b; long long ldb;
    const void* c; long long ldc;
    void* o; long long ldo;
    int da, dc;
    int reverse;
    float bscale, oscale;
    const float* init;              // [B*H] X0, or null (zeros)
    int init_t;                     // 1: X0 is stored transposed, [dc][da]
    float* fin;                     // [B*H][da][dc] final state, or null
};

constexpr int kLinMaxDim = 128;
constexpr int kLinChunk = 64;       // steps whose products form one score matrix
constexpr int kLinTcChunk = 128;    // the same on the tensor cores

struct LinArgs {
    int B, T, H;
    int batch_first;
    DType dt;
    const int* lengths;             // [B] or null
    const float* log_decay;         // [H]
    int njobs;
    LinJob job[3];
    int nseg, seg_len;              // the time axis in nseg parts of seg_len steps
    float* buf;                     // nseg > 1: [njobs][B*H][nseg][da*dc] segment states
    int from_end;                   // segments are counted from the valid steps' end (see lin_steps)
    int* status;
    uint64_t timeout_ns;
    int skip_block, skip_chunk;     // fault injection of a test (-1: none), see skip_arrival
    int num_sms;
};
// Parts the time axis is cut into for njobs products; 1: none.  `tc`: for the
// tensor-core kernel.
int lin_segments(int B, int T, int H, int njobs, int num_sms, bool tc, int* seg_len);
cudaError_t launch_lin(const void* args, cudaStream_t s, int* nlaunch);

// The tensor-core kernel: whether these products can run on it (types, sizes,
// alignment), and its launches.
bool lin_tc_ok(const LinArgs& a);
cudaError_t launch_lin_tc(const LinArgs& a, cudaStream_t s, int* n);

// Limit of a bounded wait (lstm_query_status).
uint64_t wait_limit_ns();
// The block and chunk of LSTM_B200_DEBUG_SKIP_ARRIVAL="att:<block>:<chunk>", -1 without it.
void lin_skip(int* block, int* chunk);

struct LinStepArgs {
    int B, H, dk, dv;
    DType dt;
    float scale;
    const int* lengths;             // [B], rows with none are left alone; or null
    const void* q; const void* k; const void* v;
    long long ldq, ldk, ldv;        // elements between batch rows
    const float* log_decay;
    float* state;                   // [B][H][dk][dv], updated
    void* out;
};
cudaError_t launch_lin_step(const void* args, cudaStream_t s, int* nlaunch);

}  // namespace lstm
