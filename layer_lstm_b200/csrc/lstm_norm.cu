// Layer normalisation, forward and backward (Ba, Kiros and Hinton 2016; the
// equations are in include/lstm.h).  A row is two sums, a subtraction and a
// product per element, so HBM bounds it: x in and y out forward; x, grad_y in
// and dx out backward, with the column sums dw, db beside them.
#include "lstm_device.cuh"
#include "lstm_ops.h"

namespace lstm {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the block, in every thread.  `red` holds a value per warp.
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = warp_sum(v);
    __syncthreads();   // red may still be read from the last sum
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v += red[i];
    return v;
}

// One block per row, any width and alignment: the row is read again for each
// pass over it.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(const NormFwdArgs a) {
    __shared__ float red[kThreads / 32];
    const T* w = static_cast<const T*>(a.w);
    const T* b = static_cast<const T*>(a.b);
    const int C = a.cols;
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * C;
        T* y = static_cast<T*>(a.y) + r * C;
        float s = 0.0f;
        for (int i = threadIdx.x; i < C; i += kThreads) s += to_f(x[i]);
        const float mean = block_sum(s, red) / (float)C;
        s = 0.0f;
        for (int i = threadIdx.x; i < C; i += kThreads) {
            const float d = to_f(x[i]) - mean;
            s += d * d;
        }
        const float rstd = 1.0f / sqrtf(block_sum(s, red) / (float)C + a.eps);
        for (int i = threadIdx.x; i < C; i += kThreads) {
            float v = (to_f(x[i]) - mean) * rstd;
            if (w) v *= to_f(w[i]);
            if (b) v += to_f(b[i]);
            y[i] = from_f<T>(v);
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

// dw and db of one group of rows: 32 columns a block, 8 rows at a time.
// Runs before the dx kernel, which may overwrite grad_y or x.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_cols_kernel(const NormBwdArgs a, int groups) {
    __shared__ float sw[8][33], sb[8][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), wr = threadIdx.x >> 5;
    for (int grp = blockIdx.y; grp < groups; grp += gridDim.y) {
        const long long r0 = a.rows * grp / groups, r1 = a.rows * (grp + 1) / groups;
        float dw = 0.0f, db = 0.0f;
        if (c < a.cols) {
            for (long long r = r0 + wr; r < r1; r += 8) {
                const float g = to_f(static_cast<const T*>(a.gy)[r * a.cols + c]);
                const float x = to_f(static_cast<const T*>(a.x)[r * a.cols + c]);
                dw += g * ((x - a.mean[r]) * a.rstd[r]);
                db += g;
            }
        }
        sw[wr][threadIdx.x & 31] = dw;
        sb[wr][threadIdx.x & 31] = db;
        __syncthreads();
        if (wr == 0 && c < a.cols) {
            for (int i = 1; i < 8; ++i) { dw += sw[i][threadIdx.x]; db += sb[i][threadIdx.x]; }
            a.part[((size_t)grp * 2 + 0) * a.cols + c] = dw;
            a.part[((size_t)grp * 2 + 1) * a.cols + c] = db;
        }
        __syncthreads();
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_dx_kernel(const NormBwdArgs a) {
    __shared__ float red[kThreads / 32];
    const T* w = static_cast<const T*>(a.w);
    const int C = a.cols;
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * C;
        const T* gy = static_cast<const T*>(a.gy) + r * C;
        T* dx = static_cast<T*>(a.dx) + r * C;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s1 = 0.0f, s2 = 0.0f;
        for (int i = threadIdx.x; i < C; i += kThreads) {
            const float g = to_f(gy[i]) * (w ? to_f(w[i]) : 1.0f);
            s1 += g;
            s2 += g * ((to_f(x[i]) - mean) * rstd);
        }
        s1 = block_sum(s1, red) / (float)C;
        s2 = block_sum(s2, red) / (float)C;
        for (int i = threadIdx.x; i < C; i += kThreads) {
            const float g = to_f(gy[i]) * (w ? to_f(w[i]) : 1.0f);
            const float xh = (to_f(x[i]) - mean) * rstd;
            dx[i] = from_f<T>(rstd * (g - s1 - xh * s2));
        }
    }
}

// dw[c], db[c]: the groups' sums added in group order.
__global__ void __launch_bounds__(kThreads) norm_add_kernel(const float* part, int groups, int cols, float* dw,
                                                            float* db) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= cols) return;
    float w = 0.0f, b = 0.0f;
    for (int g = 0; g < groups; ++g) {
        w += part[((size_t)g * 2 + 0) * cols + c];
        b += part[((size_t)g * 2 + 1) * cols + c];
    }
    if (dw) dw[c] = w;
    if (db) db[c] = b;
}

template <typename T>
cudaError_t fwd(const NormFwdArgs& a, cudaStream_t s, int* n) {
    const long long grid = a.rows < 8ll * a.num_sms ? a.rows : 8ll * a.num_sms;
    norm_fwd_kernel<T><<<(int)grid, kThreads, 0, s>>>(a);
    *n = 1;
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const NormBwdArgs& a, cudaStream_t s, int* n) {
    *n = 0;
    cudaError_t e = cudaSuccess;
    if (a.dw || a.db) {
        const int groups = norm_partials(a.rows, a.cols, a.num_sms);
        if (groups > 0) {
            norm_cols_kernel<T><<<dim3((a.cols + 31) / 32, groups), kThreads, 0, s>>>(a, groups);
            ++*n;
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
        }
        norm_add_kernel<<<(a.cols + kThreads - 1) / kThreads, kThreads, 0, s>>>(a.part, groups, a.cols, a.dw, a.db);
        ++*n;
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (a.dx && a.rows > 0) {
        const long long grid = a.rows < 8ll * a.num_sms ? a.rows : 8ll * a.num_sms;
        norm_dx_kernel<T><<<(int)grid, kThreads, 0, s>>>(a);
        ++*n;
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace

int norm_partials(long long rows, int cols, int num_sms) {
    (void)cols;
    return (int)(rows < num_sms ? rows : num_sms);
}

cudaError_t launch_norm_fwd(const void* args, cudaStream_t s, int* nlaunch) {
    const NormFwdArgs& a = *static_cast<const NormFwdArgs*>(args);
    return a.dt == DType::F32 ? fwd<float>(a, s, nlaunch) : fwd<bf16>(a, s, nlaunch);
}

cudaError_t launch_norm_bwd(const void* args, cudaStream_t s, int* nlaunch) {
    const NormBwdArgs& a = *static_cast<const NormBwdArgs*>(args);
    return a.dt == DType::F32 ? bwd<float>(a, s, nlaunch) : bwd<bf16>(a, s, nlaunch);
}

}  // namespace lstm
