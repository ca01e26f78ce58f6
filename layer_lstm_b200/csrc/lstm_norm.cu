// Layer normalisation, forward and backward (Ba, Kiros and Hinton 2016; the
// equations are in include/lstm.h).  A row is two sums, a subtraction and a
// product per element, so HBM bounds it: x in and y out forward; x, grad_y in
// and dx out backward, with the column sums dw, db beside them.
#include <initializer_list>
#include <type_traits>

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

// One block per row, for rows too wide for a block's registers: the row is
// read again for each pass over it.
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

// dw[c], db[c]: the groups' sums, every eighth by one of 8 warps, the warps'
// added in order.
__global__ void __launch_bounds__(kThreads) norm_add_kernel(const float* part, int groups, int cols, float* dw,
                                                            float* db) {
    __shared__ float sw[8][33], sb[8][33];
    const int l = threadIdx.x & 31, wr = threadIdx.x >> 5, c = blockIdx.x * 32 + l;
    float w = 0.0f, b = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int g = wr; g < groups; g += 8) {
            w += part[((size_t)g * 2 + 0) * cols + c];
            b += part[((size_t)g * 2 + 1) * cols + c];
        }
    }
    sw[wr][l] = w;
    sb[wr][l] = b;
    __syncthreads();
    if (wr != 0 || c >= cols) return;
    for (int i = 1; i < 8; ++i) { w += sw[i][l]; b += sb[i][l]; }
    if (dw) dw[c] = w;
    if (db) db[c] = b;
}

// ------------------------------------------------------------ rows in registers
// A row is held by a group of G threads, PER values each, and read once: W
// consecutive values per load (16 bytes, or 1 where rows are not 16-byte
// multiples), loads G * W columns apart.  PER is 16 for packed bf16 and 8
// otherwise: the backward keeps two rows' x and grad_y and two column sums
// in registers, 120 a thread, so that two blocks of 256 share an SM (with 16
// float32 values it takes 165, one block).  A block of
// at least 256 threads takes 256 / G rows at a time and walks the rows with
// the next row's loads issued before the current row's sums, which is what
// keeps HBM busy across the two reductions; weight and bias stay in registers.
template <typename T, int W>
constexpr int per_of() { return sizeof(T) == 2 && W > 1 ? 16 : 8; }

constexpr int block_of(int G) { return G > kThreads ? G : kThreads; }

// W consecutive elements, zeros past the row's end (c is a multiple of W, the
// row's length too).
template <typename T, int W>
struct Vec {
    uint4 q;
    __device__ __forceinline__ void load(const T* p) { q = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
    }
};
template <typename T>
struct Vec<T, 1> {
    T q;
    __device__ __forceinline__ void load(const T* p) { q = *p; }
    __device__ __forceinline__ void zero() { q = from_f<T>(0.0f); }
    __device__ __forceinline__ float get(int) const { return to_f(q); }
};

template <typename T, int W>
__device__ __forceinline__ void store_vec(T* p, const float* v) {
    if constexpr (W == 1) {
        *p = from_f<T>(v[0]);
    } else if constexpr (sizeof(T) == 4) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    }
}

// A group's part of a row (or of weight, bias).
template <typename T, int G, int W>
struct Part {
    static constexpr int NV = per_of<T, W>() / W;
    Vec<T, W> v[NV];
    __device__ __forceinline__ void load(const T* p, int lane, int cols, bool on) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * G + lane) * W;
            if (on && c < cols) v[j].load(p + c);
            else v[j].zero();
        }
    }
    __device__ __forceinline__ float get(int i) const { return v[i / W].get(i % W); }
};

// Sums of N values over each group of G threads, in every thread of it.
// `red` holds two sets of N values per warp, used in turn (`flip`), so one
// barrier per sum is enough.
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* red, int& flip) {
#pragma unroll
    for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (G > 32) {
        constexpr int kWarps = block_of(G) / 32, kOf = G / 32;
        float* r = red + flip * kWarps * N;
        flip ^= 1;
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) r[warp * N + i] = v[i];
        __syncthreads();
        const int first = warp / kOf * kOf;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.0f;
#pragma unroll
            for (int k = 0; k < kOf; ++k) v[i] += r[(first + k) * N + i];
        }
    }
}

template <typename T, int G, int W>
__global__ void __launch_bounds__(block_of(G), 1024 / block_of(G)) norm_fwd_rows_kernel(const NormFwdArgs a) {
    constexpr int kPer = per_of<T, W>();
    constexpr int RPB = block_of(G) / G;
    __shared__ float red[2 * block_of(G) / 32];
    int flip = 0;
    const int lane = threadIdx.x % G, grp = threadIdx.x / G;
    const int C = a.cols;
    const float inv = 1.0f / (float)C;
    Part<T, G, W> w, b, x, nx;
    w.load(static_cast<const T*>(a.w), lane, C, a.w != nullptr);
    b.load(static_cast<const T*>(a.b), lane, C, a.b != nullptr);
    const long long step = (long long)gridDim.x * RPB;
    long long r = (long long)blockIdx.x * RPB + grp;
    const T* X = static_cast<const T*>(a.x);
    nx.load(X + r * C, lane, C, r < a.rows);
    for (long long r0 = (long long)blockIdx.x * RPB; r0 < a.rows; r0 += step, r += step) {
        const bool on = r < a.rows;
        x = nx;
        nx.load(X + (r + step) * C, lane, C, r + step < a.rows);
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kPer; ++i) s[0] += x.get(i);
        group_sum<G>(s, red, flip);
        const float mean = s[0] * inv;
        s[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = ((i / W) * G + lane) * W;
            const float d = x.get(i) - mean;
            if (c < C) s[0] = fmaf(d, d, s[0]);
        }
        group_sum<G>(s, red, flip);
        const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
        if (on) {
            T* y = static_cast<T*>(a.y) + r * C;
#pragma unroll
            for (int j = 0; j < kPer / W; ++j) {
                const int c = (j * G + lane) * W;
                if (c >= C) continue;
                float o[W];
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    o[i] = (x.get(j * W + i) - mean) * rstd;
                    if (a.w) o[i] *= w.get(j * W + i);
                    if (a.b) o[i] += b.get(j * W + i);
                }
                store_vec<T, W>(y + c, o);
            }
            if (lane == 0) {
                if (a.mean) a.mean[r] = mean;
                if (a.rstd) a.rstd[r] = rstd;
            }
        }
    }
}

// dx, and the block's sums of dw and db over its rows: every thread keeps the
// sums of its own 16 columns in registers, the groups are added at the end.
template <typename T, int G, int W>
__global__ void __launch_bounds__(block_of(G), 512 / block_of(G)) norm_bwd_rows_kernel(const NormBwdArgs a) {
    constexpr int kPer = per_of<T, W>();
    constexpr int RPB = block_of(G) / G;
    __shared__ float red[4 * block_of(G) / 32];
    __shared__ float part[RPB > 1 ? kPer * block_of(G) : 1];
    int flip = 0;
    const int lane = threadIdx.x % G, grp = threadIdx.x / G;
    const int C = a.cols;
    const float inv = 1.0f / (float)C;
    const bool sums = a.dw != nullptr || a.db != nullptr;
    Part<T, G, W> w, x, g, nx, ng;
    w.load(static_cast<const T*>(a.w), lane, C, a.w != nullptr);
    float dw[kPer] = {}, db[kPer] = {};
    const long long step = (long long)gridDim.x * RPB;
    long long r = (long long)blockIdx.x * RPB + grp;
    const T* X = static_cast<const T*>(a.x);
    const T* Y = static_cast<const T*>(a.gy);
    float nmean = 0.0f, nrstd = 0.0f;
    nx.load(X + r * C, lane, C, r < a.rows);
    ng.load(Y + r * C, lane, C, r < a.rows);
    if (r < a.rows) { nmean = a.mean[r]; nrstd = a.rstd[r]; }
    for (long long r0 = (long long)blockIdx.x * RPB; r0 < a.rows; r0 += step, r += step) {
        const bool on = r < a.rows;
        x = nx; g = ng;
        const float mean = nmean, rstd = nrstd;
        const bool more = r + step < a.rows;
        nx.load(X + (r + step) * C, lane, C, more);
        ng.load(Y + (r + step) * C, lane, C, more);
        if (more) { nmean = a.mean[r + step]; nrstd = a.rstd[r + step]; }
        float s[2] = {0.0f, 0.0f};
        if (on) {   // past the last row there is nothing to sum (0 times a stale mean could be NaN)
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int c = ((i / W) * G + lane) * W;
                const float gy = g.get(i), xh = (x.get(i) - mean) * rstd;
                if (c < C) {
                    dw[i] = fmaf(gy, xh, dw[i]);
                    db[i] += gy;
                    const float gw = a.w ? gy * w.get(i) : gy;
                    s[0] += gw;
                    s[1] = fmaf(gw, xh, s[1]);
                }
            }
        }
        if (a.dx) {
            group_sum<G>(s, red, flip);
            const float s1 = s[0] * inv, s2 = s[1] * inv;
            if (on) {
                T* dx = static_cast<T*>(a.dx) + r * C;
#pragma unroll
                for (int j = 0; j < kPer / W; ++j) {
                    const int c = (j * G + lane) * W;
                    if (c >= C) continue;
                    float o[W];
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const float gy = g.get(j * W + i), xh = (x.get(j * W + i) - mean) * rstd;
                        o[i] = rstd * ((a.w ? gy * w.get(j * W + i) : gy) - s1 - xh * s2);
                    }
                    store_vec<T, W>(dx + c, o);
                }
            }
        }
    }
    if (!sums) return;
    float* out = a.part + (size_t)blockIdx.x * 2 * C;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float* v = k ? db : dw;
        if constexpr (RPB > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kPer; ++i) part[(i * RPB + grp) * G + lane] = v[i];
            __syncthreads();
            // column (i, lane): its RPB groups' sums in group order
            for (int t = threadIdx.x; t < kPer * G; t += block_of(G)) {
                const int i = t / G, l = t % G, c = ((i / W) * G + l) * W + i % W;
                if (c >= C) continue;
                float sum = 0.0f;
#pragma unroll 4
                for (int q = 0; q < RPB; ++q) sum += part[(i * RPB + q) * G + l];
                out[(size_t)k * C + c] = sum;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int c = ((i / W) * G + lane) * W + i % W;
                if (c < C) out[(size_t)k * C + c] = v[i];
            }
        }
    }
}

// Group width for `cols` columns at `per` a thread, or 0 when a row does not
// fit a block.
int group_of(int cols, int per) {
    for (int g = 4; g <= 512; g *= 2)
        if (cols <= g * per) return g;
    return 0;
}

// Blocks for `rows` rows: enough threads on every SM for `threads` of them.
long long row_blocks(long long rows, int group, int threads, int num_sms) {
    const int rpb = block_of(group) / group;
    const long long need = (rows + rpb - 1) / rpb, most = (long long)(threads / block_of(group)) * num_sms;
    return need < most ? need : most;
}
constexpr int kFwdThreads = 1024, kBwdThreads = 512;   // per SM, as the launch bounds say

template <typename F>
bool with_group(int group, F&& f) {
    switch (group) {
        case 4: f(std::integral_constant<int, 4>{}); return true;
        case 8: f(std::integral_constant<int, 8>{}); return true;
        case 16: f(std::integral_constant<int, 16>{}); return true;
        case 32: f(std::integral_constant<int, 32>{}); return true;
        case 64: f(std::integral_constant<int, 64>{}); return true;
        case 128: f(std::integral_constant<int, 128>{}); return true;
        case 256: f(std::integral_constant<int, 256>{}); return true;
        case 512: f(std::integral_constant<int, 512>{}); return true;
        default: return false;
    }
}

// 16-byte loads need rows and pointers on 16 bytes.
template <typename T>
bool wide(int cols, std::initializer_list<const void*> ps) {
    if (cols % (16 / (int)sizeof(T)) != 0) return false;
    for (const void* p : ps)
        if ((uintptr_t)p & 15) return false;
    return true;
}

template <typename T, int W>
bool fwd_rows(const NormFwdArgs& a, cudaStream_t s) {
    return with_group(group_of(a.cols, per_of<T, W>()), [&](auto g) {
        constexpr int G = decltype(g)::value;
        norm_fwd_rows_kernel<T, G, W><<<(int)row_blocks(a.rows, G, kFwdThreads, a.num_sms), block_of(G), 0, s>>>(a);
    });
}

// *groups: blocks, each of which leaves its sums of dw and db.
template <typename T, int W>
bool bwd_rows(const NormBwdArgs& a, cudaStream_t s, int* groups) {
    return with_group(group_of(a.cols, per_of<T, W>()), [&](auto g) {
        constexpr int G = decltype(g)::value;
        *groups = (int)row_blocks(a.rows, G, kBwdThreads, a.num_sms);
        norm_bwd_rows_kernel<T, G, W><<<*groups, block_of(G), 0, s>>>(a);
    });
}

template <typename T>
cudaError_t fwd(const NormFwdArgs& a, cudaStream_t s, int* n) {
    *n = 1;
    constexpr int W = 16 / sizeof(T);
    const bool done = wide<T>(a.cols, {a.x, a.y, a.w, a.b}) ? fwd_rows<T, W>(a, s) : fwd_rows<T, 1>(a, s);
    if (!done) {
        const long long grid = a.rows < 8ll * a.num_sms ? a.rows : 8ll * a.num_sms;
        norm_fwd_kernel<T><<<(int)grid, kThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const NormBwdArgs& a, cudaStream_t s, int* n) {
    *n = 0;
    cudaError_t e = cudaSuccess;
    constexpr int W = 16 / sizeof(T);
    int groups = (int)(a.rows < a.num_sms ? a.rows : a.num_sms);
    bool rows = false;
    if (a.rows > 0) {
        rows = wide<T>(a.cols, {a.gy, a.x, a.w, a.dx}) ? bwd_rows<T, W>(a, s, &groups) : bwd_rows<T, 1>(a, s, &groups);
        if (rows) ++*n;
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (a.dw || a.db) {
        if (groups > 0 && !rows) {
            norm_cols_kernel<T><<<dim3((a.cols + 31) / 32, groups), kThreads, 0, s>>>(a, groups);
            ++*n;
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
        }
        norm_add_kernel<<<(a.cols + 31) / 32, kThreads, 0, s>>>(a.part, groups, a.cols, a.dw, a.db);
        ++*n;
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (a.dx && a.rows > 0 && !rows) {
        const long long grid = a.rows < 8ll * a.num_sms ? a.rows : 8ll * a.num_sms;
        norm_dx_kernel<T><<<(int)grid, kThreads, 0, s>>>(a);
        ++*n;
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace

int norm_partials(long long rows, int cols, int num_sms) {
    // the most that any of the backward's kernels leaves for this size; which
    // one runs depends on the pointers too
    long long n = rows < num_sms ? rows : num_sms;
    for (int per : {8, 16}) {
        const int g = group_of(cols, per);
        if (g == 0) continue;
        const long long r = row_blocks(rows, g, kBwdThreads, num_sms);
        n = r > n ? r : n;
    }
    return (int)n;
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
