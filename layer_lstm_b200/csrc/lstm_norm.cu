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

// One block per row, for rows too wide for a block's registers (from 16385
// columns in bf16, 8193 in float32, 4097 where rows are not 16-byte multiples):
// the row is read again for each pass over it, an element a thread, mostly from
// L2.  1024 x 32768 bf16: 88 us forward (1.5 TB/s), 427 backward (0.5); 4096 x
// 4097: 36 and 99.
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

// dw[c] (blockIdx.y 0) or db[c]: the groups' sums, every 32nd by one of 32
// warps, the warps' added in order.  A programmatic dependent of the kernel
// that leaves the sums.
constexpr int kAddThreads = 1024;
__global__ void __launch_bounds__(kAddThreads) norm_add_kernel(const float* part, int groups, int cols, float* dw,
                                                               float* db) {
    __shared__ float sums[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float* out = blockIdx.y ? db : dw;
    if (!out) return;
    const int l = threadIdx.x & 31, wr = threadIdx.x >> 5, c = blockIdx.x * 32 + l;
    float v = 0.0f;
    if (c < cols) {
#pragma unroll 4
        for (int g = wr; g < groups; g += 32) v += part[((size_t)g * 2 + blockIdx.y) * cols + c];
    }
    sums[wr][l] = v;
    __syncthreads();
    if (wr != 0 || c >= cols) return;
#pragma unroll
    for (int i = 1; i < 32; ++i) v += sums[i][l];
    out[c] = v;
}

// ------------------------------------------------------------ rows in registers
// A row is held by a group of G threads, PER values each, and read once: W
// consecutive values per load (16 bytes, or 1 where rows are not 16-byte
// multiples), loads G * W columns apart.  PER is 64 bytes of packed elements (8
// elements otherwise): what a row costs beside its elements, some 120
// instructions of sums over the group, root and addresses, is then a third of
// it.  (With 32 bytes, 8192 x 2048 bf16 forward and backward took 47 us instead
// of 40.)  The backward keeps a row and two column sums in registers, one block
// of 256 an SM; the forward two.  A block of at least 256 threads takes 256 / G
// rows at a time.  Blocks of 512 threads have 128 registers each: the backward
// of the widest bf16 rows, 8193 to 16384 columns, spills (1024 x 16384: 71 us,
// 1.4 TB/s; 8192 x 2048: 32 us, 3.2 TB/s).
template <typename T, int W>
constexpr int per_of() { return W == 1 ? 8 : sizeof(T) == 2 ? 32 : 16; }

constexpr int kFwdThreads = 512, kBwdThreads = 256;   // per SM, with their registers
constexpr int block_of(int G) { return G > kThreads ? G : kThreads; }

// Two float32 values in one register pair: sm_100a adds, multiplies and fuses
// them in one instruction, which is what keeps the arithmetic (a fifth of the
// issue slots otherwise spent) out of HBM's way.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f2 both(float a) { return pair(a, a); }
__device__ __forceinline__ void split(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum2(f2 v) {
    float a, b;
    split(v, a, b);
    return a + b;
}

// A group's part of a row as it is stored: PER elements, loads of W.
template <typename T, int G, int W, int PER>
struct Part {
    static constexpr int NV = PER / W, NP = PER / 2;
    uint4 q[W > 1 ? NV : 1];
    T e[W > 1 ? 1 : NV];

    __device__ __forceinline__ void load(const T* p, int lane, int cols, bool on, float fill) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * G + lane) * W;
            const bool in = on && c < cols;
            if constexpr (W > 1) {
                if (in) q[j] = __ldg(reinterpret_cast<const uint4*>(p + c));
                else if constexpr (sizeof(T) == 4) q[j] = fill_of(__float_as_uint(fill));
                else q[j] = fill_of((__float_as_uint(fill) >> 16) * 0x10001u);
            } else {
                e[j] = in ? p[c] : from_f<T>(fill);
            }
        }
    }
    static __device__ __forceinline__ uint4 fill_of(uint32_t w) { return make_uint4(w, w, w, w); }
    // Elements 2 i and 2 i + 1.
    __device__ __forceinline__ f2 get(int i) const {
        if constexpr (W == 1) {
            return pair(to_f(e[2 * i]), to_f(e[2 * i + 1]));
        } else if constexpr (sizeof(T) == 4) {
            const uint4 v = q[i / 2];
            return i & 1 ? pair(__uint_as_float(v.z), __uint_as_float(v.w)) : pair(__uint_as_float(v.x), __uint_as_float(v.y));
        } else {
            const uint4 v = q[i / 4];
            const uint32_t w = (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
            return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
        }
    }
    // Stores values v where columns exist.
    static __device__ __forceinline__ void store(T* p, int lane, int cols, const f2 (&v)[NP]) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * G + lane) * W;
            if (c >= cols) continue;
            if constexpr (W == 1) {
                float a, b;
                split(v[j / 2], a, b);
                p[c] = from_f<T>(j & 1 ? b : a);
            } else if constexpr (sizeof(T) == 4) {
                float4 o;
                split(v[2 * j], o.x, o.y);
                split(v[2 * j + 1], o.z, o.w);
                *reinterpret_cast<float4*>(p + c) = o;
            } else {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a, b;
                    split(v[4 * j + i], a, b);
                    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
                    w[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
                *reinterpret_cast<uint4*>(p + c) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    // Zeros in the places past the row's end.
    static __device__ __forceinline__ void clear(int lane, int cols, f2 (&v)[NP]) {
        if (cols == G * PER) return;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if ((j * G + lane) * W < cols) continue;
            if constexpr (W == 1) {
                float a, b;
                split(v[j / 2], a, b);
                v[j / 2] = j & 1 ? pair(a, 0.0f) : pair(0.0f, b);
            } else {
#pragma unroll
                for (int i = 0; i < W / 2; ++i) v[j * (W / 2) + i] = 0;
            }
        }
    }
};

// The rows ahead of the current one, in shared memory: every thread copies
// (cp.async) and reads back only its own part, so no barrier is involved, and
// three rows of a group (one of the widest, by shared memory's size) are in
// flight without a register.  (HBM's latency times an SM's share of its rate is
// some 50 KB.)  Rows that 16-byte copies cannot take (W = 1) keep one row ahead
// in registers.
constexpr int ahead_of(int G) { return G > kThreads ? 1 : 3; }

template <typename T, int G, int W, int PER, int ARRAYS>
struct Ring {
    static constexpr int NV = PER / W, THREADS = block_of(G), AHEAD = ahead_of(G);
    static constexpr size_t BYTES = W > 1 ? (size_t)(AHEAD + 1) * ARRAYS * NV * THREADS * 16 : 0;
    uint4* slots;   // [AHEAD + 1][ARRAYS][NV][THREADS]
    Part<T, G, W, PER> next[W > 1 ? 1 : ARRAYS];

    __device__ __forceinline__ uint4* slot(int stage, int a, int j) const {
        return slots + ((stage * ARRAYS + a) * NV + j) * THREADS + threadIdx.x;
    }
    // Array a's part of a row, to stage `stage` (W = 1: to registers).
    __device__ __forceinline__ void issue(int stage, int a, const T* p, int lane, int cols, bool on) {
        if constexpr (W > 1) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * G + lane) * W;
                if (on && c < cols)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                     (uint32_t)__cvta_generic_to_shared(slot(stage, a, j))),
                                 "l"(p + c)
                                 : "memory");
            }
        } else {
            next[a].load(p, lane, cols, on, 0.0f);
        }
    }
    __device__ __forceinline__ void commit() const {
        if constexpr (W > 1) asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // All but the newest AHEAD - 1 rows have landed.
    __device__ __forceinline__ void wait() const {
        if constexpr (W > 1) asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
    }
    __device__ __forceinline__ void take(int stage, int a, int lane, int cols, Part<T, G, W, PER>& x) const {
        if constexpr (W > 1) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                x.q[j] = (j * G + lane) * W < cols ? *slot(stage, a, j) : make_uint4(0, 0, 0, 0);
            }
        } else {
            x = next[a];
        }
    }
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
__global__ void __launch_bounds__(block_of(G), kFwdThreads / block_of(G)) norm_fwd_rows_kernel(const NormFwdArgs a) {
    constexpr int PER = per_of<T, W>();
    using P = Part<T, G, W, PER>;
    constexpr int RPB = block_of(G) / G;
    __shared__ float red[2 * block_of(G) / 32];
    int flip = 0;
    const int lane = threadIdx.x % G, grp = threadIdx.x / G;
    const int C = a.cols;
    const float inv = 1.0f / (float)C;
    constexpr int AHEAD = ahead_of(G), kRows = W > 1 ? AHEAD : 1;
    extern __shared__ uint4 ring_slots[];
    Ring<T, G, W, PER, 1> ring;
    ring.slots = ring_slots;
    P w, b, x;
    const long long step = (long long)gridDim.x * RPB;
    long long r = (long long)blockIdx.x * RPB + grp;
    const T* X = static_cast<const T*>(a.x);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        ring.issue(k, 0, X + (r + k * step) * C, lane, C, r + k * step < a.rows);
        ring.commit();
    }
    w.load(static_cast<const T*>(a.w), lane, C, a.w != nullptr, 1.0f);
    b.load(static_cast<const T*>(a.b), lane, C, a.b != nullptr, 0.0f);
    int stage = 0;
    for (long long r0 = (long long)blockIdx.x * RPB; r0 < a.rows; r0 += step, r += step) {
        const bool on = r < a.rows;
        ring.wait();
        ring.take(stage, 0, lane, C, x);
        // (the stage before this one: what it held has been read)
        const int behind = stage == 0 ? AHEAD : stage - 1;
        ring.issue(behind, 0, X + (r + kRows * step) * C, lane, C, r + kRows * step < a.rows);
        ring.commit();
        stage = stage == AHEAD ? 0 : stage + 1;
        f2 d[P::NP], acc = 0;
#pragma unroll
        for (int i = 0; i < P::NP; ++i) {
            d[i] = x.get(i);
            acc = add2(acc, d[i]);
        }
        float s[1] = {sum2(acc)};
        group_sum<G>(s, red, flip);
        const float mean = s[0] * inv;
        const f2 minus = both(-mean);
#pragma unroll
        for (int i = 0; i < P::NP; ++i) d[i] = add2(d[i], minus);
        P::clear(lane, C, d);
        acc = 0;
#pragma unroll
        for (int i = 0; i < P::NP; ++i) acc = fma2(d[i], d[i], acc);
        s[0] = sum2(acc);
        group_sum<G>(s, red, flip);
        const float rstd = rsqrtf(s[0] * inv + a.eps);
        if (on) {
            const f2 scale = both(rstd);
#pragma unroll
            for (int i = 0; i < P::NP; ++i) d[i] = fma2(mul2(d[i], scale), w.get(i), b.get(i));
            P::store(static_cast<T*>(a.y) + r * C, lane, C, d);
            if (lane == 0) {
                if (a.mean) a.mean[r] = mean;
                if (a.rstd) a.rstd[r] = rstd;
            }
        }
    }
}

// dx, and the block's sums of dw and db over its rows: every thread keeps the
// sums of its own kPer columns in registers, the groups are added at the end.
template <typename T, int G, int W>
__global__ void __launch_bounds__(block_of(G), 1) norm_bwd_rows_kernel(const NormBwdArgs a) {
    constexpr int kPer = per_of<T, W>();
    using P = Part<T, G, W, kPer>;
    constexpr int RPB = block_of(G) / G;
    __shared__ float red[4 * block_of(G) / 32];
    __shared__ float part[RPB > 1 ? kPer * block_of(G) : 1];
    int flip = 0;
    const int lane = threadIdx.x % G, grp = threadIdx.x / G;
    const int C = a.cols;
    const float inv = 1.0f / (float)C;
    const bool sums = a.dw != nullptr || a.db != nullptr;
    constexpr int AHEAD = ahead_of(G), kRows = W > 1 ? AHEAD : 1;
    extern __shared__ uint4 ring_slots[];
    Ring<T, G, W, kPer, 2> ring;
    ring.slots = ring_slots;
    P w, x, g;
    f2 dw[P::NP] = {}, db[P::NP] = {};
    const long long step = (long long)gridDim.x * RPB;
    long long r = (long long)blockIdx.x * RPB + grp;
    const T* X = static_cast<const T*>(a.x);
    const T* Y = static_cast<const T*>(a.gy);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        ring.issue(k, 0, X + (r + k * step) * C, lane, C, r + k * step < a.rows);
        ring.issue(k, 1, Y + (r + k * step) * C, lane, C, r + k * step < a.rows);
        ring.commit();
    }
    w.load(static_cast<const T*>(a.w), lane, C, a.w != nullptr, 1.0f);
    float nmean = 0.0f, nrstd = 0.0f;
    if (r < a.rows) { nmean = a.mean[r]; nrstd = a.rstd[r]; }
    int stage = 0;
    for (long long r0 = (long long)blockIdx.x * RPB; r0 < a.rows; r0 += step, r += step) {
        const bool on = r < a.rows;
        const float mean = nmean, rstd = nrstd;
        if (r + step < a.rows) { nmean = a.mean[r + step]; nrstd = a.rstd[r + step]; }
        ring.wait();
        ring.take(stage, 0, lane, C, x);
        ring.take(stage, 1, lane, C, g);
        const int behind = stage == 0 ? AHEAD : stage - 1;
        const bool more = r + kRows * step < a.rows;
        ring.issue(behind, 0, X + (r + kRows * step) * C, lane, C, more);
        ring.issue(behind, 1, Y + (r + kRows * step) * C, lane, C, more);
        ring.commit();
        stage = stage == AHEAD ? 0 : stage + 1;
        f2 xh[P::NP], gw[P::NP], s1 = 0, s2 = 0;
        const f2 scale = both(rstd), minus = both(-mean);
        if (on) {   // past the last row there is nothing to sum
#pragma unroll
            for (int i = 0; i < P::NP; ++i) {
                const f2 gy = g.get(i);
                xh[i] = mul2(add2(x.get(i), minus), scale);
                dw[i] = fma2(gy, xh[i], dw[i]);
                db[i] = add2(db[i], gy);
                gw[i] = mul2(gy, w.get(i));
                s1 = add2(s1, gw[i]);
                s2 = fma2(gw[i], xh[i], s2);
            }
        }
        if (a.dx) {
            float s[2] = {sum2(s1), sum2(s2)};
            group_sum<G>(s, red, flip);
            if (on) {
                const f2 m1 = both(-s[0] * inv), m2 = both(-s[1] * inv);
#pragma unroll
                for (int i = 0; i < P::NP; ++i) gw[i] = mul2(scale, fma2(xh[i], m2, add2(gw[i], m1)));
                P::store(static_cast<T*>(a.dx) + r * C, lane, C, gw);
            }
        }
    }
    if (!sums) return;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // norm_add_kernel sets off
    float* out = a.part + (size_t)blockIdx.x * 2 * C;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float v[kPer];
#pragma unroll
        for (int i = 0; i < P::NP; ++i) split(k ? db[i] : dw[i], v[2 * i], v[2 * i + 1]);
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

// Blocks for `rows` rows: at most `threads` threads (one block) on every SM.
long long row_blocks(long long rows, int group, int threads, int num_sms) {
    const int rpb = block_of(group) / group;
    const long long need = (rows + rpb - 1) / rpb, most = (long long)(threads >= block_of(group) ? threads / block_of(group) : 1) * num_sms;
    return need < most ? need : most;
}

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
        constexpr size_t bytes = Ring<T, G, W, per_of<T, W>(), 1>::BYTES;
        if (bytes > 16 * 1024)   // with the static part it may pass 48 KB
            cudaFuncSetAttribute(norm_fwd_rows_kernel<T, G, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        norm_fwd_rows_kernel<T, G, W><<<(int)row_blocks(a.rows, G, kFwdThreads, a.num_sms), block_of(G), bytes, s>>>(a);
    });
}

// *groups: blocks, each of which leaves its sums of dw and db.
template <typename T, int W>
bool bwd_rows(const NormBwdArgs& a, cudaStream_t s, int* groups) {
    return with_group(group_of(a.cols, per_of<T, W>()), [&](auto g) {
        constexpr int G = decltype(g)::value;
        *groups = (int)row_blocks(a.rows, G, kBwdThreads, a.num_sms);
        constexpr size_t bytes = Ring<T, G, W, per_of<T, W>(), 2>::BYTES;
        if (bytes > 16 * 1024)   // with the static part it may pass 48 KB
            cudaFuncSetAttribute(norm_bwd_rows_kernel<T, G, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        norm_bwd_rows_kernel<T, G, W><<<*groups, block_of(G), bytes, s>>>(a);
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
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((a.cols + 31) / 32, 2);
        cfg.blockDim = dim3(kAddThreads);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, norm_add_kernel, (const float*)a.part, groups, a.cols, a.dw, a.db);
        ++*n;
        if (e != cudaSuccess) return e;
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
    for (int per : {8, 16, 32}) {
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
