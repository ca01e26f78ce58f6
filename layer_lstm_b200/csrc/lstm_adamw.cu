// AdamW over every tensor of a model in one launch (Loshchilov and Hutter
// 2019, "Decoupled Weight Decay Regularization"), moments in float32 or in 8
// bits.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v / (1 - b2^t)) + eps).
//
// The step moves 28 bytes per element with float32 moments and gradients, 18
// with 8-bit moments and a bf16 copy of p, for some 20 or 80 operations: HBM
// bounds it.  The tensors' table travels in the kernel's parameters, so a
// call needs no copy to the device and can be captured into a graph.
//
// Every operation below is rounded on its own (no contraction to FMA): the
// 8-bit codes depend on the last bit of what is encoded, and with one order
// of roundings they are a function of the inputs that does not move with the
// compiler's choices.
#include "lstm_device.cuh"
#include "lstm_ops.h"

namespace lstm {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 2048;   // elements a block takes at a time: one block of 256 moments per warp

struct Table {
    AdamwTensor t[kAdamwTensors];
    long long tile_end[kAdamwTensors];   // tiles of tensors 0..i
    uint8_t vec[kAdamwTensors];          // every pointer allows 4-element accesses
    int count, first;
};

struct Params {
    Table tab;
    double lr, beta1, beta2, wd;
    float b1, b2, c1, c2, eps;
    uint64_t seed;
    const long long* step;
    const float* scalars;
};

// A permutation of 32-bit words whose outputs pass for random (Jarzynski and
// Olano 2020, "Hash Functions for GPU Rendering", PCG): one word per element.
__device__ __forceinline__ uint32_t pcg(uint32_t x) {
    const uint32_t s = x * 747796405u + 2891336453u;
    const uint32_t w = ((s >> ((s >> 28) + 4u)) ^ s) * 277803737u;
    return (w >> 22) ^ w;
}

// Code c of a first moment stands for sign (c / 127)^2 a, of a second for
// (c / 255)^4 a, with a the largest magnitude of the element's block of 256.
// The codes are dense where the values are small next to the block's largest:
// the smallest nonzero first moment is 6e-5 a, second moment 2e-10 a.
__device__ __forceinline__ float decode_m(int c, float a) {
    const float q = __fmul_rn((float)c, 1.0f / 127.0f);
    return __fmul_rn(__fmul_rn(fabsf(q), q), a);
}
__device__ __forceinline__ float decode_v(int c, float a) {
    const float q = __fmul_rn((float)c, 1.0f / 255.0f);
    const float q2 = __fmul_rn(q, q);
    return __fmul_rn(__fmul_rn(q2, q2), a);
}

// Rounds up with the probability that keeps the mean of the value the code
// stands for: rounding to the nearest code would hold a second moment still
// for as long as a step changes it by less than half a code, which at
// b2 = 0.999 is nearly always.  z = |x| / a; u random in [0, 1).
__device__ __forceinline__ int encode_m(float z, float u) {
    const float X = __fmul_rn(z, 16129.0f);
    float c = floorf(__fsqrt_rn(X));
    const float lo = __fmul_rn(c, c), c1 = __fadd_rn(c, 1.0f), hi = __fmul_rn(c1, c1);
    if (__fmul_rn(u, __fsub_rn(hi, lo)) < __fsub_rn(X, lo)) c = c1;
    return (int)fminf(c, 127.0f);
}
// A second moment that is not zero keeps a code of at least 1: a zero under
// the root would let the next step divide by eps alone.
__device__ __forceinline__ int encode_v(float z, float u) {
    const float X = __fmul_rn(z, 4228250625.0f);
    float c = floorf(__fsqrt_rn(__fsqrt_rn(X)));
    const float c1 = __fadd_rn(c, 1.0f);
    const float lo2 = __fmul_rn(c, c), hi2 = __fmul_rn(c1, c1);
    const float lo = __fmul_rn(lo2, lo2), hi = __fmul_rn(hi2, hi2);
    if (__fmul_rn(u, __fsub_rn(hi, lo)) < __fsub_rn(X, lo)) c = c1;
    if (X > 0.0f) c = fmaxf(c, 1.0f);
    return (int)fminf(c, 255.0f);
}

struct Coef {
    float size, root, keep, gs;   // lr / (1 - b1^t), 1 / sqrt(1 - b2^t), 1 - lr wd, gradient factor
    uint32_t k1;                  // random key of (seed, step)
};

__device__ __forceinline__ Coef make_coef(const Params& P) {
    const long long t = *P.step + 1;
    double lr = P.lr;
    Coef c;
    c.gs = 1.0f;
    if (P.scalars) {
        lr *= (double)P.scalars[0];
        c.gs = P.scalars[1];
    }
    c.size = (float)(lr / (1.0 - pow(P.beta1, (double)t)));
    c.root = (float)(1.0 / sqrt(1.0 - pow(P.beta2, (double)t)));
    c.keep = (float)(1.0 - lr * P.wd);
    c.k1 = pcg((uint32_t)t ^ pcg((uint32_t)P.seed ^ pcg((uint32_t)(P.seed >> 32))));
    return c;
}

__device__ __forceinline__ void update(float& p, float g, float& m, float& v, const Params& P, const Coef& c) {
    g = __fmul_rn(g, c.gs);
    m = __fadd_rn(__fmul_rn(m, P.b1), __fmul_rn(g, P.c1));
    v = __fadd_rn(__fmul_rn(v, P.b2), __fmul_rn(__fmul_rn(g, g), P.c2));
    const float den = __fadd_rn(__fmul_rn(__fsqrt_rn(v), c.root), P.eps);
    p = __fsub_rn(__fmul_rn(p, c.keep), __fmul_rn(c.size, __fdiv_rn(m, den)));
}

// Four elements from e (e < n), as float; zeros past the end.
template <typename T>
__device__ __forceinline__ void get4(const T* x, long long e, long long n, bool vec, float (&v)[4]) {
    if (vec && e + 4 <= n) {
        load4(x + e, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = e + i < n ? to_f(x[e + i]) : 0.0f;
    }
}
template <typename C>
__device__ __forceinline__ void get_codes(const C* x, long long e, long long n, bool vec, int (&v)[4]) {
    if (vec && e + 4 <= n) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(x + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (int)(C)(w >> (8 * i));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = e + i < n ? (int)x[e + i] : 0;
    }
}
__device__ __forceinline__ void put4(float* x, long long e, long long n, bool vec, const float (&v)[4]) {
    if (vec && e + 4 <= n) {
        *reinterpret_cast<float4*>(x + e) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e + i < n) x[e + i] = v[i];
    }
}
// The copy is rounded to nearest even; p itself stays float32.
__device__ __forceinline__ void put4(bf16* x, long long e, long long n, bool vec, const float (&v)[4]) {
    if (vec && e + 4 <= n) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(x + e) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                      *reinterpret_cast<const uint32_t*>(&b));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e + i < n) x[e + i] = __float2bfloat16_rn(v[i]);
    }
}
__device__ __forceinline__ void put_codes(uint8_t* x, long long e, long long n, bool vec, const int (&v)[4]) {
    if (vec && e + 4 <= n) {
        *reinterpret_cast<uint32_t*>(x + e) = (uint32_t)(v[0] & 255) | (uint32_t)(v[1] & 255) << 8 |
                                              (uint32_t)(v[2] & 255) << 16 | (uint32_t)(v[3] & 255) << 24;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e + i < n) x[e + i] = (uint8_t)v[i];
    }
}

// Tensor of tile `t`: the first whose tile_end exceeds it.
__device__ __forceinline__ int find_tensor(const Table& tab, long long t) {
    int lo = 0, hi = tab.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (tab.tile_end[mid] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Largest value of the warp; NaN if any lane holds one.
__device__ __forceinline__ float warp_max_nan(float a) {
    bool bad = !(a == a);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    return __any_sync(0xffffffffu, bad) ? __int_as_float(0x7fc00000) : a;
}

template <typename G, int BITS>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Params P) {
    __shared__ Coef coef;
    if (threadIdx.x == 0) coef = make_coef(P);
    __syncthreads();
    const Coef c = coef;
    const Table& tab = P.tab;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long tiles = tab.tile_end[tab.count - 1];
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int ti = find_tensor(tab, tile);
        const AdamwTensor& t = tab.t[ti];
        const bool vec = tab.vec[ti] != 0;
        const long long base = (tile - (ti ? tab.tile_end[ti - 1] : 0)) * kTile + warp * kAdamwBlock;
        const long long n = t.n;
        if (base >= n) continue;   // the whole warp: base is the warp's
        const G* g = static_cast<const G*>(t.g);
        float p[2][4], gg[2][4], m[2][4], v[2][4];
        const long long e0 = base + lane * 4;
        if constexpr (BITS == 8) {
            const long long blk = base / kAdamwBlock;
            const float ams = t.ms[blk], avs = t.vs[blk];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                int cm[4], cv[4];
                get_codes(static_cast<const int8_t*>(t.m), e0 + j * 128, n, vec, cm);
                get_codes(static_cast<const uint8_t*>(t.v), e0 + j * 128, n, vec, cv);
#pragma unroll
                for (int i = 0; i < 4; ++i) { m[j][i] = decode_m(cm[i], ams); v[j][i] = decode_v(cv[i], avs); }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                get4(static_cast<const float*>(t.m), e0 + j * 128, n, vec, m[j]);
                get4(static_cast<const float*>(t.v), e0 + j * 128, n, vec, v[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            get4(t.p, e0 + j * 128, n, vec, p[j]);
            get4(g, e0 + j * 128, n, vec, gg[j]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                update(p[j][i], gg[j][i], m[j][i], v[j][i], P, c);
                // past the end nothing counts towards the block's scale
                if (BITS == 8 && e0 + j * 128 + i >= n) m[j][i] = v[j][i] = 0.0f;
            }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            put4(t.p, e0 + j * 128, n, vec, p[j]);
            if (t.copy) put4(static_cast<bf16*>(t.copy), e0 + j * 128, n, vec, p[j]);
        }
        if constexpr (BITS == 32) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                put4(static_cast<float*>(t.m), e0 + j * 128, n, vec, m[j]);
                put4(static_cast<float*>(t.v), e0 + j * 128, n, vec, v[j]);
            }
        } else {
            // A block with a NaN or an infinity decodes to NaN as a whole
            // (scale NaN); one whose largest magnitude is below float32's
            // normal range, or zero, to zero.
            const float inf = __int_as_float(0x7f800000);
            float am = 0.0f, av = 0.0f;
            bool badm = false, badv = false;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    am = fmaxf(am, fabsf(m[j][i]));
                    av = fmaxf(av, fabsf(v[j][i]));
                    badm = badm || !(m[j][i] == m[j][i]);
                    badv = badv || !(v[j][i] == v[j][i]);
                }
            am = warp_max_nan(badm ? __int_as_float(0x7fc00000) : am);
            av = warp_max_nan(badv ? __int_as_float(0x7fc00000) : av);
            const bool finem = am < inf, finev = av < inf;
            const bool somem = finem && am >= 1.17549435e-38f, somev = finev && av >= 1.17549435e-38f;
            const float im = somem ? __fdiv_rn(1.0f, am) : 0.0f, iv = somev ? __fdiv_rn(1.0f, av) : 0.0f;
            const uint32_t key = pcg(c.k1 ^ (uint32_t)(tab.first + ti));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                int cm[4], cv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const unsigned long long e = (unsigned long long)(e0 + j * 128 + i);
                    const uint32_t r = pcg((uint32_t)e ^ key ^ (uint32_t)(e >> 32) * 0x9E3779B9u);
                    const float um = (float)(r & 0xffffu) * 1.52587890625e-05f;
                    const float uv = (float)(r >> 16) * 1.52587890625e-05f;
                    const float zm = somem ? fminf(__fmul_rn(fabsf(m[j][i]), im), 1.0f) : 0.0f;
                    const float zv = somev ? fminf(__fmul_rn(fabsf(v[j][i]), iv), 1.0f) : 0.0f;
                    const int k = encode_m(zm, um);
                    cm[i] = m[j][i] < 0.0f ? -k : k;
                    cv[i] = encode_v(zv, uv);
                }
                put_codes(static_cast<uint8_t*>(t.m), e0 + j * 128, n, vec, cm);
                put_codes(static_cast<uint8_t*>(t.v), e0 + j * 128, n, vec, cv);
            }
            if (lane == 0) {
                const long long blk = base / kAdamwBlock;
                t.ms[blk] = somem ? am : (finem ? 0.0f : __int_as_float(0x7fc00000));
                t.vs[blk] = somev ? av : (finev ? 0.0f : __int_as_float(0x7fc00000));
            }
        }
    }
}

__global__ void adamw_advance_kernel(long long* step) { *step += 1; }

struct ReadParams {
    Table tab;
    float* m_out[kAdamwTensors];
    float* v_out[kAdamwTensors];
};

// The 8-bit moments as float32 values.
__global__ void __launch_bounds__(kThreads) adamw_read_kernel(const __grid_constant__ ReadParams P) {
    const Table& tab = P.tab;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long tiles = tab.tile_end[tab.count - 1];
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int ti = find_tensor(tab, tile);
        const AdamwTensor& t = tab.t[ti];
        const bool vec = tab.vec[ti] != 0;
        const long long base = (tile - (ti ? tab.tile_end[ti - 1] : 0)) * kTile + warp * kAdamwBlock;
        if (base >= t.n) continue;
        const long long blk = base / kAdamwBlock;
        const float am = t.ms[blk], av = t.vs[blk];
        const long long e0 = base + lane * 4;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            int cm[4], cv[4];
            float m[4], v[4];
            get_codes(static_cast<const int8_t*>(t.m), e0 + j * 128, t.n, vec, cm);
            get_codes(static_cast<const uint8_t*>(t.v), e0 + j * 128, t.n, vec, cv);
#pragma unroll
            for (int i = 0; i < 4; ++i) { m[i] = decode_m(cm[i], am); v[i] = decode_v(cv[i], av); }
            put4(P.m_out[ti], e0 + j * 128, t.n, vec, m);
            put4(P.v_out[ti], e0 + j * 128, t.n, vec, v);
        }
    }
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Fills the table; returns the number of tiles.
long long fill(Table& tab, const AdamwTensor* t, int count, int first, int bits, size_t gsize) {
    tab.count = count;
    tab.first = first;
    long long tiles = 0;
    const size_t sa = bits == 32 ? 16 : 4;
    for (int i = 0; i < count; ++i) {
        tab.t[i] = t[i];
        tiles += (t[i].n + kTile - 1) / kTile;
        tab.tile_end[i] = tiles;
        tab.vec[i] = aligned(t[i].p, 16) && aligned(t[i].copy, 8) && aligned(t[i].g, 4 * gsize) &&
                     aligned(t[i].m, sa) && aligned(t[i].v, sa);
    }
    return tiles;
}

}  // namespace

cudaError_t launch_adamw(const void* args, cudaStream_t s, int* nlaunch) {
    const AdamwArgs& a = *static_cast<const AdamwArgs*>(args);
    *nlaunch = 0;
    Params P{};
    const long long tiles = fill(P.tab, a.t, a.count, a.first, a.bits, dtype_size(a.gdt));
    P.lr = a.lr; P.beta1 = a.beta1; P.beta2 = a.beta2; P.wd = a.weight_decay;
    P.b1 = (float)a.beta1; P.b2 = (float)a.beta2;
    P.c1 = (float)(1.0 - a.beta1); P.c2 = (float)(1.0 - a.beta2);
    P.eps = (float)a.eps;
    P.seed = a.seed; P.step = a.step; P.scalars = a.scalars;
    if (tiles > 0) {
        const int grid = (int)(tiles < (long long)a.num_sms * 4 ? tiles : (long long)a.num_sms * 4);
        const bool gf = a.gdt == DType::F32;
        if (a.bits == 32) {
            if (gf) adamw_kernel<float, 32><<<grid, kThreads, 0, s>>>(P);
            else adamw_kernel<bf16, 32><<<grid, kThreads, 0, s>>>(P);
        } else {
            if (gf) adamw_kernel<float, 8><<<grid, kThreads, 0, s>>>(P);
            else adamw_kernel<bf16, 8><<<grid, kThreads, 0, s>>>(P);
        }
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        ++*nlaunch;
    }
    if (a.advance) {
        adamw_advance_kernel<<<1, 1, 0, s>>>(a.step);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        ++*nlaunch;
    }
    return cudaSuccess;
}

cudaError_t launch_adamw_read(const void* args, cudaStream_t s, int* nlaunch) {
    const AdamwReadArgs& a = *static_cast<const AdamwReadArgs*>(args);
    *nlaunch = 0;
    ReadParams P{};
    const long long tiles = fill(P.tab, a.t, a.count, 0, 8, 4);
    if (tiles == 0) return cudaSuccess;
    for (int i = 0; i < a.count; ++i) {
        P.m_out[i] = a.m_out[i];
        P.v_out[i] = a.v_out[i];
        P.tab.vec[i] = aligned(a.t[i].m, 4) && aligned(a.t[i].v, 4) && aligned(a.m_out[i], 16) &&
                       aligned(a.v_out[i], 16);
    }
    const int grid = (int)(tiles < (long long)a.num_sms * 8 ? tiles : (long long)a.num_sms * 8);
    adamw_read_kernel<<<grid, kThreads, 0, s>>>(P);
    ++*nlaunch;
    return cudaGetLastError();
}

}  // namespace lstm
