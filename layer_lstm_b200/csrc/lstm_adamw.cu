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

// Small whole numbers to float32 and back by the exponent of 2^23 (the
// conversion instructions run at an eighth of the rate of an addition, and
// eight of them per element would take as long as the rest).
__device__ __forceinline__ float small_float(uint32_t n) { return __uint_as_float(0x4B000000u | n) - 8388608.0f; }
__device__ __forceinline__ uint32_t small_bits(float x) { return __float_as_uint(x + 8388608.0f); }   // low bytes: x

// Code c of a first moment stands for sign (c / 127)^2 a, of a second for
// (c / 255)^4 a, with a the largest magnitude of the element's block of 256.
// The codes are dense where the values are small next to the block's largest:
// the smallest nonzero first moment is 6e-5 a, second moment 2e-10 a.
__device__ __forceinline__ float decode_m(float c, float a) {
    const float q = __fmul_rn(c, 1.0f / 127.0f);
    return __fmul_rn(__fmul_rn(fabsf(q), q), a);
}
__device__ __forceinline__ float decode_v(float c, float a) {
    const float q = __fmul_rn(c, 1.0f / 255.0f);
    const float q2 = __fmul_rn(q, q);
    return __fmul_rn(__fmul_rn(q2, q2), a);
}

__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Rounds up with the probability that keeps the mean of the value the code
// stands for: rounding to the nearest code would hold a second moment still
// for as long as a step changes it by less than half a code, which at
// b2 = 0.999 is nearly always.  z = |x| / a; u random in [0, 1).  The root may
// be off by its last bits: where that moves floor() by one, x lies within them
// of a code, and either start leads to that code (below it, the gap to it
// exceeds u times the gap; at it, nothing remains to round up).
__device__ __forceinline__ float encode_m(float z, float u) {
    const float X = __fmul_rn(z, 16129.0f);
    float c = floorf(sqrt_approx(X));
    const float lo = __fmul_rn(c, c), c1 = __fadd_rn(c, 1.0f), hi = __fmul_rn(c1, c1);
    if (__fmul_rn(u, __fsub_rn(hi, lo)) < __fsub_rn(X, lo)) c = c1;
    return fminf(c, 127.0f);
}
// A second moment that is not zero keeps a code of at least 1: a zero under
// the root would let the next step divide by eps alone.
__device__ __forceinline__ float encode_v(float z, float u) {
    const float X = __fmul_rn(z, 4228250625.0f);
    float c = floorf(sqrt_approx(sqrt_approx(X)));
    const float c1 = __fadd_rn(c, 1.0f);
    const float lo2 = __fmul_rn(c, c), hi2 = __fmul_rn(c1, c1);
    const float lo = __fmul_rn(lo2, lo2), hi = __fmul_rn(hi2, hi2);
    if (__fmul_rn(u, __fsub_rn(hi, lo)) < __fsub_rn(X, lo)) c = c1;
    if (X > 0.0f) c = fmaxf(c, 1.0f);
    return fminf(c, 255.0f);
}

struct Coef {
    float size, root, keep, gs;   // lr / (1 - b1^t), 1 / sqrt(1 - b2^t), 1 - lr wd, gradient factor
    uint32_t k1;                  // random key of (seed, step)
};

// Warp 0 and warp 1 each take a power in float64 (a microsecond).
__device__ __forceinline__ void make_coef(const Params& P, Coef& c) {
    if ((threadIdx.x & 31) != 0 || threadIdx.x >= 64) return;
    const long long t = *P.step + 1;
    if (threadIdx.x == 0) {
        double lr = P.lr;
        float gs = 1.0f;
        if (P.scalars) {
            lr *= (double)P.scalars[0];
            gs = P.scalars[1];
        }
        c.size = (float)(lr / (1.0 - pow(P.beta1, (double)t)));
        c.keep = (float)(1.0 - lr * P.wd);
        c.gs = gs;
    } else {
        c.root = (float)(1.0 / sqrt(1.0 - pow(P.beta2, (double)t)));
        c.k1 = pcg((uint32_t)t ^ pcg((uint32_t)P.seed ^ pcg((uint32_t)(P.seed >> 32))));
    }
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
// Four codes as the bytes of a word.
__device__ __forceinline__ uint32_t get_codes(const void* p, long long e, long long n, bool vec) {
    const uint8_t* x = static_cast<const uint8_t*>(p);
    if (vec && e + 4 <= n) return *reinterpret_cast<const uint32_t*>(x + e);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= e + i < n ? (uint32_t)x[e + i] << (8 * i) : 0u;
    return w;
}
// Values of four first-moment codes (signed bytes) and second-moment codes.
__device__ __forceinline__ void decode4(uint32_t cm, uint32_t cv, float am, float av, float (&m)[4], float (&v)[4]) {
    cm ^= 0x80808080u;   // signed byte + 128
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = decode_m(small_float((cm >> (8 * i)) & 255u) - 128.0f, am);
        v[i] = decode_v(small_float((cv >> (8 * i)) & 255u), av);
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
__device__ __forceinline__ void put_codes(void* p, long long e, long long n, bool vec, uint32_t w) {
    uint8_t* x = static_cast<uint8_t*>(p);
    if (vec && e + 4 <= n) {
        *reinterpret_cast<uint32_t*>(x + e) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e + i < n) x[e + i] = (uint8_t)(w >> (8 * i));
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

// Largest magnitude; NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}
__device__ __forceinline__ float warp_max_nan(float a) {
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(a));
    return r;
}

// What a warp holds of one block of 256 elements: 2 x 4 of each lane.
template <int BITS>
struct Piece {
    int ti;              // tensor; -1: none
    long long base;      // its first element
    float p[2][4], g[2][4];
    float m[2][4], v[2][4];   // BITS 32
    uint32_t cm[2], cv[2];    // BITS 8
    float am, av;
};

template <typename G, int BITS>
__device__ __forceinline__ void load_piece(const Table& tab, long long tile, Piece<BITS>& x) {
    x.ti = -1;
    if (tile >= tab.tile_end[tab.count - 1]) return;
    const int ti = find_tensor(tab, tile);
    const AdamwTensor& t = tab.t[ti];
    const bool vec = tab.vec[ti] != 0;
    const long long n = t.n;
    x.base = (tile - (ti ? tab.tile_end[ti - 1] : 0)) * kTile + (threadIdx.x >> 5) * kAdamwBlock;
    if (x.base >= n) return;   // (the whole warp)
    x.ti = ti;
    const long long e0 = x.base + (threadIdx.x & 31) * 4;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const long long e = e0 + j * 128;
        get4(t.p, e, n, vec, x.p[j]);
        get4(static_cast<const G*>(t.g), e, n, vec, x.g[j]);
        if constexpr (BITS == 8) {
            x.cm[j] = get_codes(t.m, e, n, vec);
            x.cv[j] = get_codes(t.v, e, n, vec);
        } else {
            get4(static_cast<const float*>(t.m), e, n, vec, x.m[j]);
            get4(static_cast<const float*>(t.v), e, n, vec, x.v[j]);
        }
    }
    if constexpr (BITS == 8) {
        x.am = t.ms[x.base / kAdamwBlock];
        x.av = t.vs[x.base / kAdamwBlock];
    }
}

// A warp per block of 256 elements, the next block's loads issued before the
// current one is computed (the first one's before the coefficients).
template <typename G, int BITS>
__global__ void __launch_bounds__(kThreads, BITS == 8 ? 3 : 2) adamw_kernel(const __grid_constant__ Params P) {
    __shared__ Coef coef;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Table& tab = P.tab;
    Piece<BITS> x;
    load_piece<G, BITS>(tab, blockIdx.x, x);
    make_coef(P, coef);
    __syncthreads();
    const Coef c = coef;
    const int lane = threadIdx.x & 31;
    const long long tiles = tab.tile_end[tab.count - 1];
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const Piece<BITS> w = x;
        load_piece<G, BITS>(tab, tile + gridDim.x, x);
        if (w.ti < 0) continue;
        const AdamwTensor& t = tab.t[w.ti];
        const bool vec = tab.vec[w.ti] != 0;
        const long long n = t.n, e0 = w.base + lane * 4;
        const bool whole = w.base + kAdamwBlock <= n;
        float p[2][4], m[2][4], v[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if constexpr (BITS == 8) decode4(w.cm[j], w.cv[j], w.am, w.av, m[j], v[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[j][i] = w.p[j][i];
                if constexpr (BITS == 32) { m[j][i] = w.m[j][i]; v[j][i] = w.v[j][i]; }
                update(p[j][i], w.g[j][i], m[j][i], v[j][i], P, c);
            }
            put4(t.p, e0 + j * 128, n, vec, p[j]);
            if (t.copy) put4(static_cast<bf16*>(t.copy), e0 + j * 128, n, vec, p[j]);
            if constexpr (BITS == 32) {
                put4(static_cast<float*>(t.m), e0 + j * 128, n, vec, m[j]);
                put4(static_cast<float*>(t.v), e0 + j * 128, n, vec, v[j]);
            }
        }
        if constexpr (BITS == 8) {
            // A block with a NaN or an infinity decodes to NaN as a whole
            // (scale NaN); one whose largest magnitude is below float32's
            // normal range, or zero, to zero.
            const float inf = __int_as_float(0x7f800000), nan = __int_as_float(0x7fc00000);
            float am = 0.0f, av = 0.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // past the end nothing counts towards the block's scale
                    if (!whole && e0 + j * 128 + i >= n) m[j][i] = v[j][i] = 0.0f;
                    am = max_nan(am, m[j][i]);
                    av = max_nan(av, v[j][i]);
                }
            am = warp_max_nan(am);
            av = warp_max_nan(av);
            const bool finem = am < inf, finev = av < inf;
            const bool somem = finem && am >= 1.17549435e-38f, somev = finev && av >= 1.17549435e-38f;
            const float im = somem ? __frcp_rn(am) : 0.0f, iv = somev ? __frcp_rn(av) : 0.0f;
            const uint32_t key = pcg(c.k1 ^ (uint32_t)(tab.first + w.ti)) ^ (uint32_t)((unsigned long long)w.base >> 32) * 0x9E3779B9u;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t cm = 0, cv = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t r = pcg((uint32_t)(e0 + j * 128 + i) ^ key);
                    const float um = small_float(r & 0xffffu) * 1.52587890625e-05f;
                    const float uv = small_float(r >> 16) * 1.52587890625e-05f;
                    // where the block has no scale the products are 0 or NaN, and 0 is stored
                    const float zm = somem ? fminf(__fmul_rn(fabsf(m[j][i]), im), 1.0f) : 0.0f;
                    const float zv = somev ? fminf(__fmul_rn(fabsf(v[j][i]), iv), 1.0f) : 0.0f;
                    const float k = encode_m(zm, um);
                    // two's complement of a negative code by its bits around 2^23
                    cm |= (small_bits(m[j][i] < 0.0f ? 256.0f - k : k) & 255u) << (8 * i);
                    cv |= (small_bits(encode_v(zv, uv)) & 255u) << (8 * i);
                }
                put_codes(t.m, e0 + j * 128, n, vec, cm);
                put_codes(t.v, e0 + j * 128, n, vec, cv);
            }
            if (lane == 0) {
                const long long blk = w.base / kAdamwBlock;
                t.ms[blk] = somem ? am : (finem ? 0.0f : nan);
                t.vs[blk] = somev ? av : (finev ? 0.0f : nan);
            }
        }
    }
}

// Runs behind the last launch of a step, as its programmatic dependent.
__global__ void adamw_advance_kernel(long long* step) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    *step += 1;
}

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
            float m[4], v[4];
            decode4(get_codes(t.m, e0 + j * 128, t.n, vec), get_codes(t.v, e0 + j * 128, t.n, vec), am, av, m, v);
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
        const int per_sm = a.bits == 8 ? 3 : 2;   // blocks an SM, as the launch bounds say
        const int grid = (int)(tiles < (long long)a.num_sms * per_sm ? tiles : (long long)a.num_sms * per_sm);
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
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(1);
        cfg.blockDim = dim3(1);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, adamw_advance_kernel, a.step);
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
