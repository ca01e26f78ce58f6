// AdamW over every tensor of a model (Loshchilov and Hutter 2019, "Decoupled
// Weight Decay Regularization"), a launch for 64 tensors and one that moves the
// step counter, moments in float32 or in 8 bits.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v / (1 - b2^t)) + eps).
//
// The step moves 28 bytes per element with float32 moments and gradients, 18
// with 8-bit moments and a bf16 copy of p.  HBM bounds the first (3.7 M
// parameters: 15.6 to 16.6 us, the copy's rate), instruction issue the second (80 %
// active, some 100 instructions an element for decoding, update, hash and
// encoding; 37.8 M parameters: 157 us where the bytes take 104).  The tensors'
// table travels in the kernel's parameters, so a call needs no copy to the
// device and can be captured into a graph.
//
// The moments and their codes are rounded operation by operation (no
// contraction to FMA): the codes depend on the last bit of what is encoded,
// and with one order of roundings they are a function of the inputs that does
// not move with the compiler's choices.
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

// Byte k of w as a float32, by the exponent of 2^23: the conversion
// instructions run at an eighth of the rate of an addition.  `off` is what the
// byte is above the number it stands for.
__device__ __forceinline__ float byte_float(uint32_t w, int k, float off) {
    return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u + k)) - (8388608.0f + off);
}

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

__device__ __forceinline__ float sqrt_ftz(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Rounds up with the probability that keeps the mean of the value the code
// stands for: rounding to the nearest code would hold a second moment still
// for as long as a step changes it by less than half a code, which at
// b2 = 0.999 is nearly always.  z = |x| / a <= 1; u a random whole number below
// 2^16.  With X = z 127^2 and c the whole part of its root, up if
// u / 2^16 ((c + 1)^2 - c^2) < X - c^2.  The root may be off by its last bits:
// where that moves c by one, X lies within them of a code, and either start
// leads to that code (below it, the gap to it exceeds u / 2^16 times the gap;
// at it, nothing remains to round up).  So the largest code is not passed.  The
// code is the low byte of what is returned.
__device__ __forceinline__ uint32_t encode_m(float z, float u) {
    const float X = __fmul_rn(z, 16129.0f);
    const float f = __fadd_rd(sqrt_ftz(X), 8388608.0f);   // the whole part, in the low bits
    const float c = f - 8388608.0f;
    const float gap = fmaf(c, 0x1p-15f, 0x1p-16f);        // 2^-16 (2 c + 1), exact
    return __float_as_uint(f) + (__fmul_rn(u, gap) < __fsub_rn(X, __fmul_rn(c, c)) ? 1u : 0u);
}
// X = z 255^4 and the fourth powers.  A second moment that is not zero keeps a
// code of at least 1: a zero under the root would let the next step divide by
// eps alone.
__device__ __forceinline__ uint32_t encode_v(float z, float u) {
    const float X = __fmul_rn(z, 4228250625.0f);
    const float f = __fadd_rd(sqrt_ftz(sqrt_ftz(X)), 8388608.0f);
    const float c = f - 8388608.0f;
    const float lo2 = __fmul_rn(c, c), hi2 = __fadd_rn(lo2, fmaf(c, 2.0f, 1.0f));
    const float lo = __fmul_rn(lo2, lo2), gap = __fsub_rn(__fmul_rn(hi2, hi2), lo);
    const uint32_t k = __float_as_uint(f) + (__fmul_rn(u * 0x1p-16f, gap) < __fsub_rn(X, lo) ? 1u : 0u);
    return max(k, 0x4B000000u + min(__float_as_uint(X), 1u));   // (X is not negative)
}

__device__ __forceinline__ uint32_t low_bytes(const uint32_t (&k)[4]) {
    return __byte_perm(__byte_perm(k[0], k[1], 0x0040u), __byte_perm(k[2], k[3], 0x0040u), 0x5410u);
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

// The root and the quotient of the update are the approximate ones (2^-22 of
// it together, under float32's step of p itself for any update below p / 4);
// the moments are rounded operation by operation.
__device__ __forceinline__ void update(float& p, float g, float& m, float& v, const Params& P, const Coef& c) {
    g = __fmul_rn(g, c.gs);
    m = __fadd_rn(__fmul_rn(m, P.b1), __fmul_rn(g, P.c1));
    v = __fadd_rn(__fmul_rn(v, P.b2), __fmul_rn(__fmul_rn(g, g), P.c2));
    const float den = fmaf(sqrt_approx(v), c.root, P.eps);
    p = fmaf(p, c.keep, -c.size * __fdividef(m, den));
}

// Four elements from e as float, zeros past n.  FAST: all four exist and lie
// on a 16-byte (bf16: 8-byte, codes: 4-byte) boundary.
template <bool FAST, typename T>
__device__ __forceinline__ void get4(const T* x, long long e, long long n, float (&v)[4]) {
    if constexpr (FAST) {
        load4(x + e, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = e + i < n ? to_f(x[e + i]) : 0.0f;
    }
}
// Four codes as the bytes of a word.
template <bool FAST>
__device__ __forceinline__ uint32_t get_codes(const void* p, long long e, long long n) {
    const uint8_t* x = static_cast<const uint8_t*>(p);
    if constexpr (FAST) return *reinterpret_cast<const uint32_t*>(x + e);
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
        m[i] = decode_m(byte_float(cm, i, 128.0f), am);
        v[i] = decode_v(byte_float(cv, i, 0.0f), av);
    }
}
template <bool FAST>
__device__ __forceinline__ void put4(float* x, long long e, long long n, const float (&v)[4]) {
    if constexpr (FAST) {
        *reinterpret_cast<float4*>(x + e) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e + i < n) x[e + i] = v[i];
    }
}
// The copy is rounded to nearest even; p itself stays float32.
template <bool FAST>
__device__ __forceinline__ void put4(bf16* x, long long e, long long n, const float (&v)[4]) {
    if constexpr (FAST) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(x + e) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                      *reinterpret_cast<const uint32_t*>(&b));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e + i < n) x[e + i] = __float2bfloat16_rn(v[i]);
    }
}
template <bool FAST>
__device__ __forceinline__ void put_codes(void* p, long long e, long long n, uint32_t w) {
    uint8_t* x = static_cast<uint8_t*>(p);
    if constexpr (FAST) {
        *reinterpret_cast<uint32_t*>(x + e) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e + i < n) x[e + i] = (uint8_t)(w >> (8 * i));
    }
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
    bool fast;           // all 256 exist, on the boundaries of 4-element accesses
    long long base;      // its first element
    float p[2][4], g[2][4];
    float m[2][4], v[2][4];   // BITS 32
    uint32_t cm[2], cv[2];    // BITS 8
    float am, av;
};

// Finds the warp's block of tile `tile`; false when there is none.  *at: the
// tensor of an earlier tile (tiles come in rising order, so it only moves up).
__device__ __forceinline__ bool find_piece(const Table& tab, long long tile, int& at, int& ti, long long& base,
                                           bool& fast) {
    ti = -1;
    if (tile >= tab.tile_end[tab.count - 1]) return false;
    int i = at;
    while (tab.tile_end[i] <= tile) ++i;
    at = i;
    base = (tile - (i ? tab.tile_end[i - 1] : 0)) * kTile + (threadIdx.x >> 5) * kAdamwBlock;
    if (base >= tab.t[i].n) return false;   // (the whole warp)
    ti = i;
    fast = tab.vec[i] != 0 && base + kAdamwBlock <= tab.t[i].n;
    return true;
}

template <bool FAST, typename G, int BITS>
__device__ __forceinline__ void load_elements(const AdamwTensor& t, Piece<BITS>& x) {
    const long long e0 = x.base + (threadIdx.x & 31) * 4;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const long long e = e0 + j * 128;
        get4<FAST>(t.p, e, t.n, x.p[j]);
        get4<FAST>(static_cast<const G*>(t.g), e, t.n, x.g[j]);
        if constexpr (BITS == 8) {
            x.cm[j] = get_codes<FAST>(t.m, e, t.n);
            x.cv[j] = get_codes<FAST>(t.v, e, t.n);
        } else {
            get4<FAST>(static_cast<const float*>(t.m), e, t.n, x.m[j]);
            get4<FAST>(static_cast<const float*>(t.v), e, t.n, x.v[j]);
        }
    }
}

template <typename G, int BITS>
__device__ __forceinline__ void load_piece(const Table& tab, long long tile, int& at, Piece<BITS>& x) {
    if (!find_piece(tab, tile, at, x.ti, x.base, x.fast)) return;
    const AdamwTensor& t = tab.t[x.ti];
    if (x.fast) load_elements<true, G>(t, x);
    else load_elements<false, G>(t, x);
    if constexpr (BITS == 8) {
        x.am = t.ms[x.base / kAdamwBlock];
        x.av = t.vs[x.base / kAdamwBlock];
    }
}

template <bool FAST, int BITS>
__device__ __forceinline__ void step_piece(const Params& P, const Coef& c, const Piece<BITS>& w) {
    const AdamwTensor& t = P.tab.t[w.ti];
    const int lane = threadIdx.x & 31;
    const long long n = t.n, e0 = w.base + lane * 4;
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
        put4<FAST>(t.p, e0 + j * 128, n, p[j]);
        if (t.copy) put4<FAST>(static_cast<bf16*>(t.copy), e0 + j * 128, n, p[j]);
        if constexpr (BITS == 32) {
            put4<FAST>(static_cast<float*>(t.m), e0 + j * 128, n, m[j]);
            put4<FAST>(static_cast<float*>(t.v), e0 + j * 128, n, v[j]);
        }
    }
    if constexpr (BITS == 8) {
        // A block with a NaN or an infinity decodes to NaN as a whole (scale
        // NaN, whatever the codes); one whose largest magnitude is below
        // float32's normal range, or zero, to zero.
        const float inf = __int_as_float(0x7f800000), nan = __int_as_float(0x7fc00000);
        float am = 0.0f, av = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // past the end nothing counts towards the block's scale
                if (!FAST && e0 + j * 128 + i >= n) m[j][i] = v[j][i] = 0.0f;
                am = max_nan(am, m[j][i]);
                av = max_nan(av, v[j][i]);
            }
        am = warp_max_nan(am);
        av = warp_max_nan(av);
        const bool finem = am < inf, finev = av < inf;
        const bool somem = finem && am >= 1.17549435e-38f, somev = finev && av >= 1.17549435e-38f;
        const float im = somem ? __frcp_rn(am) : 0.0f, iv = somev ? __frcp_rn(av) : 0.0f;
        const uint32_t key = pcg(c.k1 ^ (uint32_t)(P.tab.first + w.ti)) ^
                             (uint32_t)((unsigned long long)w.base >> 32) * 0x9E3779B9u;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t cm[4], cv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t r = pcg((uint32_t)(e0 + j * 128 + i) ^ key);
                const float um = __uint_as_float((r & 0xffffu) | 0x4B000000u) - 8388608.0f;
                const float uv = __uint_as_float(__byte_perm(r, 0x4B000000u, 0x7432u)) - 8388608.0f;
                const uint32_t k = encode_m(fminf(__fmul_rn(fabsf(m[j][i]), im), 1.0f), um);
                const uint32_t sign = (uint32_t)(__float_as_int(m[j][i]) >> 31);   // all ones below zero
                cm[i] = (k ^ sign) - sign;
                cv[i] = encode_v(fminf(__fmul_rn(v[j][i], iv), 1.0f), uv);
            }
            put_codes<FAST>(t.m, e0 + j * 128, n, low_bytes(cm));
            put_codes<FAST>(t.v, e0 + j * 128, n, low_bytes(cv));
        }
        if (lane == 0) {
            const long long blk = w.base / kAdamwBlock;
            t.ms[blk] = somem ? am : (finem ? 0.0f : nan);
            t.vs[blk] = somev ? av : (finev ? 0.0f : nan);
        }
    }
}

// A warp per block of 256 elements, the next block's loads issued before the
// current one is computed (the first one's before the coefficients).
template <typename G, int BITS>
__global__ void __launch_bounds__(kThreads, BITS == 8 ? 3 : 2) adamw_kernel(const __grid_constant__ Params P) {
    __shared__ Coef coef;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Piece<BITS> x;
    int at = 0;
    load_piece<G, BITS>(P.tab, blockIdx.x, at, x);
    make_coef(P, coef);
    __syncthreads();
    const Coef c = coef;
    const long long tiles = P.tab.tile_end[P.tab.count - 1];
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const Piece<BITS> w = x;
        load_piece<G, BITS>(P.tab, tile + gridDim.x, at, x);
        if (w.ti < 0) continue;
        if (w.fast) step_piece<true>(P, c, w);
        else step_piece<false>(P, c, w);
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

// The 8-bit moments as float32 values; two blocks of 256 a warp at a time.
__global__ void __launch_bounds__(kThreads, 6) adamw_read_kernel(const __grid_constant__ ReadParams P) {
    const Table& tab = P.tab;
    const int lane = threadIdx.x & 31;
    const long long tiles = tab.tile_end[tab.count - 1];
    int at = 0;
    for (long long tile = blockIdx.x; tile < tiles; tile += 2ll * gridDim.x) {
        int ti[2];
        long long base[2];
        bool fast[2];
        uint32_t cm[2][2], cv[2][2];
        float am[2], av[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!find_piece(tab, tile + k * (long long)gridDim.x, at, ti[k], base[k], fast[k])) continue;
            const AdamwTensor& t = tab.t[ti[k]];
            am[k] = t.ms[base[k] / kAdamwBlock];
            av[k] = t.vs[base[k] / kAdamwBlock];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const long long e = base[k] + lane * 4 + j * 128;
                cm[k][j] = fast[k] ? get_codes<true>(t.m, e, t.n) : get_codes<false>(t.m, e, t.n);
                cv[k][j] = fast[k] ? get_codes<true>(t.v, e, t.n) : get_codes<false>(t.v, e, t.n);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (ti[k] < 0) continue;
            const long long n = tab.t[ti[k]].n;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const long long e = base[k] + lane * 4 + j * 128;
                float m[4], v[4];
                decode4(cm[k][j], cv[k][j], am[k], av[k], m, v);
                if (fast[k]) {
                    put4<true>(P.m_out[ti[k]], e, n, m);
                    put4<true>(P.v_out[ti[k]], e, n, v);
                } else {
                    put4<false>(P.m_out[ti[k]], e, n, m);
                    put4<false>(P.v_out[ti[k]], e, n, v);
                }
            }
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
    const int grid = (int)(tiles < (long long)a.num_sms * 6 ? tiles : (long long)a.num_sms * 6);
    adamw_read_kernel<<<grid, kThreads, 0, s>>>(P);
    ++*nlaunch;
    return cudaGetLastError();
}

}  // namespace lstm
