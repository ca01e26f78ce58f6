// Linear attention with a decay for each head: the products of lstm_ops.h's
// LinJob on the CUDA cores, in float32, for every size, type and alignment,
// and the single-token step.
//
// A sequence is taken in chunks of 64 steps.  Inside a chunk the recurrence is
// a causal score matrix, P_ij = g^(i-j) a_i . b_j; across chunks it is the
// state X, which the chunk's outputs read once and its b^T c updates once:
//   out_i = P c + g^(i+e) a_i X,   X <- g^m X + sum_j g^(m-e-j) b_j^T c_j.
// One block owns a (batch row, head) and walks its chunks with X in shared
// memory, so X never leaves the SM.  Where rows and heads are too few to fill
// the device the time axis is cut into segments: the segments' own states
// first (from zero), one pass that carries the state over the segments, then
// every segment at once from its true initial state.
#include <algorithm>

#include "lstm_device.cuh"
#include "lstm_linatt.cuh"
#include "lstm_ops.h"

namespace lstm {
namespace {

constexpr int C = kLinChunk;
constexpr int kThreads = 256;

template <int D>
constexpr size_t smem_floats() {
    // a (the scores over it), b, c, X, powers
    return (size_t)C * (D + 4 > C + 4 ? D + 4 : C + 4) + (size_t)2 * C * (D + 4) + (size_t)D * (D + 4) + C + 1;
}

// N consecutive floats of shared memory (N = 2 or a multiple of 4).
template <int N>
__device__ __forceinline__ void lds(const float* p, float (&v)[N]) {
    if constexpr (N == 2) {
        const float2 q = *reinterpret_cast<const float2*>(p);
        v[0] = q.x; v[1] = q.y;
    } else {
        static_assert(N == 4, "2 or 4");
        const float4 q = *reinterpret_cast<const float4*>(p);
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    }
}

// Rows [0, m) of a chunk (d of D columns) into shared memory, zeros elsewhere.
template <typename T, int D>
__device__ __forceinline__ void load_chunk(float* dst, const T* src, const LinRow& row, int tau0, int m, long long ld,
                                           int d, bool vec) {
    constexpr int P = D + 4;
    if (vec) {
        // all of a thread's loads in flight at once (float32: straight to
        // shared memory, awaited by chunk_landed)
        constexpr int NL = C * (D / 4) / kThreads;
        float v[NL][4];
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int i = threadIdx.x + j * kThreads, r = i / (D / 4), c = (i % (D / 4)) * 4;
            const bool in = r < m && c < d;
            if constexpr (sizeof(T) == 4) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 (uint32_t)__cvta_generic_to_shared(dst + r * P + c)),
                             "l"(in ? src + row.at(tau0 + r) * ld + c : src), "r"(in ? 16 : 0)
                             : "memory");
            } else {
                v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0.0f;
                if (in) load4(src + row.at(tau0 + r) * ld + c, v[j]);
            }
        }
        if constexpr (sizeof(T) != 4) {
#pragma unroll
            for (int j = 0; j < NL; ++j) {
                const int i = threadIdx.x + j * kThreads, r = i / (D / 4), c = (i % (D / 4)) * 4;
                *reinterpret_cast<float4*>(dst + r * P + c) = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
            }
        }
    } else {
        for (int i = threadIdx.x; i < C * D; i += kThreads) {
            const int r = i / D, c = i % D;
            dst[r * P + c] = r < m && c < d ? to_f(src[row.at(tau0 + r) * ld + c]) : 0.0f;
        }
    }
}

__device__ __forceinline__ void chunk_landed() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <typename T>
__device__ __forceinline__ bool can_vec(const void* p, long long ld, int d) {
    return d % 4 == 0 && ld % 4 == 0 && ((uintptr_t)p & (4 * sizeof(T) - 1)) == 0;
}

// MODE: see LinMode.
template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kThreads, D == 128 ? 1 : 3) lin_kernel(const __grid_constant__ LinArgs g) {
    constexpr int P = D + 4, PC = C + 4;
    constexpr int W = D / 16 < 4 ? D / 16 : 4;   // consecutive columns of a thread's tile
    constexpr int NW = D / 16 / W;               // tiles of W columns, 16 W apart
    extern __shared__ float sm[];
    float* sa = sm;
    float* sp = sm;            // the scores, once a has been read: three blocks of D = 64 share an SM
    float* sb = sa + C * (P > PC ? P : PC);
    float* sc = sb + C * P;
    float* sx = sc + C * P;
    float* gp = sx + D * P;    // g^0 .. g^C

    if (MODE != kLinSegments && blockIdx.x == 0 && threadIdx.x == 0) *g.status = kStatusOk;
    LinItem it;
    lin_item(g, MODE, blockIdx.x, it);
    const LinJob& J = g.job[it.job];
    const LinRow& row = it.row;
    const T* a = static_cast<const T*>(J.a) + it.h * J.da;
    const T* b = static_cast<const T*>(J.b) + it.h * J.da;
    const T* c = static_cast<const T*>(J.c) + it.h * J.dc;
    T* o = static_cast<T*>(J.o) + it.h * J.dc;
    const bool va = can_vec<T>(a, J.lda, J.da), vb = can_vec<T>(b, J.ldb, J.da), vc = can_vec<T>(c, J.ldc, J.dc);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int da4 = (J.da + 3) & ~3;
    // of sizes 65 to 128 only the larger may fill the second half of a tile
    const bool a2 = NW > 1 && J.da > 16 * W, c2 = NW > 1 && J.dc > 16 * W;

    if (threadIdx.x <= C) gp[threadIdx.x] = expf(it.ld * (float)threadIdx.x);
    for (int i = threadIdx.x; i < D * D; i += kThreads) {
        const int r = i / D, q = i % D;
        sx[r * P + q] = it.init && r < J.da && q < J.dc
                            ? (it.init_t ? it.init[(size_t)q * J.da + r] : it.init[(size_t)r * J.dc + q])
                            : 0.0f;
    }
    for (int tau = it.tau0; tau < it.tau1; tau += C) {
        const int m = min(C, it.tau1 - tau);
        __syncthreads();
        if (MODE != kLinStates) load_chunk<T, D>(sa, a, row, tau, m, J.lda, J.da, va);
        load_chunk<T, D>(sb, b, row, tau, m, J.ldb, J.da, vb);
        load_chunk<T, D>(sc, c, row, tau, m, J.ldc, J.dc, vc);
        chunk_landed();
        __syncthreads();
        if (MODE != kLinStates) {
            // scores of rows ty*4 + i, columns tx + 16 j, and a X
            float p[4][4] = {};
            float acc[4][NW][W] = {};
            if (ty * 4 < m) {
#pragma unroll 2
                for (int k = 0; k < da4; k += 4) {
                    float x[4][4], y[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        lds<4>(sa + (ty * 4 + i) * P + k, x[i]);
                        lds<4>(sb + (tx + 16 * i) * P + k, y[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int q = 0; q < 4; ++q) p[i][j] = fmaf(x[i][q], y[j][q], p[i][j]);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int u = 0; u < NW; ++u) {
                            if (u && !c2) continue;
                            float z[W];
                            lds<W>(sx + (k + q) * P + u * 16 * W + tx * W, z);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int j = 0; j < W; ++j) acc[i][u][j] = fmaf(x[i][q], z[j], acc[i][u][j]);
                        }
                }
            }
            __syncthreads();   // a has been read
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = ty * 4 + i, q = tx + 16 * j;
                    sp[r * PC + q] = q <= r ? p[i][j] * (gp[r - q] * J.bscale) : 0.0f;
                }
            __syncthreads();
            if (ty * 4 < m) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = gp[ty * 4 + i + it.e];
#pragma unroll
                    for (int u = 0; u < NW; ++u)
#pragma unroll
                        for (int j = 0; j < W; ++j) acc[i][u][j] *= f;
                }
                for (int k = 0; k <= ty * 4; k += 4) {
                    float x[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) lds<4>(sp + (ty * 4 + i) * PC + k, x[i]);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int u = 0; u < NW; ++u) {
                            if (u && !c2) continue;
                            float y[W];
                            lds<W>(sc + (k + q) * P + u * 16 * W + tx * W, y);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int j = 0; j < W; ++j) acc[i][u][j] = fmaf(x[i][q], y[j], acc[i][u][j]);
                        }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (ty * 4 + i >= m) continue;
                    T* dst = o + row.at(tau + ty * 4 + i) * J.ldo;
#pragma unroll
                    for (int u = 0; u < NW; ++u)
#pragma unroll
                        for (int j = 0; j < W; ++j) {
                            const int q = u * 16 * W + tx * W + j;
                            if (q < J.dc) dst[q] = from_f<T>(acc[i][u][j] * J.oscale);
                        }
                }
            }
        }
        if (!it.fin && tau + C >= it.tau1) break;   // nothing reads the last X
        // X <- g^m X + sum_j bscale g^(m-e-j) b_j^T c_j; rows like the columns
        float acc[NW][W][NW][W];
        const float gm = gp[m];
#pragma unroll
        for (int t = 0; t < NW; ++t)
#pragma unroll
            for (int i = 0; i < W; ++i)
#pragma unroll
                for (int u = 0; u < NW; ++u) {
                    lds<W>(sx + (t * 16 * W + ty * W + i) * P + u * 16 * W + tx * W, acc[t][i][u]);
#pragma unroll
                    for (int j = 0; j < W; ++j) acc[t][i][u][j] *= gm;
                }
        for (int k = 0; k < m; ++k) {
            const float f = gp[m - it.e - k] * J.bscale;
            float x[NW][W], y[NW][W];
#pragma unroll
            for (int t = 0; t < NW; ++t) {
                lds<W>(sb + k * P + t * 16 * W + ty * W, x[t]);
                lds<W>(sc + k * P + t * 16 * W + tx * W, y[t]);
#pragma unroll
                for (int i = 0; i < W; ++i) x[t][i] *= f;
            }
#pragma unroll
            for (int t = 0; t < NW; ++t) {
                if (t && !a2) continue;
#pragma unroll
                for (int u = 0; u < NW; ++u) {
                    if (u && !c2) continue;
#pragma unroll
                    for (int i = 0; i < W; ++i)
#pragma unroll
                        for (int j = 0; j < W; ++j) acc[t][i][u][j] = fmaf(x[t][i], y[u][j], acc[t][i][u][j]);
                }
            }
        }
        __syncthreads();   // every thread has read the old X
#pragma unroll
        for (int t = 0; t < NW; ++t)
#pragma unroll
            for (int i = 0; i < W; ++i)
#pragma unroll
                for (int u = 0; u < NW; ++u)
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        sx[(t * 16 * W + ty * W + i) * P + u * 16 * W + tx * W + j] = acc[t][i][u][j];
    }
    __syncthreads();
    if (it.fin) {
        for (int i = threadIdx.x; i < J.da * J.dc; i += kThreads) it.fin[i] = sx[(i / J.dc) * P + i % J.dc];
    }
    if (MODE != kLinStates) {
        // padded steps of this segment
        for (int i = threadIdx.x; i < (it.pad1 - it.pad0) * J.dc; i += kThreads)
            o[row.padded(it.pad0 + i / J.dc) * J.ldo + i % J.dc] = from_f<T>(0.0f);
    }
}

// Carries the state over the segments of a (row, head): buf[seg] turns from
// the segment's own state into the state it starts from.
__global__ void __launch_bounds__(kThreads) lin_carry_kernel(const __grid_constant__ LinArgs g) {
    const LinJob& J = g.job[blockIdx.z];
    const int bh = blockIdx.x, n = J.da * J.dc;
    const int b = bh / g.H, h = bh % g.H;
    const int len = lin_length(g, b);
    const float ld = lin_log_decay(g.log_decay[h]);
    float* buf = g.buf + lin_buf_offset(g, blockIdx.z) + (size_t)bh * g.nseg * n;
    for (int i = blockIdx.y * kThreads + threadIdx.x; i < n; i += gridDim.y * kThreads) {
        float x = 0.0f;
        if (J.init) x = J.init[(size_t)bh * n + (J.init_t ? (i % J.dc) * J.da + i / J.dc : i)];
        // eight segments' states at a time: a load behind each store would
        // cost its latency for every segment
        constexpr int AT = 8;
        for (int s0 = 0; s0 < g.nseg; s0 += AT) {
            float own[AT];
#pragma unroll
            for (int k = 0; k < AT; ++k) own[k] = s0 + k < g.nseg ? buf[(size_t)(s0 + k) * n + i] : 0.0f;
#pragma unroll
            for (int k = 0; k < AT; ++k) {
                if (s0 + k >= g.nseg) break;
                buf[(size_t)(s0 + k) * n + i] = x;
                x = fmaf(expf(ld * (float)lin_steps(g, len, s0 + k, J.reverse)), x, own[k]);
            }
        }
        if (J.fin) J.fin[(size_t)bh * n + i] = x;
    }
}

template <typename T, int D, int MODE>
cudaError_t run(const LinArgs& a, cudaStream_t s, int* n) {
    constexpr size_t bytes = smem_floats<D>() * 4;
    // set on every call: it is a property of the current device's function
    cudaError_t e = cudaFuncSetAttribute(lin_kernel<T, D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((long long)a.B * a.H * a.njobs * a.nseg);
    lin_kernel<T, D, MODE><<<grid, kThreads, bytes, s>>>(a);
    ++*n;
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t run_dim(const LinArgs& a, cudaStream_t s, int* n) {
    if (a.nseg <= 1) return run<T, D, kLinWhole>(a, s, n);
    cudaError_t e = run<T, D, kLinStates>(a, s, n);
    if (e != cudaSuccess) return e;
    if ((e = launch_lin_carry(a, s, n)) != cudaSuccess) return e;
    return run<T, D, kLinSegments>(a, s, n);
}

template <typename T>
cudaError_t run_type(const LinArgs& a, cudaStream_t s, int* n) {
    const int d = std::max(a.job[0].da, a.job[0].dc);
    if (d <= 32) return run_dim<T, 32>(a, s, n);
    if (d <= 64) return run_dim<T, 64>(a, s, n);
    return run_dim<T, 128>(a, s, n);
}

// ------------------------------------------------------------- single token
// A block per (batch row, head): the state is read and written once, VEC
// columns a thread, as many rows at a time as the block's threads cover.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) lin_step_kernel(const LinStepArgs g) {
    __shared__ float sq[kLinMaxDim], sk[kLinMaxDim], red[kThreads * VEC];
    const int bh = blockIdx.x, b = bh / g.H, h = bh % g.H;
    const int tpr = (g.dv + VEC - 1) / VEC;        // threads per state row
    const int rows = kThreads / tpr;               // state rows at a time
    const int r0 = threadIdx.x / tpr, c0 = (threadIdx.x % tpr) * VEC;
    T* out = static_cast<T*>(g.out) + (size_t)bh * g.dv;
    if (g.lengths && g.lengths[b] < 1) {
        for (int i = threadIdx.x; i < g.dv; i += kThreads) out[i] = from_f<T>(0.0f);
        return;
    }
    const T* q = static_cast<const T*>(g.q) + b * g.ldq + (size_t)h * g.dk;
    const T* k = static_cast<const T*>(g.k) + b * g.ldk + (size_t)h * g.dk;
    const T* v = static_cast<const T*>(g.v) + b * g.ldv + (size_t)h * g.dv;
    const float decay = expf(lin_log_decay(g.log_decay[h]));
    if (threadIdx.x < g.dk) {
        sq[threadIdx.x] = to_f(q[threadIdx.x]);
        sk[threadIdx.x] = to_f(k[threadIdx.x]);
    }
    __syncthreads();
    float acc[VEC] = {};
    if (r0 < rows) {
        float vv[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) vv[j] = to_f(v[c0 + j]);
        float* S = g.state + (size_t)bh * g.dk * g.dv + c0;
        constexpr int AT = 8;   // rows in flight: row by row the 268 MB of 512 rows took 105 us, now 83
        for (int rb = r0; rb < g.dk; rb += AT * rows) {
            float s[AT][VEC];
#pragma unroll
            for (int k = 0; k < AT; ++k) {
                const int r = rb + k * rows;
                if (r >= g.dk) break;
                if constexpr (VEC == 4) load4(S + (size_t)r * g.dv, s[k]);
                else s[k][0] = S[(size_t)r * g.dv];
            }
#pragma unroll
            for (int k = 0; k < AT; ++k) {
                const int r = rb + k * rows;
                if (r >= g.dk) break;
                const float kk = sk[r], qq = sq[r];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    s[k][j] = fmaf(decay, s[k][j], kk * vv[j]);
                    acc[j] = fmaf(qq, s[k][j], acc[j]);
                }
                if constexpr (VEC == 4)
                    *reinterpret_cast<float4*>(S + (size_t)r * g.dv) = make_float4(s[k][0], s[k][1], s[k][2], s[k][3]);
                else S[(size_t)r * g.dv] = s[k][0];
            }
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) red[(r0 * tpr) * VEC + c0 + j] = acc[j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < g.dv; i += kThreads) {
        float s = 0.0f;
        for (int r = 0; r < rows; ++r) s += red[r * tpr * VEC + i];
        out[i] = from_f<T>(s * g.scale);
    }
}

template <typename T>
cudaError_t step_type(const LinStepArgs& a, cudaStream_t s) {
    const unsigned grid = (unsigned)((long long)a.B * a.H);
    if (a.dv % 4 == 0 && ((uintptr_t)a.state & 15) == 0) lin_step_kernel<T, 4><<<grid, kThreads, 0, s>>>(a);
    else lin_step_kernel<T, 1><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

int lin_segments(int B, int T, int H, int njobs, int num_sms, bool tc, int* seg_len) {
    // Where rows, heads and products leave SMs idle, the time axis is shared
    // out: up to two blocks for every SM (one of the tensor-core kernel's), a
    // chunk each at least.  A segment's own state costs some 0.6 of its
    // outputs' time, and the two launches more 6 us; a chunk takes 2 us on the
    // tensor cores, 6 to 16 on the CUDA cores, so it pays from 6 and 3 chunks.
    const long long have = (long long)B * H * njobs;
    const int chunk = tc ? kLinTcChunk : C, from = tc ? 6 : 3;
    const long long want = tc ? num_sms : 2ll * num_sms;
    const int chunks = (int)(((long long)T + chunk - 1) / chunk);
    int n = 1;
    if (have > 0 && have * 2 <= want && chunks >= from) n = (int)std::min<long long>(want / have, chunks);
    if (n < 1) n = 1;
    const int per = std::max(1, (chunks + n - 1) / n);
    *seg_len = per * chunk;
    return std::max(1, (chunks + per - 1) / per);
}

cudaError_t launch_lin_carry(const LinArgs& a, cudaStream_t s, int* n) {
    const unsigned parts = (unsigned)std::min(16, (a.job[0].da * a.job[0].dc + kThreads - 1) / kThreads);
    lin_carry_kernel<<<dim3((unsigned)(a.B * a.H), parts, a.njobs), kThreads, 0, s>>>(a);
    ++*n;
    return cudaGetLastError();
}

cudaError_t launch_lin(const void* args, cudaStream_t s, int* nlaunch) {
    LinArgs a = *static_cast<const LinArgs*>(args);
    *nlaunch = 0;
    a.nseg = lin_segments(a.B, a.T, a.H, a.njobs, a.num_sms, true, &a.seg_len);
    if (lin_tc_ok(a)) {
        a.from_end = 1;
        return launch_lin_tc(a, s, nlaunch);
    }
    a.nseg = lin_segments(a.B, a.T, a.H, a.njobs, a.num_sms, false, &a.seg_len);
    return a.dt == DType::F32 ? run_type<float>(a, s, nlaunch) : run_type<bf16>(a, s, nlaunch);
}

cudaError_t launch_lin_step(const void* args, cudaStream_t s, int* nlaunch) {
    const LinStepArgs& a = *static_cast<const LinStepArgs*>(args);
    *nlaunch = 1;
    return a.dt == DType::F32 ? step_type<float>(a, s) : step_type<bf16>(a, s);
}

}  // namespace lstm
