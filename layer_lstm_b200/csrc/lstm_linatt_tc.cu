// Linear attention's products (lstm_ops.h, LinJob) in bf16 on the tensor cores
// (tcgen05), 128 steps of a (batch row, head) at a time.
//
//   P = a b^T (128 x 128 steps), out = D (a X + P' c), X^T <- g^m X^T + U,
//   U = (w c)^T b,
// with tau the step's place in the chunk in the product's own order, D_i =
// g^I(i), I(i) = min(tau_i + e, I*), P'_ij = P_ij g^(tau_i - tau_j - I(i)) for
// tau_j <= tau_i and w_j = g^(m - e - tau_j).  Taking D out of both terms lets
// one accumulator collect them.  g^-I stays below e^40 by I* = floor(40 /
// |log g|) (for out, not for X, decays below e^-40 act as e^-40); past I* the
// state's true share is below e^-20 of its size, 2e-9, far below the output's
// bf16 step.  X is
// float32 and stays in its owners' registers during a walk: U is read from
// tensor memory and added, and X's bf16 copy goes to shared memory as the next
// chunk's operand.  The weighted values w c enter U's product split in two
// bf16 parts (2^-16 of their size is lost), so the carried state is nearly
// what float32 products give; the scores and the state enter the outputs'
// products rounded once to bf16, as out itself is.  X is kept transposed, a
// thread per value column, so that states are read and written coalesced.
//
// Chunks end where the row's valid steps end, whatever the direction: the one
// partial chunk lies before time 0, where TMA fills zeros, and padded steps
// are never read.
//
// One block per SM walks (row, head, segment) items.  Warp 0 loads a, b, c by
// TMA; warp 1 issues P, a X and P' c; warp 2 issues U; warps 3-6 (a thread per
// step) turn P into P' and write out; warps 7-10 (a thread per value column)
// weight c, and carry X.  Tensor memory: P (P' over it) | out | U | w c.
//
// Bound: HBM (four rows of 2 d bytes a step).  A chunk's products are 2 to 4
// million multiply-adds of 8192 a clock, an eighth of its load time; what has
// to fit beside the loads are the two element passes, which is why they have
// four warps each and no common barrier.
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "lstm_linatt.cuh"
#include "lstm_ops.h"
#include "lstm_tc.cuh"

namespace lstm {
namespace {

constexpr int kC = kLinTcChunk;        // steps a chunk
constexpr int kThreadsTc = 352;
constexpr int kTab = 400, kTabZero = 130;   // g^(n), n from -130 to 269

struct Params {
    LinArgs g;
    int map_a[3], map_b[3], map_c[3];   // tensor map of each job's operands
    int items;
    int mode;
    int reset;                          // first launch of a call: the status word starts anew
    int* status;
    uint64_t timeout_ns;
};

struct alignas(64) Maps {
    CUtensorMap m[4];
};

// HALF: value sizes (dc) up to 64.  The two bf16 parts of w c are then one
// operand of 128 rows (lanes 0-63 the leading parts, 64-127 the remainders),
// and X is kept as the two sums that gives.  DA: key sizes up to 64 or 128.
template <bool HALF, int DA>
struct Cfg {
    static constexpr int DCP = HALF ? 64 : 128;
    static constexpr int A_BYTES = DA * 256, C_BYTES = DCP * 256;
    static constexpr int STAGE = 2 * A_BYTES + C_BYTES;
    static constexpr int X_BYTES = DA * 256;
    static constexpr int S = HALF && DA == 64 ? 3 : 2;
    static constexpr int XB = HALF || DA == 64 ? 2 : 1;    // copies of X
    static constexpr int TAB_BYTES = (2 * kC + kTab) * 4;
    static constexpr int BARS = 2 * S + 6 + 2 * XB;
    static constexpr size_t SMEM = (size_t)S * STAGE + XB * X_BYTES + TAB_BYTES + BARS * 8 + 16;
    static constexpr int cP = 0, cO = 128, cU = 128 + DCP, cW = cU + DA;   // tensor-memory columns
};
static_assert(Cfg<false, 128>::SMEM <= 232448, "shared memory of one block");

// The decay that the outputs are formed with.
__device__ __forceinline__ float out_decay(float ld) { return ld < -40.0f ? -40.0f : ld; }

struct Walk {
    LinItem it;
    int len, c0, c1, nct;   // chunks [c0, c1) of the row's nct
    int pad;                // steps by which nct chunks exceed len
    int b;
};

__device__ __forceinline__ void walk_of(const Params& p, int item, Walk& w) {
    lin_item(p.g, p.mode, (unsigned)item, w.it);
    const unsigned bh = ((unsigned)item / (unsigned)p.g.nseg) % (unsigned)(p.g.B * p.g.H);
    w.b = (int)(bh / (unsigned)p.g.H);
    w.len = lin_length(p.g, w.b);
    w.nct = (w.len + kC - 1) / kC;
    w.pad = w.nct * kC - w.len;
    const int seg = item % p.g.nseg, per = p.g.seg_len / kC;
    w.c0 = min(seg * per, w.nct);
    w.c1 = min(w.c0 + per, w.nct);
}

// Time of a chunk's first row (negative in the partial chunk).
__device__ __forceinline__ int chunk_time(const Walk& w, int c, int reverse) {
    return reverse ? w.len - kC * (c + 1) : w.len - kC * (w.nct - c);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lo_half(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_half(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

template <bool HALF, int DA>
__global__ void __launch_bounds__(kThreadsTc, 1)
    lin_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    using Cf = Cfg<HALF, DA>;
    constexpr int S = Cf::S, XB = Cf::XB, DCP = Cf::DCP;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* sX = smem + S * Cf::STAGE;
    float* sw = reinterpret_cast<float*>(sX + XB * Cf::X_BYTES);   // w_j: whole chunks, the reverse's partial one
    float* sf = sw + 2 * kC;                                        // factors of P
    uint64_t* full = reinterpret_cast<uint64_t*>(sf + kTab);
    uint64_t* empty = full + S;
    uint64_t* bP = empty + S;      // P computed
    uint64_t* bPb = bP + 1;        // P' written
    uint64_t* bO = bPb + 1;        // out computed
    uint64_t* bOf = bO + 1;        // out read
    uint64_t* bW = bOf + 1;        // w c written
    uint64_t* bU = bW + 1;         // U computed
    uint64_t* bX = bU + 1;         // [XB] X written
    uint64_t* bM2 = bX + XB;       // [XB] a X computed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bM2 + XB);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool outs = p.mode != kLinStates;   // outputs wanted, not only states
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], outs ? 2 : 1);
        }
        tc::mbar_init(bP, 1);
        tc::mbar_init(bPb, 4);
        tc::mbar_init(bO, 1);
        tc::mbar_init(bOf, 4);
        tc::mbar_init(bW, 4);
        tc::mbar_init(bU, 1);
        for (int i = 0; i < XB; ++i) {
            tc::mbar_init(&bX[i], 4);
            tc::mbar_init(&bM2[i], 1);
        }
        *abort_flag = 0;
        tc::fence_mbar_init();
        // a bounded wait elsewhere gives up no sooner than its limit after this
        if (p.reset && blockIdx.x == 0) *p.status = kStatusOk;
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto wait = [&](uint64_t* bar, int phase) {
        return tc::mbar_wait(bar, (uint32_t)(phase & 1), abort_flag, p.status, p.timeout_ns);
    };

    if (warp == 0) {
        // ------------------------------------------------------------- loads
        if (lane == 0) {
            int n = 0;
            bool ok = true;
            for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x) {
                Walk w;
                walk_of(p, item, w);
                const LinJob& J = p.g.job[w.it.job];
                const CUtensorMap* ma = &maps.m[p.map_a[w.it.job]];
                const CUtensorMap* mb = &maps.m[p.map_b[w.it.job]];
                const CUtensorMap* mc = &maps.m[p.map_c[w.it.job]];
                const int na = (J.da + 63) / 64, nc = (J.dc + 63) / 64;
                for (int c = w.c0; c < w.c1; ++c, ++n) {
                    const int s = n % S;
                    if (!wait(&empty[s], n / S + 1)) {
                        ok = false;
                        break;
                    }
                    unsigned char* st = smem + s * Cf::STAGE;
                    tc::mbar_arrive_expect_tx(&full[s], (uint32_t)(((outs ? 2 : 1) * na + nc) * 16384));
                    const int t = chunk_time(w, c, J.reverse);
                    for (int k = 0; k < na; ++k) {
                        const int x = w.it.h * J.da + 64 * k;
                        tc::tma_load_3d(st + Cf::A_BYTES + k * 16384, mb, x, t, w.b, &full[s]);
                        if (outs) tc::tma_load_3d(st + k * 16384, ma, x, t, w.b, &full[s]);
                    }
                    for (int k = 0; k < nc; ++k)
                        tc::tma_load_3d(st + 2 * Cf::A_BYTES + k * 16384, mc, w.it.h * J.dc + 64 * k, t, w.b, &full[s]);
                }
            }
            if (*abort_flag) {   // copies in flight land before shared memory is released
                const uint64_t t0 = globaltimer_ns();
                for (int k = n > S ? n - S : 0; k < n; ++k)
                    while (!tc::mbar_try_wait(&full[k % S], (uint32_t)((k / S) & 1)) &&
                           globaltimer_ns() - t0 < 100000000ull) {}
            }
        }
    } else if (warp == 1) {
        // --------------------------------------------- P, a X and P' c
        int n = 0, last = -1;
        bool ok = outs;
        for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x) {
            Walk w;
            walk_of(p, item, w);
            const LinJob& J = p.g.job[w.it.job];
            const int ka = J.da / 16;
            const uint32_t idP = tc::instr_desc(1, 128, 128), idX = tc::instr_desc(1, 128, J.dc), idO = idX | (1u << 16);
            for (int c = w.c0; c < w.c1; ++c, ++n) {
                const int s = n % S;
                const uint32_t sa = tc::smem_u32(smem + s * Cf::STAGE), sb = sa + Cf::A_BYTES, sc = sb + Cf::A_BYTES;
                const uint32_t sx = tc::smem_u32(sX + (n % XB) * Cf::X_BYTES);
                // P lies over the P' that the last chunk's product reads
                if (!wait(&full[s], n / S) || (n > 0 && !wait(bO, n - 1))) { ok = false; break; }
                tc::tc_fence_after();
                if (tc::elect_one()) {
                    for (int k = 0; k < ka; ++k) {
                        const uint32_t off = (uint32_t)((k >> 2) * 16384 + (k & 3) * 32);
                        tc::mma_bf16(tmem + Cf::cP, tc::smem_desc_sw128(sa + off), tc::smem_desc_sw128(sb + off), idP, k != 0);
                    }
                    tc::mma_commit(bP);
                }
                __syncwarp();
                last = n;
                if (!wait(&bX[n % XB], n / XB) || (n > 0 && !wait(bOf, n - 1))) { ok = false; break; }
                tc::tc_fence_after();
                if (tc::elect_one()) {
                    for (int h = 0; h < (HALF ? 2 : 1); ++h)
                        for (int k = 0; k < ka; ++k) {
                            const uint32_t off = (uint32_t)((k >> 2) * 16384 + (k & 3) * 32);
                            tc::mma_bf16(tmem + Cf::cO, tc::smem_desc_sw128(sa + off),
                                         tc::smem_desc_sw128(sx + (uint32_t)(h * 8192) + off), idX, (h | k) != 0);
                        }
                    tc::mma_commit(&bM2[n % XB]);
                }
                __syncwarp();
                if (!wait(bPb, n)) { ok = false; break; }
                tc::tc_fence_after();
                if (tc::elect_one()) {
                    for (int k = 0; k < kC / 16; ++k)
                        tc::mma_bf16_ts(tmem + Cf::cO, tmem + Cf::cP + 8 * k,
                                        tc::smem_desc_sw128_mn(sc + (uint32_t)(k * 2048), 16384), idO, 1);
                    tc::mma_commit(bO);
                    tc::mma_commit(&empty[s]);
                }
                __syncwarp();
            }
        }
        if (*abort_flag && last >= 0) {   // products in flight end before tensor memory is released
            if (tc::elect_one()) tc::mma_commit(&empty[last % S]);
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 1000000ull) {}
        }
    } else if (warp == 2) {
        // ---------------------------------------------------------------- U
        int n = 0;
        bool ok = true;
        for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x) {
            Walk w;
            walk_of(p, item, w);
            const uint32_t id = tc::instr_desc(1, 128, p.g.job[w.it.job].da) | (1u << 16);
            for (int c = w.c0; c < w.c1; ++c, ++n) {
                const int s = n % S;
                const uint32_t sb = tc::smem_u32(smem + s * Cf::STAGE) + Cf::A_BYTES;
                if (!wait(&full[s], n / S) || !wait(bW, n)) { ok = false; break; }
                tc::tc_fence_after();
                if (tc::elect_one()) {
                    for (int h = 0; h < (HALF ? 1 : 2); ++h)
                        for (int k = 0; k < kC / 16; ++k)
                            tc::mma_bf16_ts(tmem + Cf::cU, tmem + Cf::cW + h * 64 + 8 * k,
                                            tc::smem_desc_sw128_mn(sb + (uint32_t)(k * 2048), 16384), id, (h | k) != 0);
                    tc::mma_commit(bU);
                    tc::mma_commit(&empty[s]);
                }
                __syncwarp();
            }
        }
        if (*abort_flag) {
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 1000000ull) {}
        }
    } else if (warp < 7) {
        // ------------------------------------------------ P -> P', out
        const int q = warp & 3, i = q * 32 + lane, me = (warp - 3) * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
        int n = 0;
        bool ok = outs;
        for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x) {
            Walk w;
            walk_of(p, item, w);
            const LinJob& J = p.g.job[w.it.job];
            const int e = w.it.e, rev = J.reverse;
            const float ld = out_decay(w.it.ld);
            // I*: decays stronger than e^-40 over a chunk take their factors one by one
            const bool by_column = !(ld * (float)kC < -40.0f);
            const int cap = by_column ? 2 * kC : max(1, (int)(40.0f / -ld));
            const int first_pad = !rev && w.c0 == 0 ? w.pad : 0;   // steps missing at the front of the first chunk
            bf16* o = static_cast<bf16*>(J.o) + (size_t)w.it.h * J.dc;
            tc::named_bar_sync(1, 128);   // the last item's factors are read
            if (by_column) {
                // g^(-tau_j - e): of the first chunk, then of the others
                const int tj = rev ? kC - 1 - me : me;
                sf[me] = expf(-ld * (float)(tj - first_pad + e)) * J.bscale;
                sf[kC + me] = expf(-ld * (float)(tj + e)) * J.bscale;
            } else {
                for (int k = me; k < kTab; k += 128)
                    sf[k] = expf(fminf(ld * (float)(k - kTabZero), 41.0f)) * J.bscale;
            }
            tc::named_bar_sync(1, 128);
            bool good = true;
            for (int c = w.c0; c < w.c1; ++c, ++n) {
                const int pad = c == w.c0 ? first_pad : 0;
                const int tau = rev ? kC - 1 - i : i - pad;
                const int I = min(tau + e, cap);
                if (!wait(bP, n)) { good = false; break; }
                tc::tc_fence_after();
                const float* fc = sf + (c == w.c0 ? 0 : kC);
#pragma unroll 1
                for (int kb = 0; kb < 4; ++kb) {
                    uint32_t r[16];
                    if (rev ? kb < q : kb > q) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) r[k] = 0;
                    } else {
                        float v[32];
                        float v0[16], v1[16];
                        tc::tmem_ld16(tl + Cf::cP + kb * 32, v0);
                        tc::tmem_ld16(tl + Cf::cP + kb * 32 + 16, v1);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k) { v[k] = v0[k]; v[16 + k] = v1[k]; }
                        if (by_column) {
#pragma unroll
                            for (int k = 0; k < 32; k += 4) {
                                const float4 f = *reinterpret_cast<const float4*>(fc + kb * 32 + k);
                                v[k] *= f.x; v[k + 1] *= f.y; v[k + 2] *= f.z; v[k + 3] *= f.w;
                            }
                        } else {
                            // n = tau_i - tau_j - I(i)
                            const float* ft = sf + kTabZero - I;
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                const int d = rev ? kb * 32 + k - i : i - kb * 32 - k;   // tau_i - tau_j
                                v[k] = d >= 0 ? v[k] * ft[d] : 0.0f;
                            }
                        }
                        if (kb == q) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (rev ? k < lane : k > lane) v[k] = 0.0f;
                        }
#pragma unroll
                        for (int k = 0; k < 16; ++k) r[k] = pack2(v[2 * k], v[2 * k + 1]);
                    }
                    tc::tmem_st16(tl + Cf::cP + kb * 16, r);
                }
                tc::tmem_st_wait();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bPb);
                const float f = expf(ld * (float)I) * J.oscale;
                if (!wait(bO, n)) { good = false; break; }
                tc::tc_fence_after();
                const int t = chunk_time(w, c, rev) + i;
                bf16* dst = o + w.it.row.padded(t) * J.ldo;
#pragma unroll
                for (int cb = 0; cb < DCP / 32; ++cb) {
                    if (cb * 32 >= J.dc) break;
                    float v[16], u[16];
                    tc::tmem_ld16(tl + Cf::cO + cb * 32, v);
                    tc::tmem_ld16(tl + Cf::cO + cb * 32 + 16, u);
                    tc::tmem_ld_wait();
                    if ((cb + 1) * 32 >= J.dc) {   // all of out is in registers
                        tc::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(bOf);
                    }
                    if (t >= 0) {
                        uint4* d4 = reinterpret_cast<uint4*>(dst + cb * 32);
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            d4[k] = make_uint4(pack2(v[8 * k] * f, v[8 * k + 1] * f), pack2(v[8 * k + 2] * f, v[8 * k + 3] * f),
                                               pack2(v[8 * k + 4] * f, v[8 * k + 5] * f), pack2(v[8 * k + 6] * f, v[8 * k + 7] * f));
                        if (cb * 32 + 16 < J.dc) {
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                d4[2 + k] = make_uint4(pack2(u[8 * k] * f, u[8 * k + 1] * f), pack2(u[8 * k + 2] * f, u[8 * k + 3] * f),
                                                       pack2(u[8 * k + 4] * f, u[8 * k + 5] * f), pack2(u[8 * k + 6] * f, u[8 * k + 7] * f));
                        }
                    }
                }
            }
            // padded steps
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const int per = J.dc / 8;
            for (int k = me; k < (w.it.pad1 - w.it.pad0) * per; k += 128)
                *reinterpret_cast<uint4*>(o + w.it.row.padded(w.it.pad0 + k / per) * J.ldo + (k % per) * 8) = zero;
            // the four warps leave together
            if (tc::named_bar_or(1, 128, !good)) ok = false;
        }
    } else {
        // ------------------------------------------------ w c, X
        const int q = warp & 3, l = q * 32 + lane, me = (warp - 7) * 32 + lane;
        const int r = HALF ? (l & 63) : l;          // value column
        const bool low = HALF && l >= 64;           // the remainders' half
        const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
        int n = 0;
        bool ok = true;
        for (int item = blockIdx.x; item < p.items && ok; item += gridDim.x) {
            Walk w;
            walk_of(p, item, w);
            const LinJob& J = p.g.job[w.it.job];
            const int e = w.it.e, rev = J.reverse;
            const float ld = w.it.ld;
            // w_j of whole chunks and of the reverse's partial one (the
            // forward's partial chunk has zeros where it has no steps)
            tc::named_bar_sync(2, 128);   // the last item's are read
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int x = rev ? (k ? kC - w.pad : kC) - (kC - 1 - me) : kC - e - me;
                sw[k * kC + me] = x >= 0 ? expf(ld * (float)x) * J.bscale : 0.0f;
            }
            float X[DA];
#pragma unroll
            for (int k = 0; k < DA; ++k) X[k] = 0.0f;
            if (w.it.init && !low && r < J.dc) {
                if (w.it.init_t) {
                    const float4* x0 = reinterpret_cast<const float4*>(w.it.init + (size_t)r * J.da);
#pragma unroll
                    for (int k = 0; k < DA; k += 4)
                        if (k < J.da) {
                            const float4 v = x0[k / 4];
                            X[k] = v.x; X[k + 1] = v.y; X[k + 2] = v.z; X[k + 3] = v.w;
                        }
                } else {
                    const float* x0 = w.it.init + r;
#pragma unroll
                    for (int k = 0; k < DA; ++k)
                        if (k < J.da) X[k] = x0[(size_t)k * J.dc];
                }
            }
            tc::named_bar_sync(2, 128);
            // X's bf16 copy for chunk n: 128-byte rows of 64 keys, swizzled
            auto put_x = [&]() {
                if (n >= XB && !wait(&bM2[n % XB], n / XB - 1)) return false;
                unsigned char* x = sX + (n % XB) * Cf::X_BYTES + l * 128;
#pragma unroll
                for (int k = 0; k < DA; k += 8)
                    *reinterpret_cast<uint4*>(x + (k >> 6) * 16384 + ((((k & 63) >> 3) ^ (l & 7)) << 4)) =
                        make_uint4(pack2(X[k], X[k + 1]), pack2(X[k + 2], X[k + 3]), pack2(X[k + 4], X[k + 5]),
                                   pack2(X[k + 6], X[k + 7]));
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bX[n % XB]);
                return true;
            };
            bool good = true;
            if (outs && w.c0 < w.c1) good = put_x();
            for (int c = w.c0; c < w.c1 && good; ++c) {
                const int m = c == (rev ? w.nct - 1 : 0) ? kC - w.pad : kC;
                const float* wj = sw + (rev && c == w.nct - 1 ? kC : 0);
                const int s = n % S;
                if (!wait(&full[s], n / S)) { good = false; break; }
                const unsigned char* sc = smem + s * Cf::STAGE + 2 * Cf::A_BYTES + (r >> 6) * 16384 + (r & 7) * 2;
                const int ch = (r & 63) >> 3;
#pragma unroll 1
                for (int jb = 0; jb < kC; jb += 32) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(wj + jb + k);
                        float v[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            v[u] = __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t*>(
                                                       sc + (jb + k + u) * 128 + ((ch ^ ((k + u) & 7)) << 4))
                                                   << 16);
                        v[0] *= f.x; v[1] *= f.y; v[2] *= f.z; v[3] *= f.w;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const uint32_t h = pack2(v[2 * u], v[2 * u + 1]);
                            hi[k / 2 + u] = h;
                            lo[k / 2 + u] = pack2(v[2 * u] - lo_half(h), v[2 * u + 1] - hi_half(h));
                        }
                    }
                    if constexpr (HALF) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) hi[k] = low ? lo[k] : hi[k];
                        tc::tmem_st16(tl + Cf::cW + jb / 2, hi);
                    } else {
                        tc::tmem_st16(tl + Cf::cW + jb / 2, hi);
                        tc::tmem_st16(tl + Cf::cW + 64 + jb / 2, lo);
                    }
                }
                tc::tmem_st_wait();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bW);
                const float gm = expf(ld * (float)m);
                if (!wait(bU, n)) { good = false; break; }
                tc::tc_fence_after();
#pragma unroll
                for (int cb = 0; cb < DA / 16; ++cb) {
                    if (cb * 16 >= J.da) break;
                    float v[16];
                    tc::tmem_ld16(tl + Cf::cU + cb * 16, v);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 16; ++k) X[cb * 16 + k] = fmaf(gm, X[cb * 16 + k], v[k]);
                }
                tc::tc_fence_before();
                ++n;
                if (outs && c + 1 < w.c1) good = put_x();   // the next chunk's
            }
            if (w.it.fin) {
                if constexpr (HALF) {
                    // the two sums are added in the place of X's copies, once
                    // the last products that read those have ended
                    float* x = reinterpret_cast<float*>(sX);
                    if (outs)
                        for (int k = 1; k <= XB; ++k)
                            if (n - k >= 0 && good) good = wait(&bM2[(n - k) % XB], (n - k) / XB);
                    if (low) {
#pragma unroll
                        for (int k = 0; k < DA; ++k) x[k * 64 + r] = X[k];
                    }
                    tc::named_bar_sync(2, 128);
                    if (!low) {
#pragma unroll
                        for (int k = 0; k < DA; ++k) X[k] += x[k * 64 + r];
                    }
                    tc::named_bar_sync(2, 128);
                }
                if (!low && r < J.dc) {
                    float* f = w.it.fin + r;
#pragma unroll
                    for (int k = 0; k < DA; ++k)
                        if (k < J.da) f[(size_t)k * J.dc] = X[k];
                }
            }
            // the four warps leave together
            if (tc::named_bar_or(2, 128, !good)) ok = false;
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    return fn;
}

// (inner, time, batch row) map of an operand: boxes of 64 columns, 128 times.
bool make_map(CUtensorMap* map, const LinArgs& g, const void* base, long long ld, long long inner) {
    const unsigned long long row = (unsigned long long)ld * 2;
    cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)g.T, (cuuint64_t)g.B};
    cuuint64_t strides[2] = {g.batch_first ? row : row * g.B, g.batch_first ? row * g.T : row};
    cuuint32_t box[3] = {64, (cuuint32_t)kC, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool HALF, int DA>
cudaError_t run(const Maps& maps, const Params& p, cudaStream_t s) {
    using Cf = Cfg<HALF, DA>;
    cudaError_t e = cudaFuncSetAttribute(lin_tc_kernel<HALF, DA>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Cf::SMEM);
    if (e != cudaSuccess) return e;
    lin_tc_kernel<HALF, DA><<<std::min(p.items, p.g.num_sms), kThreadsTc, Cf::SMEM, s>>>(maps, p);
    return cudaGetLastError();
}

// All products of `a` whose sizes take the same kernel, one launch.
cudaError_t run_mode(const LinArgs& a, int mode, cudaStream_t s, int* n) {
    for (int half = 0; half < 2; ++half)
        for (int da = 64; da <= 128; da += 64) {
            Params p{};
            Maps maps{};
            p.g = a;
            p.g.njobs = 0;
            int nmaps = 0;
            struct { const void* x; long long ld; int d; } have[4];
            auto map_of = [&](const void* x, long long ld, int d) {
                for (int i = 0; i < nmaps; ++i)
                    if (have[i].x == x && have[i].ld == ld && have[i].d == d) return i;
                if (nmaps == 4 || !make_map(&maps.m[nmaps], a, x, ld, (long long)a.H * d)) return -1;
                have[nmaps] = {x, ld, d};
                return nmaps++;
            };
            int first = -1;
            for (int j = 0; j < a.njobs; ++j) {
                const LinJob& J = a.job[j];
                if ((J.dc <= 64) != (half == 1) || (J.da <= 64) != (da == 64)) continue;
                const int k = p.g.njobs++;
                if (first < 0) first = j;
                p.g.job[k] = J;
                p.map_a[k] = map_of(J.a, J.lda, J.da);
                p.map_b[k] = map_of(J.b, J.ldb, J.da);
                p.map_c[k] = map_of(J.c, J.ldc, J.dc);
                if (p.map_a[k] < 0 || p.map_b[k] < 0 || p.map_c[k] < 0) return cudaErrorInvalidValue;
            }
            if (p.g.njobs == 0) continue;
            // the products of one launch are neighbours in `a`, and so are their states in the buffer
            p.g.buf = a.buf + (size_t)first * a.B * a.H * a.nseg * a.job[0].da * a.job[0].dc;
            p.items = a.B * a.H * p.g.njobs * a.nseg;
            p.mode = mode;
            p.reset = *n == 0;
            p.status = a.status;
            p.timeout_ns = a.timeout_ns;
            cudaError_t e = half ? (da == 64 ? run<true, 64>(maps, p, s) : run<true, 128>(maps, p, s))
                                 : (da == 64 ? run<false, 64>(maps, p, s) : run<false, 128>(maps, p, s));
            if (e != cudaSuccess) return e;
            ++*n;
        }
    return cudaSuccess;
}

bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace

bool lin_tc_ok(const LinArgs& a) {
    if (a.dt != DType::BF16 || a.T < 1 || !encode_fn()) return false;
    if ((long long)a.B * a.H * a.njobs * a.nseg > (1ll << 30)) return false;
    for (int j = 0; j < a.njobs; ++j) {
        const LinJob& J = a.job[j];
        // K steps and output columns of 16; a box of 64 columns inside the rows
        if (J.da % 16 || J.dc % 16 || a.H * std::min(J.da, J.dc) < 64) return false;
        if (J.lda % 8 || J.ldb % 8 || J.ldc % 8 || J.ldo % 8) return false;
        if (!on16(J.a) || !on16(J.b) || !on16(J.c) || !on16(J.o) || !on16(J.init)) return false;
        // strides of the maps stay below 2^40 bytes
        if (std::max({J.lda, J.ldb, J.ldc}) * 2 * std::max(a.B, a.T) >= (1ll << 40)) return false;
    }
    return true;
}

cudaError_t launch_lin_tc(const LinArgs& a, cudaStream_t s, int* n) {
    if (a.nseg <= 1) return run_mode(a, kLinWhole, s, n);
    cudaError_t e = run_mode(a, kLinStates, s, n);
    if (e != cudaSuccess) return e;
    if ((e = launch_lin_carry(a, s, n)) != cudaSuccess) return e;
    return run_mode(a, kLinSegments, s, n);
}

}  // namespace lstm
