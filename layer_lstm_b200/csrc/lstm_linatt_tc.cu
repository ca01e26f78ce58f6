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
// bf16 step.  X is float32 and stays in its owners' registers during a walk: U
// is read from tensor memory and added, and X's bf16 copy goes to shared memory
// as the next chunk's operand.  The weighted values w c enter U's product split
// in four bf16 parts, which hold all of float32, so the carried state is what
// float32 products give (2.5e-7 of it off; 1.5e-6 with two parts); the scores
// and the state enter the outputs' products rounded once to bf16, as out itself
// is.  X is kept transposed, a thread per value column, so that states are read
// and written coalesced.
//
// Chunks end where the row's valid steps end, whatever the direction: the one
// partial chunk lies before time 0, where TMA fills zeros, and padded steps
// are never read.
//
// One block per SM walks (row, head, segment) items; its warps are stages of a
// pipeline that runs across chunks and items, joined by mbarriers only:
//   warp 0 loads a, b, c and stores out by TMA; warp 1 issues P and P' c, warp 2
//   U, warp 3 a X;
//   warps 4-7 (a thread per step) turn P into P';
//   warps 8-11 (a thread per step) turn out into bf16, in the place of a;
//   warps 12-15 (a thread per value column) weight c, 32 steps at a time;
//   warps 16-19 (a thread per value column) carry X.
// Tensor memory: P (P' over it; two of them for value sizes up to 64) | out | U
// | w c (two sets of 32 steps).
//
// Bound: HBM (four rows of 2 d bytes a step; 1.5 us of an SM's share for 128
// steps of 64).  The products keep the tensor pipe busy for 0.7 us of that (M =
// 128 runs at N / 2 cycles an MMA).  What a chunk takes is 2.4 us: the seven
// programs share each scheduler, and their element passes and hand-overs run at
// the pace at which instructions arrive (32767 steps, 16 heads of 64: 74 us for
// the outputs, 3.3 TB/s, tensor pipe at 33 %, issue at 40 %; with one program
// for scores and outputs 20 % slower, with their loops unrolled 40 %).
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "lstm_linatt.cuh"
#include "lstm_ops.h"
#include "lstm_tc.cuh"

namespace lstm {
namespace {

constexpr int kC = kLinTcChunk;        // steps a chunk
constexpr int kThreadsTc = 640;
// Registers a thread of each group of four warps (96 at launch): the threads
// that carry X hold up to 128 sums.
constexpr int kRegsControl = 72, kRegsScore = 80, kRegsOut = 64, kRegsWeight = 80, kRegsCarry = 184;
static_assert(kRegsControl + kRegsScore + kRegsOut + kRegsWeight + kRegsCarry <= 5 * 96, "registers of the block");
constexpr int kSub = 32;               // steps weighted at a time
constexpr int kTab = 322, kTabZero = 192;   // g^(n), n from -192 to 129

struct Params {
    LinArgs g;
    int map_a[3], map_b[3], map_c[3];   // tensor map of each job's operands
    int tma_out[3];                     // out goes through shared memory and TMA (see run_mode)
    int nmaps;
    int items;
    int mode;
    int reset;                          // first launch of a call: the status word starts anew
    int* status;
    uint64_t timeout_ns;
    int skip_block, skip_chunk;         // this block's weighing warps withhold this chunk's arrivals (a test; -1: none)
};

struct alignas(64) Maps {
    CUtensorMap m[4];
    CUtensorMap o[3];   // the jobs' outputs
};

// HALF: value sizes (dc) up to 64.  An operand of 128 rows then holds two of
// the four bf16 parts of w c (lanes 0-63 one, 64-127 the other), and X is kept
// as the two sums that gives.  DA:
// key sizes up to 64 or 128.
template <bool HALF, int DA>
struct Cfg {
    static constexpr int DCP = HALF ? 64 : 128;
    static constexpr int A_BYTES = DA * 256, C_BYTES = DCP * 256;
    static constexpr int STAGE = 2 * A_BYTES + C_BYTES;
    static constexpr int X_BYTES = DA * 256;
    static constexpr int S = HALF && DA == 64 ? 3 : 2;
    static constexpr int XB = HALF || DA == 64 ? 2 : 1;    // copies of X
    static constexpr int PB = HALF ? 2 : 1;                // scores in tensor memory
    static constexpr int PARTS = HALF ? 2 : 4;             // operands that hold w c
    static constexpr int SETS = 2;                             // sets of 32 steps of them
    static constexpr int TAB_BYTES = (2 * 3 * kC / 2 + kTab) * 4;
    static constexpr int BARS = 4 * S + 4 + 2 * SETS + 2 * XB + 2 * PB;
    static constexpr size_t SMEM = (size_t)S * STAGE + XB * X_BYTES + TAB_BYTES + BARS * 8 + 48;
    // tensor-memory columns; a set of w c takes 16 of them for each operand
    static constexpr int cP = 0, cO = PB * 128, cU = cO + DCP, cW = cU + DA;
    static_assert(cW + SETS * PARTS * kSub / 2 <= 512, "tensor memory");
};
// (the largest is value sizes up to 64 with key sizes up to 128)
constexpr size_t kSmemMost = 232448;   // of one block
static_assert(Cfg<false, 64>::SMEM <= kSmemMost && Cfg<false, 128>::SMEM <= kSmemMost, "shared memory of one block");
static_assert(Cfg<true, 64>::SMEM <= kSmemMost && Cfg<true, 128>::SMEM <= kSmemMost, "shared memory of one block");

// The decay that the outputs are formed with, and I*.
__device__ __forceinline__ float out_decay(float ld) { return ld < -40.0f ? -40.0f : ld; }
__device__ __forceinline__ int power_cap(float ld) {
    return ld * (float)kC < -40.0f ? max(1, (int)(40.0f / -ld)) : 2 * kC;
}

// Where a block is in the list of items, ((job B + b) H + h) nseg + seg, as its
// digits; the next item is gridDim.x further, added digit by digit (a division
// per item and role would be a third of the kernel's code).
struct Walk {
    int item, seg, h, b, job;
    int len, c0, c1, nct;   // chunks [c0, c1) of the row's nct
    int pad;                // steps by which nct chunks exceed len

    __device__ __forceinline__ explicit Walk(const int* digits) {
        item = (int)blockIdx.x - (int)gridDim.x;
        seg = digits[0]; h = digits[1]; b = digits[2]; job = digits[3];
        c1 = 0;
    }
    // Moves to the block's next item; false at the end.  digits[4..7]: those of gridDim.x.
    __device__ __forceinline__ bool next(const Params& p, const int* digits) {
        if (item >= 0) {
            seg += digits[4];
            h += digits[5];
            b += digits[6];
            job += digits[7];
            if (seg >= p.g.nseg) { seg -= p.g.nseg; ++h; }
            if (h >= p.g.H) { h -= p.g.H; ++b; }
            if (b >= p.g.B) { b -= p.g.B; ++job; }
        }
        item += (int)gridDim.x;
        if (item >= p.items) return false;
        len = lin_length(p.g, b);
        nct = (len + kC - 1) / kC;
        pad = nct * kC - len;
        const int per = p.g.seg_len / kC;
        c0 = min(seg * per, nct);
        c1 = min(c0 + per, nct);
        return true;
    }
};
// Row of the arrays that holds batch row b at time t.
__device__ __forceinline__ long long time_row(const Params& p, int b, int t) {
    return p.g.batch_first ? (long long)b * p.g.T + t : (long long)t * p.g.B + b;
}
// An item's states: the first, from the caller or the segments' buffer, and
// where the last goes.
__device__ __forceinline__ void state_of(const Params& p, const Walk& w, const float*& init, bool& init_t, float*& fin) {
    const LinJob& J = p.g.job[w.job];
    const size_t bh = (size_t)w.b * p.g.H + w.h, n = (size_t)J.da * J.dc;
    if (p.mode == kLinWhole) {
        init = J.init ? J.init + bh * n : nullptr;
        init_t = J.init_t != 0;
        fin = J.fin ? J.fin + bh * n : nullptr;
    } else {
        float* own = p.g.buf + lin_buf_offset(p.g, w.job) + (bh * p.g.nseg + w.seg) * n;
        init = p.mode == kLinStates ? nullptr : own;
        init_t = false;
        fin = p.mode == kLinStates ? own : nullptr;
    }
}
// The digits of item `n`.
__device__ __forceinline__ void digits_of(const Params& p, int n, int* d) {
    d[0] = n % p.g.nseg; n /= p.g.nseg;
    d[1] = n % p.g.H; n /= p.g.H;
    d[2] = n % p.g.B;
    d[3] = n / p.g.B;
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

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t*>(&v); }

// Four 8 x 8 matrices of 16-bit elements, transposed: lane t gets elements
// (2 (t % 4), t / 4) and (2 (t % 4) + 1, t / 4) of each.
__device__ __forceinline__ void ldmatrix_t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void lds4(const uint32_t* p, uint32_t (&r)[4]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    r[0] = q.x; r[1] = q.y; r[2] = q.z; r[3] = q.w;
}

// 16 lanes x 16 columns of tensor memory from the registers of four such
// matrices side by side: lane t holds rows t / 4 and t / 4 + 8, column t % 4
// of each group of four.
__device__ __forceinline__ void tmem_st_rows(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Columns of this thread's lane of tensor memory: the wait of one load is some
// 300 cycles here, however many columns it brings.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, "
        "%21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31 "
        "}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]),
          "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]),
          "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]),
          "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr)
        : "memory");
}

// Tile of shared memory to box {c0, c1, c2} of a tensor, in this thread's bulk group.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(tc::smem_u32(src))
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// This thread's stores have read shared memory / have ended.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Two float32 products at once.
__device__ __forceinline__ void mul2(float& a, float& b, unsigned long long f) {
    unsigned long long x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(x), "l"(f));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}

template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Bounded waits in few instructions: this kernel's warps run seven programs on
// each scheduler, and its speed hangs on how much of them the instruction
// caches hold.  The loads' warp keeps the time: in its own waits, which end only
// with the other roles' progress, and then in a wait for the other warps' ends.
// When it gives up it sets the flag that every other wait looks at.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort) {
    uint32_t i = 0;
#pragma unroll 1
    while (!tc::mbar_try_wait(bar, parity))
        if ((++i & 255u) == 0 && *abort) return false;
    return true;
}

// The chunks of a block's items, one after another.
struct Chunks {
    int c;
    Walk w;
    __device__ __forceinline__ explicit Chunks(const int* digits) : c(0), w(digits) {}
    // Moves to the next chunk; false at the end.
    __device__ __forceinline__ bool next(const Params& p, const int* digits) {
        ++c;
#pragma unroll 1
        while (c >= w.c1) {
            if (!w.next(p, digits)) return false;
            c = w.c0;
        }
        return true;
    }
};

// ENDS: every item forms U in its last chunk, with no test.  Without it, the
// last chunk of a product whose last state nobody asked for forms none: of
// the two chunks of 256 steps a half (forward and backward of 32 rows, 8 heads
// of 128, lengths 128 to 256: 86.6 -> 82.8 us).  The test costs where chunks
// are many: one row of 32767 steps, 16 heads of 64, in segments 121 -> 127 us,
// so segments have ENDS.  256 rows of 64 steps, 8 heads of 64, with a last
// state (one chunk each): 79.4 us with it, 81.5 without.
template <bool HALF, int DA, bool ENDS>
__global__ void __launch_bounds__(kThreadsTc, 1)
    lin_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    using Cf = Cfg<HALF, DA>;
    constexpr int S = Cf::S, XB = Cf::XB, PB = Cf::PB, SETS = Cf::SETS;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* sX = smem + S * Cf::STAGE;
    // w of each pair of steps in three bf16 parts [2][3][kC / 2]: whole chunks,
    // the reverse's partial one
    uint32_t* sw = reinterpret_cast<uint32_t*>(sX + XB * Cf::X_BYTES);
    float* sf = reinterpret_cast<float*>(sw + 2 * 3 * kC / 2);      // factors of P
    uint64_t* full = reinterpret_cast<uint64_t*>(sf + kTab);
    uint64_t* empty = full + S;
    uint64_t* bS = empty + S;      // [S] out written in the place of a
    uint64_t* bP = bS + S;         // [PB] P computed
    uint64_t* bPb = bP + PB;       // [PB] P' written
    uint64_t* bO = bPb + PB;       // out computed
    uint64_t* bOf = bO + 1;        // out read
    uint64_t* bW = bOf + 1;        // [SETS] w c written
    uint64_t* bWf = bW + SETS;     // [SETS] w c read by the products
    uint64_t* bU = bWf + SETS;     // U computed
    uint64_t* bUf = bU + 1;        // U read
    uint64_t* bX = bUf + 1;        // [XB] X written
    uint64_t* bM2 = bX + XB;       // [XB] a X computed
    uint64_t* bK = bM2 + XB;       // [S] the weighing warps have seen a chunk without U
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bK + S);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* ended = reinterpret_cast<volatile int*>(tmem_slot + 2);   // warps that are done
    int* digits = reinterpret_cast<int*>(tmem_slot + 3);   // [8]: the first item's, gridDim.x's

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool outs = p.mode != kLinStates;   // outputs wanted, not only states
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.nmaps; ++i) tc::prefetch_tmap(&maps.m[i]);
        for (int s = 0; s < S; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], outs ? 2 : 1);
            tc::mbar_init(&bS[s], 4);
            tc::mbar_init(&bK[s], 4);
        }
        for (int i = 0; i < PB; ++i) {
            tc::mbar_init(&bP[i], 1);
            tc::mbar_init(&bPb[i], 4);
        }
        tc::mbar_init(bO, 1);
        tc::mbar_init(bOf, 4);
        for (int i = 0; i < SETS; ++i) {
            tc::mbar_init(&bW[i], 4);
            tc::mbar_init(&bWf[i], 1);
        }
        tc::mbar_init(bU, 1);
        tc::mbar_init(bUf, 4);
        for (int i = 0; i < XB; ++i) {
            tc::mbar_init(&bX[i], 4);
            tc::mbar_init(&bM2[i], 1);
        }
        *abort_flag = 0;
        *ended = 0;
        digits_of(p, (int)blockIdx.x, digits);
        digits_of(p, (int)gridDim.x, digits + 4);
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
    // A warp gives up as a whole: a lane that left alone would leave the others
    // in front of a warp-wide instruction.  (The votes take 0.7 of 29.5 us with 32
    // rows of 256 steps, 8 heads of 128.)
    auto poll = [&](uint64_t* bar, int phase) { return wait_phase(bar, (uint32_t)(phase & 1), abort_flag); };
    auto wait = [&](uint64_t* bar, int phase) { return __all_sync(0xffffffffu, poll(bar, phase)) != 0; };
    auto wait2 = [&](uint64_t* bar, int phase, uint64_t* bar2, int phase2) {
        return __all_sync(0xffffffffu, poll(bar, phase) && poll(bar2, phase2)) != 0;
    };
    // descriptor of `d` moved by `bytes`
    auto at = [](uint64_t d, uint32_t bytes) { return d + (bytes >> 4); };

    if (warp < 4) {
        regs_dec<kRegsControl>();
        if (warp == 0) {
            // ------------------------------------------------- loads, stores
            // (the whole warp waits, one lane issues: a wait by one lane of a
            // diverged warp takes 600 cycles, by the warp 100)
            auto wait_timed = [&](uint64_t* bar, int phase) {
                return __all_sync(0xffffffffu, tc::mbar_wait(bar, (uint32_t)(phase & 1), abort_flag, p.status,
                                                             p.timeout_ns)) != 0;
            };
            int n = 0;
            Chunks k(digits);
            // where out of the chunk that holds a stage goes: job (-1:
            // nowhere by TMA), columns, time, batch row
            int oj[S], ox[S], ot[S], ob[S];
#pragma unroll
            for (int s = 0; s < S; ++s) oj[s] = -1;
            auto store = [&](int s, int nn) {   // out of chunk nn
                if (!wait_timed(&bS[s], nn / S)) return false;
                int j = -1, x = 0, t = 0, b = 0;
#pragma unroll
                for (int i = 0; i < S; ++i)
                    if (i == s) { j = oj[i]; x = ox[i]; t = ot[i]; b = ob[i]; }
                if (j >= 0 && lane == 0) {
                    tma_store_3d(&maps.o[j], smem + s * Cf::STAGE, x, t, b);
                    if (p.g.job[j].dc > 64) tma_store_3d(&maps.o[j], smem + s * Cf::STAGE + 16384, x + 64, t, b);
                    bulk_commit();
                    bulk_wait_read();
                }
                __syncwarp();
                return true;
            };
            bool ok = true;
            for (; k.next(p, digits); ++n) {
                const int jn = k.w.job, h = k.w.h;
                const LinJob& J = p.g.job[jn];
                const int s = n % S;
                if (!wait_timed(&empty[s], n / S + 1)) { ok = false; break; }
                unsigned char* st = smem + s * Cf::STAGE;
                const int t = chunk_time(k.w, k.c, J.reverse);
                const bool a2 = DA == 128 && J.da > 64, c2 = !HALF && J.dc > 64;
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(&full[s], (uint32_t)((outs ? 2 : 1) * (a2 ? 2 : 1) + (c2 ? 2 : 1)) * 16384u);
                    const CUtensorMap* mb = &maps.m[p.map_b[jn]];
                    const CUtensorMap* mc = &maps.m[p.map_c[jn]];
                    tc::tma_load_3d(st + Cf::A_BYTES, mb, h * J.da, t, k.w.b, &full[s]);
                    if (a2) tc::tma_load_3d(st + Cf::A_BYTES + 16384, mb, h * J.da + 64, t, k.w.b, &full[s]);
                    tc::tma_load_3d(st + 2 * Cf::A_BYTES, mc, h * J.dc, t, k.w.b, &full[s]);
                    if (c2) tc::tma_load_3d(st + 2 * Cf::A_BYTES + 16384, mc, h * J.dc + 64, t, k.w.b, &full[s]);
                }
                __syncwarp();
                if (outs) {
                    // out of the stage's last chunk leaves before a comes in
                    if (n >= S && !store(s, n - S)) { ok = false; break; }
#pragma unroll
                    for (int i = 0; i < S; ++i)
                        if (i == s) {
                            oj[i] = p.tma_out[jn] && t >= 0 ? jn : -1;
                            ox[i] = h * J.dc; ot[i] = t; ob[i] = k.w.b;
                        }
                    if (lane == 0) {
                        const CUtensorMap* ma = &maps.m[p.map_a[jn]];
                        tc::tma_load_3d(st, ma, h * J.da, t, k.w.b, &full[s]);
                        if (a2) tc::tma_load_3d(st + 16384, ma, h * J.da + 64, t, k.w.b, &full[s]);
                    }
                    __syncwarp();
                }
            }
            if (outs && ok) {
#pragma unroll 1
                for (int i = n > S ? n - S : 0; i < n && ok; ++i) ok = store(i % S, i);
            }
            // keeps the time for the warps that are still at work
            const uint64_t t1 = globaltimer_ns();
            while (*ended < kThreadsTc / 32 - 1) {
                if (globaltimer_ns() - t1 > p.timeout_ns && !*abort_flag) {
                    atomicCAS(p.status, kStatusOk, kStatusTimeout);
                    *abort_flag = 1;
                }
            }
            __syncwarp();
            if (lane == 0) bulk_wait_all();
            if (*abort_flag) {   // copies in flight land before shared memory is released
                const uint64_t t0 = globaltimer_ns();
                for (int i = n > S ? n - S : 0; i <= n; ++i)
                    while (!tc::mbar_try_wait(&full[i % S], (uint32_t)((i / S) & 1)) &&
                           globaltimer_ns() - t0 < 100000000ull) {}
                // (a stage that got only a part of its loads has them ended by then)
            }
        } else if (warp == 1 && outs) {
            // ------------------------------------------------- P and P' c
            int n = 0;          // chunk of P' c
            int np = 0;         // chunk of P
            Chunks k(digits), kp(digits);
            // P of chunk np; it lies over the P' of PB chunks before, whose product has ended
            auto scores = [&]() {
                if (!kp.next(p, digits)) return true;
                if (!wait(&full[np % S], np / S)) return false;
                tc::tc_fence_after();
                const int ka = p.g.job[kp.w.job].da / 16;
                const uint64_t da = tc::smem_desc_sw128(tc::smem_u32(smem + (np % S) * Cf::STAGE));
                const uint64_t db = at(da, Cf::A_BYTES);
                const uint32_t id = tc::instr_desc(1, 128, 128), d = tmem + Cf::cP + (np % PB) * 128;
                if (tc::elect_one()) {
#pragma unroll 2
                    for (int i = 0; i < ka; ++i) {
                        const uint32_t off = (uint32_t)((i >> 2) * 16384 + (i & 3) * 32);
                        tc::mma_bf16(d, at(da, off), at(db, off), id, i != 0);
                    }
                    tc::mma_commit(&bP[np % PB]);
                }
                __syncwarp();
                ++np;
                return true;
            };
            bool ok = scores();
            for (; ok && k.next(p, digits); ++n) {
                const int s = n % S;
                const uint64_t dc = tc::smem_desc_sw128_mn(tc::smem_u32(smem + s * Cf::STAGE + 2 * Cf::A_BYTES), 16384);
                const uint32_t id = tc::instr_desc(1, 128, p.g.job[k.w.job].dc) | (1u << 16);
                // with two score buffers the next chunk's product runs beside this chunk's P'
                if (PB == 2 && ((n > 0 && !wait(bO, n - 1)) || !scores())) break;
                // out's accumulator already holds a X
                if (!wait2(&bM2[n % XB], n / XB, &bPb[n % PB], n / PB)) break;
                tc::tc_fence_after();
                if (tc::elect_one()) {
#pragma unroll 2
                    for (int i = 0; i < kC / 16; ++i)
                        tc::mma_bf16_ts(tmem + Cf::cO, tmem + Cf::cP + (n % PB) * 128 + 8 * i, at(dc, i * 2048), id, 1);
                    tc::mma_commit(bO);
                    tc::mma_commit(&empty[s]);
                }
                __syncwarp();
                if (PB == 1 && (!wait(bO, n) || !scores())) break;
            }
            if (*abort_flag) {   // products in flight end before tensor memory is released
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 1000000ull) {}
            }
        } else if (warp == 3 && outs) {
            // ----------------------------------------------------------- a X
            int n = 0;
            Chunks k(digits);
            for (; k.next(p, digits); ++n) {
                const LinJob& J = p.g.job[k.w.job];
                const int s = n % S, ka = J.da / 16;
                const uint64_t da = tc::smem_desc_sw128(tc::smem_u32(smem + s * Cf::STAGE));
                const uint64_t dx = tc::smem_desc_sw128(tc::smem_u32(sX + (n % XB) * Cf::X_BYTES));
                const uint32_t id = tc::instr_desc(1, 128, J.dc);
                // (the phase before the first counts as ended)
                if (!__all_sync(0xffffffffu, poll(&full[s], n / S) && poll(&bX[n % XB], n / XB) && poll(bOf, n + 1))) break;
                tc::tc_fence_after();
                if (tc::elect_one()) {
#pragma unroll 1
                    for (int h = 0; h < (HALF ? 2 : 1); ++h)
#pragma unroll 2
                        for (int i = 0; i < ka; ++i) {
                            const uint32_t off = (uint32_t)((i >> 2) * 16384 + (i & 3) * 32);
                            tc::mma_bf16(tmem + Cf::cO, at(da, off), at(dx, off + h * 8192), id, (h | i) != 0);
                        }
                    tc::mma_commit(&bM2[n % XB]);
                }
                __syncwarp();
            }
            if (*abort_flag) {
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 1000000ull) {}
            }
        } else if (warp == 2) {
            // ------------------------------------------------------------ U
            int n = 0, nu = 0;   // chunk, U
            uint32_t seen = 0;   // phase of each stage's bK
            Chunks k(digits);
            bool ok = true;
            for (; ok && k.next(p, digits); ++n) {
                const int s = n % S;
                if (!ENDS && k.c + 1 == k.w.c1 && p.g.job[k.w.job].fin == nullptr) {
                    // nothing else of such a chunk waits for the weighing warps:
                    // the stage stays until they have looked at it, so that
                    // full[s] cannot run two phases ahead of them
                    if (!wait2(&full[s], n / S, &bK[s], (int)(seen >> s))) break;
                    seen ^= 1u << s;
                    if (lane == 0) tc::mbar_arrive(&empty[s]);
                    __syncwarp();
                    continue;
                }
                const uint64_t db = tc::smem_desc_sw128_mn(tc::smem_u32(smem + s * Cf::STAGE) + Cf::A_BYTES, 16384);
                const uint32_t id = tc::instr_desc(1, 128, p.g.job[k.w.job].da) | (1u << 16);
                if (!wait2(&full[s], n / S, bUf, nu + 1)) break;   // (the phase before the first counts as ended)
#pragma unroll 1
                for (int r = 0; r < kC / kSub; ++r) {
                    const int set = r % SETS, turn = nu * (kC / kSub / SETS) + r / SETS;
                    if (!wait(&bW[set], turn)) { ok = false; break; }
                    tc::tc_fence_after();
                    if (tc::elect_one()) {
#pragma unroll
                        for (int h = 0; h < Cf::PARTS; ++h)
#pragma unroll
                            for (int i = 0; i < kSub / 16; ++i)
                                tc::mma_bf16_ts(tmem + Cf::cU, tmem + Cf::cW + (set * Cf::PARTS + h) * (kSub / 2) + 8 * i,
                                                at(db, (uint32_t)(r * kSub + 16 * i) * 128), id, (r | h | i) != 0);
                        tc::mma_commit(&bWf[set]);
                        if (r == kC / kSub - 1) {
                            tc::mma_commit(bU);
                            tc::mma_commit(&empty[s]);
                        }
                    }
                    __syncwarp();
                }
                ++nu;
            }
            if (*abort_flag) {
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 1000000ull) {}
            }
        }
    } else if (warp < 8) {
        // ------------------------------------------------ P -> P'
        regs_dec<kRegsScore>();
        const int q = warp & 3, i = q * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
        int n = 0;
        bool ok = outs;
        Walk w(digits);
        while (ok && w.next(p, digits)) {
            const LinJob& J = p.g.job[w.job];
            const int rev = J.reverse, e = rev ? 0 : 1;
            const float ld = out_decay(lin_log_decay(p.g.log_decay[w.h]));
            const int cap = power_cap(ld);
            // decays stronger than e^-40 over a chunk take their factors one by one
            const bool by_column = cap > kC;
            const int first_pad = !rev && w.c0 == 0 ? w.pad : 0;   // steps missing at the front of the first chunk
            tc::named_bar_sync(1, 128);   // the last item's factors are read
            if (by_column) {
                // g^(-tau_j - e): of the first chunk, then of the others
                const int tj = rev ? kC - 1 - i : i;
                sf[i] = expf(-ld * (float)(tj - first_pad + e)) * J.bscale;
                sf[kC + i] = expf(-ld * (float)(tj + e)) * J.bscale;
            } else {
#pragma unroll 1
                for (int k = i; k < kTab; k += 128)
                    sf[k] = expf(fminf(ld * (float)(k - kTabZero), 41.0f)) * J.bscale;
            }
            tc::named_bar_sync(1, 128);
            bool good = true;
#pragma unroll 1
            for (int c = w.c0; c < w.c1; ++c, ++n) {
                if (!wait(&bP[n % PB], n / PB)) { good = false; break; }
                tc::tc_fence_after();
                const uint32_t tp = tl + Cf::cP + (n % PB) * 128;
                const int pad = c == w.c0 ? first_pad : 0;
                const float* fc = sf + (c == w.c0 ? 0 : kC);
                const float* ft = sf + kTabZero - min(max(rev ? kC - 1 - i : i - pad, 0) + e, cap);
                // blocks of 32 columns that the mask leaves: up to the diagonal
                // one, or from it on; the next one's scores are on their way
                // while a block is weighed
                const int k0 = rev ? q : 0, k1 = rev ? 4 : q + 1;
                float v[32];
                uint32_t r[16];
                tmem_ld(tp + k0 * 32, v);
#pragma unroll 1
                for (int kb = k0; kb < k1; ++kb) {
                    tc::tmem_ld_wait();
                    if (by_column) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(fc + kb * 32 + k);
                            mul2(v[k], v[k + 1], f.x);
                            mul2(v[k + 2], v[k + 3], f.y);
                        }
                    } else {
                        // by tau_i - tau_j (what the mask takes lies at negative ones)
                        const float* fi = ft + (rev ? kb * 32 - i : i - kb * 32);
                        const int step = rev ? 1 : -1;
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] *= fi[k * step];
                    }
                    if (kb == q) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (rev ? k < lane : k > lane) v[k] = 0.0f;
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k) r[k] = pack2(v[2 * k], v[2 * k + 1]);
                    if (kb + 1 < k1) tmem_ld(tp + kb * 32 + 32, v);
                    tc::tmem_st16(tp + kb * 16, r);
                }
                // (these columns held scores that are read by now)
#pragma unroll
                for (int k = 0; k < 16; ++k) r[k] = 0;
#pragma unroll 1
                for (int kb = rev ? 0 : q + 1; kb < (rev ? q : 4); ++kb) tc::tmem_st16(tp + kb * 16, r);
                tc::tmem_st_wait();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bPb[n % PB]);
            }
            // the four warps leave together
            if (tc::named_bar_or(1, 128, !good)) ok = false;
        }
    } else if (warp < 12) {
        // ------------------------------------------------ out
        regs_dec<kRegsOut>();
        const int q = warp & 3, i = q * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16) + Cf::cO;
        int n = 0;
        bool ok = outs;
        Walk w(digits);
        while (ok && w.next(p, digits)) {
            const LinJob& J = p.g.job[w.job];
            const int rev = J.reverse, e = rev ? 0 : 1;
            const float ld = out_decay(lin_log_decay(p.g.log_decay[w.h]));
            const int cap = power_cap(ld);
            bf16* o = static_cast<bf16*>(J.o) + (size_t)w.h * J.dc;
            bool good = true;
#pragma unroll 1
            for (int c = w.c0; c < w.c1; ++c, ++n) {
                // g to the exponent of the step's state term
                const int tau = rev ? kC - 1 - i : i - (c == 0 ? w.pad : 0);
                const float f = expf(ld * (float)min(max(tau, 0) + e, cap)) * J.oscale;
                const int t0 = chunk_time(w, c, rev), t = t0 + i;
                const bool tma = p.tma_out[w.job] && t0 >= 0;
                uint4* dst = reinterpret_cast<uint4*>(o + time_row(p, w.b, t) * J.ldo);
                // the row's place among a's: 128-byte rows of 64 columns, swizzled
                unsigned char* so = smem + (n % S) * Cf::STAGE + i * 128;
                if (!wait(bO, n)) { good = false; break; }
                tc::tc_fence_after();
                float v[32];
                tmem_ld(tl, v);
#pragma unroll 1
                for (int cb = 0; cb < J.dc; cb += 32) {
                    tc::tmem_ld_wait();
                    uint4 r[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float* x = v + k * 8;
                        r[k] = make_uint4(pack2(x[0] * f, x[1] * f), pack2(x[2] * f, x[3] * f),
                                          pack2(x[4] * f, x[5] * f), pack2(x[6] * f, x[7] * f));
                    }
                    if (cb + 32 < J.dc) {
                        tmem_ld(tl + cb + 32, v);
                    } else {   // all of out is in registers
                        tc::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(bOf);
                    }
                    if (tma) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *reinterpret_cast<uint4*>(so + (cb >> 6) * 16384 + ((((cb & 32) / 8 + k) ^ (i & 7)) << 4)) = r[k];
                    } else if (t >= 0) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (cb + k * 8 < J.dc) dst[cb / 8 + k] = r[k];
                    }
                }
                if (tma) tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bS[n % S]);
            }
            // padded steps
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const int s1 = min(p.g.T, (w.seg + 1) * p.g.seg_len);
#pragma unroll 1
            for (int t = max(w.len, w.seg * p.g.seg_len) + i; t < s1; t += 128)
#pragma unroll 1
                for (int k = 0; k < J.dc / 8; ++k)
                    *reinterpret_cast<uint4*>(o + time_row(p, w.b, t) * J.ldo + k * 8) = zero;
            if (tc::named_bar_or(4, 128, !good)) ok = false;
        }
    } else if (warp < 16) {
        // ------------------------------------------------ w c
        // A pair of steps at a time in packed bf16, without leaving it: with
        // w = w0 + w1 + w2 in three bf16 parts, a product of two of 8 bits has
        // 16, so its rounding error is a bf16 number, too:
        //   p0 = rn(c w0), p1 = c w0 - p0, p2 = rn(c w1), p3 = rn(c w1 - p2 + c w2),
        // seven instructions for the four parts of two elements.  ldmatrix
        // turns the tile's rows (steps) into pairs of steps of one column, as
        // the 16-lane store to tensor memory wants them.
        regs_dec<kRegsWeight>();
        const int q = warp & 3, l = q * 32 + lane;
        const bool second = HALF && q >= 2;         // the rows of the second parts
        const int col = (HALF ? q & 1 : q) * 32;    // first value column of the warp
        const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16) + Cf::cW;
        // this lane's row of ldmatrix: step `row` of 16, 16-byte unit `unit` of the row
        const int row = ((lane >> 4) << 3) + (lane & 7), unit = ((col & 63) >> 3) + ((lane >> 3) & 1);
        const uint32_t lm = tc::smem_u32(smem) + 2 * Cf::A_BYTES + (uint32_t)((col >> 6) * 16384 + row * 128);
        const uint32_t u0 = (uint32_t)((unit ^ (row & 7)) << 4), u1 = (uint32_t)(((unit + 2) ^ (row & 7)) << 4);
        const int skip = (int)blockIdx.x == p.skip_block ? p.skip_chunk : -1;
        int n = 0, nu = 0;   // chunk, U
        bool ok = true;
        Walk w(digits);
        while (ok && w.next(p, digits)) {
            const LinJob& J = p.g.job[w.job];
            const int rev = J.reverse, e = rev ? 0 : 1;
            const float ld = lin_log_decay(p.g.log_decay[w.h]);
            // w_j of whole chunks and of the reverse's partial one (the
            // forward's partial chunk has zeros where it has no steps)
            tc::named_bar_sync(2, 128);   // the last item's are read
            {
                const int k = l >> 6, j = (l & 63) * 2;   // variant, pair
                // a thread of the loop below reads every fourth pair of 16: side by side
                const int place = (j >> 5) * 16 + ((j >> 1) & 3) * 4 + ((j >> 3) & 3);
                float f[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int x = rev ? (k ? kC - w.pad : kC) - (kC - 1 - j - u) : kC - e - j - u;
                    f[u] = x >= 0 ? expf(ld * (float)x) * J.bscale : 0.0f;
                }
#pragma unroll
                for (int u = 0; u < 3; ++u) {
                    const uint32_t h = pack2(f[0], f[1]);
                    sw[(k * 3 + u) * (kC / 2) + place] = h;
                    f[0] -= lo_half(h);
                    f[1] -= hi_half(h);
                }
            }
            tc::named_bar_sync(2, 128);
            bool good = true;
            const int c1 = ENDS || p.g.job[w.job].fin != nullptr ? w.c1 : w.c1 - 1;   // (an item of no chunks walks none)
            for (int c = w.c0; c < c1 && good; ++c, ++n, ++nu) {
                const uint32_t* wj = sw + (rev && c == w.nct - 1 ? 3 * kC / 2 : 0) + (lane & 3) * 4;
                const int s = n % S;
                if (!wait(&full[s], n / S)) { good = false; break; }
#pragma unroll 1
                for (int b = 0; b < kC / kSub; ++b) {
                    const int set = b % SETS, turn = nu * (kC / kSub / SETS) + b / SETS;
                    const uint32_t src = lm + (uint32_t)(s * Cf::STAGE + b * kSub * 128);
                    // [lane half][8 registers: columns of 8 steps, rows 0-7 and 8-15 of the half]
                    uint32_t x[2][8];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        ldmatrix_t(src + t * 2048 + u0, &x[0][4 * t]);
                        ldmatrix_t(src + t * 2048 + u1, &x[1][4 * t]);
                    }
                    uint32_t w0[4], w1[4], w2[4];
                    lds4(wj + b * 16, w0);
                    lds4(wj + kC / 2 + b * 16, w1);
                    lds4(wj + kC + b * 16, w2);
                    // bf16 pairs: columns of 4 pairs k, rows 0-7 and 8-15 of lane half h
                    auto part = [&](int which, int h, uint32_t (&r)[8]) {
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const __nv_bfloat162 c2 = as_bf2(x[h][u]);
                            const __nv_bfloat162 v = as_bf2(which < 2 ? w0[u / 2] : w1[u / 2]);
                            __nv_bfloat162 y = __hmul2_rn(c2, v);
                            if (which & 1) {
                                y = __hfma2(c2, v, __hneg2(y));
                                if (which == 3) y = __hfma2(c2, as_bf2(w2[u / 2]), y);
                            }
                            r[u] = as_u32(y);
                        }
                    };
                    if (turn > 0 && !wait(&bWf[set], turn - 1)) { good = false; break; }
                    tc::tc_fence_after();
                    const uint32_t d = tl + set * Cf::PARTS * (kSub / 2);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t dh = d + ((uint32_t)(h * 16) << 16);
                        uint32_t r[8];
                        if constexpr (HALF) {
                            if (second) {
                                part(1, h, r);
                                tmem_st_rows(dh, r);
                                part(3, h, r);
                                tmem_st_rows(dh + 16, r);
                            } else {
                                part(0, h, r);
                                tmem_st_rows(dh, r);
                                part(2, h, r);
                                tmem_st_rows(dh + 16, r);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                part(i, h, r);
                                tmem_st_rows(dh + i * 16, r);
                            }
                        }
                    }
                    tc::tmem_st_wait();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0 && n != skip) tc::mbar_arrive(&bW[set]);
                }
            }
            if (!ENDS && w.c0 < w.c1 && c1 < w.c1) {
                // (a wait that skipped a phase would take an older one for its own)
                good = good && wait(&full[n % S], n / S);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bK[n % S]);
                ++n;
            }
            if (tc::named_bar_or(2, 128, !good)) ok = false;
        }
    } else {
        // ------------------------------------------------ X
        regs_inc<kRegsCarry>();
        const int q = warp & 3, l = q * 32 + lane;
        const int r = HALF ? (l & 63) : l;          // value column
        const bool second = HALF && l >= 64;        // the second parts' sums
        const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16) + Cf::cU;
        int n = 0, nu = 0;   // chunk, U
        bool ok = true;
        Walk w(digits);
        while (ok && w.next(p, digits)) {
            const LinJob& J = p.g.job[w.job];
            const float ld = lin_log_decay(p.g.log_decay[w.h]);
            const float* init;
            float* fin;
            bool init_t;
            state_of(p, w, init, init_t, fin);
            float X[DA];
            if (init && !second && r < J.dc) {
#pragma unroll
                for (int kb = 0; kb < DA; kb += 16) {
                    if (kb < J.da) {
                        if (init_t) {
                            const float4* x0 = reinterpret_cast<const float4*>(init + (size_t)r * J.da + kb);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float4 v = x0[k];
                                X[kb + 4 * k] = v.x; X[kb + 4 * k + 1] = v.y;
                                X[kb + 4 * k + 2] = v.z; X[kb + 4 * k + 3] = v.w;
                            }
                        } else {
                            const float* x0 = init + (size_t)kb * J.dc + r;
#pragma unroll
                            for (int k = 0; k < 16; ++k) X[kb + k] = x0[(size_t)k * J.dc];
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k) X[kb + k] = 0.0f;
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < DA; ++k) X[k] = 0.0f;
            }
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
            const int c1 = ENDS || p.g.job[w.job].fin != nullptr ? w.c1 : w.c1 - 1;
            for (int c = w.c0; c < c1 && good; ++c) {
                const int m = c == (J.reverse ? w.nct - 1 : 0) ? kC - w.pad : kC;
                const float gm = expf(ld * (float)m);
                if (!wait(bU, nu)) { good = false; break; }
                tc::tc_fence_after();
#pragma unroll
                for (int kb = 0; kb < DA; kb += 32) {
                    if (kb >= J.da) break;
                    float v[32];
                    tmem_ld(tl + kb, v);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 32; ++k) X[kb + k] = fmaf(gm, X[kb + k], v[k]);
                }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bUf);
                ++n;
                ++nu;
                if (outs && c + 1 < w.c1) good = put_x();   // the next chunk's
            }
            if (!ENDS && w.c0 < w.c1 && c1 < w.c1) ++n;
            if (fin) {
                if constexpr (HALF) {
                    // the two sums are added in the place of X's copies, once
                    // the last products that read those have ended
                    float* x = reinterpret_cast<float*>(sX);
                    if (outs)
                        for (int k = 1; k <= XB; ++k)
                            if (n - k >= 0 && good) good = wait(&bM2[(n - k) % XB], (n - k) / XB);
                    if (second) {
#pragma unroll
                        for (int k = 0; k < DA; ++k) x[k * 64 + r] = X[k];
                    }
                    tc::named_bar_sync(3, 128);
                    if (!second) {
#pragma unroll
                        for (int k = 0; k < DA; ++k) X[k] += x[k * 64 + r];
                    }
                    tc::named_bar_sync(3, 128);
                }
                if (!second && r < J.dc) {
                    float* f = fin + r;
#pragma unroll
                    for (int kb = 0; kb < DA; kb += 16)
                        if (kb < J.da) {
#pragma unroll
                            for (int k = 0; k < 16; ++k) f[(size_t)(kb + k) * J.dc] = X[kb + k];
                        }
                }
            }
            if (tc::named_bar_or(3, 128, !good)) ok = false;
        }
    }
    if (warp != 0 && lane == 0) atomicAdd(const_cast<int*>(ended), 1);
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

template <bool HALF, int DA, bool ENDS>
cudaError_t launch(const Maps& maps, const Params& p, cudaStream_t s) {
    using Cf = Cfg<HALF, DA>;
    cudaError_t e = cudaFuncSetAttribute(lin_tc_kernel<HALF, DA, ENDS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Cf::SMEM);
    if (e != cudaSuccess) return e;
    lin_tc_kernel<HALF, DA, ENDS><<<std::min(p.items, p.g.num_sms), kThreadsTc, Cf::SMEM, s>>>(maps, p);
    return cudaGetLastError();
}

template <bool HALF, int DA>
cudaError_t run(const Maps& maps, const Params& p, cudaStream_t s) {
    return p.mode != kLinWhole ? launch<HALF, DA, true>(maps, p, s) : launch<HALF, DA, false>(maps, p, s);
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
                // out's tile takes a's place: no wider than a, in whole boxes of
                // 64 columns (a box over the head's end would write the next)
                p.tma_out[k] = J.dc % 64 == 0 && J.dc <= da && a.T >= kC;
                if (!make_map(&maps.o[k], a, J.o, J.ldo, (long long)a.H * J.dc)) return cudaErrorInvalidValue;
            }
            if (p.g.njobs == 0) continue;
            // the products of one launch are neighbours in `a`, and so are their states in the buffer
            p.g.buf = a.buf + (size_t)first * a.B * a.H * a.nseg * a.job[0].da * a.job[0].dc;
            p.items = a.B * a.H * p.g.njobs * a.nseg;
            p.nmaps = nmaps;
            p.mode = mode;
            p.reset = *n == 0;
            p.status = a.status;
            p.timeout_ns = a.timeout_ns;
            p.skip_block = a.skip_block;
            p.skip_chunk = a.skip_chunk;
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
