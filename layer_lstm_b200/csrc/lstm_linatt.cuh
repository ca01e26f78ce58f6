// What the linear-attention kernels share: which part of which product a
// block computes, and where its rows lie.
#pragma once

#include "lstm_ops.h"

namespace lstm {

enum LinMode {
    kLinWhole = 0,      // one segment: from the caller's state to the caller's state
    kLinStates = 1,     // a segment's own state, from zero, into the buffer; no outputs
    kLinSegments = 2    // a segment's outputs, from its state in the buffer
};

// Decays above 1 act as 1; 1e-4343 forgets at once (and 0 * -inf never forms).
__device__ __forceinline__ float lin_log_decay(float x) { return x > 0.0f ? 0.0f : (x < -1e4f ? -1e4f : x); }

__device__ __forceinline__ int lin_length(const LinArgs& g, int b) {
    return g.lengths ? min(g.T, max(0, g.lengths[b])) : g.T;
}

// Valid steps of segment `seg` of a row of `len`.  The tensor-core kernel's
// chunks end where the row ends, so forwards its first chunk is the short one.
__device__ __forceinline__ int lin_steps(const LinArgs& g, int len, int seg, int reverse) {
    const int pad = g.from_end && !reverse ? (kLinTcChunk - len % kLinTcChunk) % kLinTcChunk : 0;
    const int t0 = max(0, seg * g.seg_len - pad), t1 = (seg + 1) * g.seg_len - pad;
    return max(0, min(t1, len) - t0);
}

// Where the steps of one batch row lie: step tau of the product's own order
// is time row `at(tau)` of the arrays.
struct LinRow {
    long long base, step;   // array row of time 0, rows between two times
    int first, sign;        // time of tau = 0, and its direction
    __device__ __forceinline__ long long at(int tau) const { return base + (long long)(first + sign * tau) * step; }
    __device__ __forceinline__ long long padded(int t) const { return base + (long long)t * step; }
};

// What one block does.
struct LinItem {
    int job, h;
    LinRow row;
    int tau0, tau1;         // its valid steps
    int pad0, pad1;         // its padded times
    int e;                  // 1 forwards, 0 backwards (lstm_ops.h)
    float ld;
    const float* init;
    int init_t;
    float* fin;
};

// Offset of a product's segment states in the buffer.
__device__ __forceinline__ size_t lin_buf_offset(const LinArgs& g, int job) {
    return (size_t)job * g.B * g.H * g.nseg * g.job[0].da * g.job[0].dc;
}

__device__ __forceinline__ void lin_item(const LinArgs& g, int mode, unsigned block, LinItem& it) {
    const unsigned heads = (unsigned)(g.B * g.H);
    const int seg = (int)(block % (unsigned)g.nseg);
    const unsigned rest = block / (unsigned)g.nseg;
    const unsigned bh = rest % heads;
    it.job = (int)(rest / heads);
    const LinJob& J = g.job[it.job];
    const int b = (int)(bh / (unsigned)g.H);
    it.h = (int)(bh % (unsigned)g.H);
    const int len = lin_length(g, b);
    it.row.base = g.batch_first ? (long long)b * g.T : b;
    it.row.step = g.batch_first ? 1 : g.B;
    it.row.first = J.reverse ? len - 1 : 0;
    it.row.sign = J.reverse ? -1 : 1;
    const int s0 = seg * g.seg_len, s1 = min(g.T, s0 + g.seg_len);
    it.tau0 = min(s0, len);
    it.tau1 = min(s1, len);
    it.pad0 = max(s0, len);
    it.pad1 = max(s1, it.pad0);
    it.e = J.reverse ? 0 : 1;
    it.ld = lin_log_decay(g.log_decay[it.h]);
    const size_t n = (size_t)J.da * J.dc;
    float* own = g.buf + lin_buf_offset(g, it.job) + ((size_t)bh * g.nseg + seg) * n;
    it.init = mode == kLinWhole ? (J.init ? J.init + bh * n : nullptr) : (mode == kLinStates ? nullptr : own);
    it.init_t = mode == kLinWhole ? J.init_t : 0;
    it.fin = mode == kLinWhole ? (J.fin ? J.fin + bh * n : nullptr) : (mode == kLinStates ? own : nullptr);
}

cudaError_t launch_lin_carry(const LinArgs& a, cudaStream_t s, int* n);

}  // namespace lstm
