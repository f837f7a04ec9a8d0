// deltanet_scan_fwd / _bwd / _step: the gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t,
// channel by channel, and its gradients.
#pragma once

#include "dn_common.cuh"
#include "dn_step.cuh"
#include "dn_vec.cuh"

namespace dn {

constexpr int kScanThreads = 256;

struct ScanParams {
    const void *x, *g;           // forward: x, g; backward: d_out, g
    const void* h;               // backward: the forward output
    void *y, *dg;                // forward: out; backward: d_x, d_g
    const float *s0, *sT;        // forward: initial state; backward: initial state, d_final_state
    float* fin;                  // forward: final state; backward: d_initial_state
    const int* cu;               // packed: [N + 1]; null: one sequence per row
    int* err;
    int64_t x_sb, x_st, g_sb, g_st, h_sb, h_st, y_sb, y_st, dg_sb, dg_st;
    int64_t s0_sn, sT_sn, fin_sn;
    int B, T, D, N;
};

// Packed input: every CTA clamps its token range, the first reports boundaries that are not
// 0 = cu[0] <= cu[1] <= .. <= cu[N] = T.
__device__ __forceinline__ void scan_check_cu(const ScanParams& p) {
    if (!p.cu || blockIdx.x != 0) return;
    bool bad = false;
    for (int n = threadIdx.x; n <= p.N; n += blockDim.x) {
        const int c = p.cu[n];
        bad |= n == 0 ? c != 0 : c < p.cu[n - 1];
        if (n == p.N) bad |= c != p.T;
    }
    if (bad) *p.err = kErrSeqlens;
}

// A token range of one sequence for serial kernels.
__device__ __forceinline__ void scan_range(const ScanParams& p, int n, int& b, int& t0, int& t1) {
    b = p.cu ? 0 : n;
    t0 = p.cu ? min(max(p.cu[n], 0), p.T) : 0;
    t1 = p.cu ? min(max(p.cu[n + 1], t0), p.T) : p.T;
}

// One thread per (sequence, channel), token after token.
template <typename X, typename G>
__global__ void __launch_bounds__(kScanThreads) k_scan_serial(ScanParams p) {
    scan_check_cu(p);
    const int per = (p.D + kScanThreads - 1) / kScanThreads;
    const int n = blockIdx.x / per, c = (blockIdx.x % per) * kScanThreads + threadIdx.x;
    if (c >= p.D) return;
    int b, t0, t1;
    scan_range(p, n, b, t0, t1);
    const X* x = static_cast<const X*>(p.x) + b * p.x_sb + c;
    const G* g = static_cast<const G*>(p.g) + b * p.g_sb + c;
    X* y = static_cast<X*>(p.y) + b * p.y_sb + c;
    float h = p.s0 ? p.s0[n * p.s0_sn + c] : 0.f;
    for (int t = t0; t < t1; ++t) {
        h = fmaf(expf(ld_elem(g + t * p.g_st)), h, ld_elem(x + t * p.x_st));
        st_elem(y + t * p.y_st, h);
    }
    if (p.fin) p.fin[n * p.fin_sn + c] = h;
}

template <typename X, typename G>
__global__ void __launch_bounds__(kScanThreads) k_scan_bwd_serial(ScanParams p) {
    scan_check_cu(p);
    const int per = (p.D + kScanThreads - 1) / kScanThreads;
    const int n = blockIdx.x / per, c = (blockIdx.x % per) * kScanThreads + threadIdx.x;
    if (c >= p.D) return;
    int b, t0, t1;
    scan_range(p, n, b, t0, t1);
    const X* dh = static_cast<const X*>(p.x) + b * p.x_sb + c;
    const X* h = static_cast<const X*>(p.h) + b * p.h_sb + c;
    const G* g = static_cast<const G*>(p.g) + b * p.g_sb + c;
    X* dx = static_cast<X*>(p.y) + b * p.y_sb + c;
    G* dg = static_cast<G*>(p.dg) + b * p.dg_sb + c;
    float carry = p.sT ? p.sT[n * p.sT_sn + c] : 0.f;
    for (int t = t1 - 1; t >= t0; --t) {
        const float a = expf(ld_elem(g + t * p.g_st));
        const float before = t > t0 ? ld_elem(h + (t - 1) * p.h_st) : p.s0 ? p.s0[n * p.s0_sn + c] : 0.f;
        const float d = ld_elem(dh + t * p.x_st) + carry;
        carry = a * d;
        st_elem(dx + t * p.y_st, d);
        st_elem(dg + t * p.dg_st, carry * before);
    }
    if (p.fin) p.fin[n * p.fin_sn + c] = carry;
}

struct ScanStepParams {
    const void *x, *g;
    void* y;
    float* state;
    const int* slots;
    int* err;
    int64_t x_sn, x_st, g_sn, g_st, y_sn, y_st, s_sm, M;
    int N, T, D;
};

// One thread per (request, channel).
template <typename X, typename G>
__global__ void __launch_bounds__(kScanThreads) k_scan_step(ScanStepParams p) {
    const int per = (p.D + kScanThreads - 1) / kScanThreads;
    const int n = blockIdx.x / per, c = (blockIdx.x % per) * kScanThreads + threadIdx.x;
    const int64_t slot = step_slot(p.slots, p.M, n, p.err);
    if (c >= p.D) return;
    X* y = static_cast<X*>(p.y) + n * p.y_sn + c;
    if (slot < 0) {
        for (int t = 0; t < p.T; ++t) st_elem(y + t * p.y_st, 0.f);
        return;
    }
    const X* x = static_cast<const X*>(p.x) + n * p.x_sn + c;
    const G* g = static_cast<const G*>(p.g) + n * p.g_sn + c;
    float h = p.state[slot * p.s_sm + c];
    for (int t = 0; t < p.T; ++t) {
        h = fmaf(expf(ld_elem(g + t * p.g_st)), h, ld_elem(x + t * p.x_st));
        st_elem(y + t * p.y_st, h);
    }
    p.state[slot * p.s_sm + c] = h;
}

}  // namespace dn
