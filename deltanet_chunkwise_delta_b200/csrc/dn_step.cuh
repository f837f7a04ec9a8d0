// deltanet_step: the delta-rule recurrences for a few tokens per request on a cache of
// states, updated in place.
//
// Column b of k S, u, S and o depends only on column b of S, so a CTA takes 32 columns
// of one (request, head) and keeps its DK x 32 block of S in registers for all tokens:
// one read and one write of the state, which is nearly all the bytes there are.
#pragma once

#include "dn_common.cuh"
#include "dn_vec.cuh"

namespace dn {

constexpr int kErrSlots = 8;          // matches DN_ERR_SLOTS
constexpr int kStepThreads = 128;
constexpr int kStepCols = 32;         // state columns per CTA

struct StepParams {
    const void *q, *k, *v;
    void* o;
    const float *beta, *g;
    float* state;
    const int* slots;                 // null: request n uses state row n
    int* err;
    int N, T, H, nh;
    int64_t M;
    int64_t q_sn, q_st, q_sh, k_sn, k_st, k_sh, v_sn, v_st, v_sh, o_sn, o_st, o_sh;
    int64_t b_sn, b_st, b_sh, g_sn, g_st, g_sh, s_sm, s_sh;
};

// The state row of request n for all threads of the CTA, or -1 where nothing may be
// touched: a padding request, an index out of range, or one that an earlier request of
// the call names (found by looking at the n indices before it; they stay in L1).
__device__ __forceinline__ int64_t step_slot(const int* slots, int64_t M, int n, int* err) {
    if (!slots) return n;
    const int slot = slots[n];
    bool twice = false;
    if (slot >= 0)
        for (int j = threadIdx.x; j < n; j += blockDim.x) twice |= slots[j] == slot;
    const bool bad = __syncthreads_or(twice) || slot >= M || slot < -1;
    if (bad && threadIdx.x == 0) *err = kErrSlots;
    return bad || slot < 0 ? -1 : slot;
}

// GATE: 0 none, 1 one log decay per token and head, 2 one per key channel.
template <typename E, int DK, int DV, int GATE>
__global__ void __launch_bounds__(kStepThreads) k_step(StepParams p) {
    constexpr int RPT = DK / 16;      // rows of S per thread: rows i * 16 + warp * 4 + lane / 8
    __shared__ float sk[2][DK], sq[2][DK], sa[2][DK];
    __shared__ __align__(16) float red[2][4][kStepCols];
    __shared__ float redqk[4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cb = blockIdx.x % (DV / kStepCols);
    const int nh_i = blockIdx.x / (DV / kStepCols);
    const int h = nh_i % p.H, n = nh_i / p.H;
    const int r0 = warp * 4 + (lane >> 3);
    const int c0 = cb * kStepCols + (lane & 7) * 4;

    E* o = static_cast<E*>(p.o) + n * p.o_sn + h * p.o_sh;
    const int64_t slot = step_slot(p.slots, p.M, n, p.err);
    if (slot < 0) {
        if (tid < 8)
            for (int t = 0; t < p.T; ++t)
                st_elem4(o + t * p.o_st + cb * kStepCols + tid * 4, make_float4(0.f, 0.f, 0.f, 0.f));
        return;
    }
    float* sp = p.state + slot * p.s_sm + h * p.s_sh + (int64_t)r0 * DV + c0;
    float4 S[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) S[i] = *reinterpret_cast<const float4*>(sp + (int64_t)i * 16 * DV);

    const E* q = static_cast<const E*>(p.q) + n * p.q_sn + h * p.q_sh;
    const E* k = static_cast<const E*>(p.k) + n * p.k_sn + h * p.k_sh;
    const E* v = static_cast<const E*>(p.v) + n * p.v_sn + h * p.v_sh + c0;
    const float* beta = p.beta + n * p.b_sn + h * p.b_sh;
    const float* g = GATE ? p.g + n * p.g_sn + h * p.g_sh : nullptr;

    int m = 0;
    for (int t = 0; t < p.T; ++t) {
        for (int j = 0; j < p.nh; ++j, ++m) {
            const bool first = j == 0, last = j == p.nh - 1;
            const int b = m & 1;
            if (tid < DK) {
                sk[b][tid] = ld_elem(k + m * p.k_st + tid);
                if (last) sq[b][tid] = ld_elem(q + t * p.q_st + tid);
                if (GATE == 2 && first) sa[b][tid] = expf(g[t * p.g_st + tid]);
            }
            const float4 v4 = ld_elem4(v + m * p.v_st);
            const float bt = beta[m * p.b_st];
            const float a = GATE == 1 && first ? expf(g[t * p.g_st]) : 1.f;
            __syncthreads();
            float4 kS = make_float4(0.f, 0.f, 0.f, 0.f), qS = kS;
            float qk = 0.f;
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int r = r0 + i * 16;
                if (GATE && first) {
                    const float ar = GATE == 2 ? sa[b][r] : a;
                    S[i].x *= ar; S[i].y *= ar; S[i].z *= ar; S[i].w *= ar;
                }
                const float kr = sk[b][r];
                kS.x = fmaf(kr, S[i].x, kS.x); kS.y = fmaf(kr, S[i].y, kS.y);
                kS.z = fmaf(kr, S[i].z, kS.z); kS.w = fmaf(kr, S[i].w, kS.w);
                if (last) {
                    // o = q (S + k^T u) = q S + (q k^T) u: both sums in one pass
                    const float qr = sq[b][r];
                    qS.x = fmaf(qr, S[i].x, qS.x); qS.y = fmaf(qr, S[i].y, qS.y);
                    qS.z = fmaf(qr, S[i].z, qS.z); qS.w = fmaf(qr, S[i].w, qS.w);
                    qk = fmaf(qr, kr, qk);
                }
            }
#pragma unroll
            for (int x = 8; x < 32; x <<= 1) {
                kS.x += __shfl_xor_sync(~0u, kS.x, x); kS.y += __shfl_xor_sync(~0u, kS.y, x);
                kS.z += __shfl_xor_sync(~0u, kS.z, x); kS.w += __shfl_xor_sync(~0u, kS.w, x);
                if (last) {
                    qS.x += __shfl_xor_sync(~0u, qS.x, x); qS.y += __shfl_xor_sync(~0u, qS.y, x);
                    qS.z += __shfl_xor_sync(~0u, qS.z, x); qS.w += __shfl_xor_sync(~0u, qS.w, x);
                    qk += __shfl_xor_sync(~0u, qk, x);
                }
            }
            if (lane < 8) {
                *reinterpret_cast<float4*>(&red[0][warp][lane * 4]) = kS;
                if (last) *reinterpret_cast<float4*>(&red[1][warp][lane * 4]) = qS;
                if (last && lane == 0) redqk[warp] = qk;
            }
            __syncthreads();
            float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float4 x = *reinterpret_cast<const float4*>(&red[0][w][(lane & 7) * 4]);
                u.x += x.x; u.y += x.y; u.z += x.z; u.w += x.w;
            }
            u = make_float4(bt * (v4.x - u.x), bt * (v4.y - u.y), bt * (v4.z - u.z), bt * (v4.w - u.w));
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float kr = sk[b][r0 + i * 16];
                S[i].x = fmaf(kr, u.x, S[i].x); S[i].y = fmaf(kr, u.y, S[i].y);
                S[i].z = fmaf(kr, u.z, S[i].z); S[i].w = fmaf(kr, u.w, S[i].w);
            }
            if (last && tid < 8) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float4 y = *reinterpret_cast<const float4*>(&red[1][w][tid * 4]);
                    x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
                    s += redqk[w];
                }
                st_elem4(o + t * p.o_st + c0, make_float4(fmaf(s, u.x, x.x), fmaf(s, u.y, x.y),
                                                          fmaf(s, u.z, x.z), fmaf(s, u.w, x.w)));
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) *reinterpret_cast<float4*>(sp + (int64_t)i * 16 * DV) = S[i];
}

}  // namespace dn
