// deltanet_step: the delta-rule recurrences for a few tokens per request on a cache of
// states, updated in place.
//
// Column b of k S, u, S and o depends only on column b of S, so a CTA takes 32 columns
// of one (request, head) and keeps its DK x 32 block of S in registers for all tokens:
// one read and one write of the state, which is nearly all the bytes there are.  B200: 256
// requests of 16 heads of 128 x 128 take 87 us, 95 % of the measured copy rate; one request
// alone 2.5 us, the latency of its chain of loads.  Four tokens of 33 requests (8 heads, 64 x
// 128, fp32) take 8.7 us, 33 %: the tokens' sums and barriers one after another.
#pragma once

#include "dn_common.cuh"
#include "dn_vec.cuh"

namespace dn {

constexpr int kErrSlots = 8;          // matches DN_ERR_SLOTS
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

// GATE: 0 none, 1 one log decay per token and head, 2 one per key channel.  DK threads: lane
// l & 7 of a warp has columns 4 (l & 7) .. + 3, the rows go round the DK / 8 groups of 8 lanes.
// ONE: a single token with a single write, the rule when decoding: no loop, and registers for
// seven CTAs of 128 threads on an SM instead of four (256 requests of 16 heads: 87 us, not 108).
template <typename E, int DK, int DV, int GATE, bool ONE>
__global__ void __launch_bounds__(DK, ONE ? 7 * 128 / DK : 1) k_step(StepParams p) {
    const int T = ONE ? 1 : p.T, nh = ONE ? 1 : p.nh;
    constexpr int RPT = 8, GROUPS = DK / 8, WARPS = DK / 32;
    __shared__ float sk[2][DK], sq[2][DK], sa[2][DK];
    __shared__ __align__(16) float red[2][WARPS][kStepCols];
    __shared__ float redqk[WARPS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cb = blockIdx.x % (DV / kStepCols);
    const int nh_i = blockIdx.x / (DV / kStepCols);
    const int h = nh_i % p.H, n = nh_i / p.H;
    const int r0 = tid >> 3;                        // rows r0 + i * GROUPS
    const int c0 = cb * kStepCols + (lane & 7) * 4;

    E* o = static_cast<E*>(p.o) + n * p.o_sn + h * p.o_sh + c0;
    const int64_t slot = step_slot(p.slots, p.M, n, p.err);
    if (slot < 0) {
        if (tid < 8)
            for (int t = 0; t < T; ++t, o += p.o_st) st_elem4(o, make_float4(0.f, 0.f, 0.f, 0.f));
        return;
    }
    float* sp = p.state + slot * p.s_sm + h * p.s_sh + (int64_t)r0 * DV + c0;
    float S[RPT][4];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(sp + i * GROUPS * DV);
        S[i][0] = x.x; S[i][1] = x.y; S[i][2] = x.z; S[i][3] = x.w;
    }
    const E* q = static_cast<const E*>(p.q) + n * p.q_sn + h * p.q_sh + tid;
    const E* k = static_cast<const E*>(p.k) + n * p.k_sn + h * p.k_sh + tid;
    const E* v = static_cast<const E*>(p.v) + n * p.v_sn + h * p.v_sh + c0;
    const float* beta = p.beta + n * p.b_sn + h * p.b_sh;
    const float* g = GATE ? p.g + n * p.g_sn + h * p.g_sh + (GATE == 2 ? tid : 0) : nullptr;

    // The next write's rows are on their way while one is worked on.
    float kn, qn = 0.f, gn = 0.f, bn;
    float4 vn;
    auto fetch = [&](bool first, bool last) {
        kn = ld_elem(k);
        vn = ld_elem4(v);
        bn = *beta;
        k += p.k_st;
        v += p.v_st;
        beta += p.b_st;
        if (last) {
            qn = ld_elem(q);
            q += p.q_st;
        }
        if (GATE && first) {
            gn = *g;
            g += p.g_st;
        }
    };
    int b = 0;
    fetch(true, nh == 1);
    for (int t = 0; t < T; ++t, o += p.o_st) {
        for (int j = 0; j < nh; ++j, b ^= 1) {
            const bool first = j == 0, last = j == nh - 1;
            sk[b][tid] = kn;
            if (last) sq[b][tid] = qn;
            if (GATE == 2 && first) sa[b][tid] = expf(gn);
            const float4 v4 = vn;
            const float bt = bn;
            const float a = GATE == 1 && first ? expf(gn) : 1.f;
            if (!last) fetch(false, j + 1 == nh - 1);
            else if (t + 1 < T) fetch(true, nh == 1);
            __syncthreads();
            // o = q (S + k^T u) = q S + (q k^T) u: q S in the same pass as k S
            float kS[4] = {}, qS[4] = {}, qk = 0.f;
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int r = r0 + i * GROUPS;
                if (GATE && first) {
                    const float ar = GATE == 2 ? sa[b][r] : a, aa[2] = {ar, ar};
                    mul2(S[i], aa, S[i]);
                    mul2(S[i] + 2, aa, S[i] + 2);
                }
                const float kr = sk[b][r], kk[2] = {kr, kr};
                fma2(kk, S[i], kS, kS);
                fma2(kk, S[i] + 2, kS + 2, kS + 2);
                if (last) {
                    const float qr = sq[b][r], qq[2] = {qr, qr};
                    fma2(qq, S[i], qS, qS);
                    fma2(qq, S[i] + 2, qS + 2, qS + 2);
                    qk = fmaf(qr, kr, qk);
                }
            }
#pragma unroll
            for (int x = 8; x < 32; x <<= 1) {
#pragma unroll
                for (int c = 0; c < 4; ++c) kS[c] += __shfl_xor_sync(~0u, kS[c], x);
                if (last) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) qS[c] += __shfl_xor_sync(~0u, qS[c], x);
                    qk += __shfl_xor_sync(~0u, qk, x);
                }
            }
            if (lane < 8) {
                *reinterpret_cast<float4*>(&red[0][warp][lane * 4]) = make_float4(kS[0], kS[1], kS[2], kS[3]);
                if (last) {
                    *reinterpret_cast<float4*>(&red[1][warp][lane * 4]) = make_float4(qS[0], qS[1], qS[2], qS[3]);
                    if (lane == 0) redqk[warp] = qk;
                }
            }
            __syncthreads();
            float u[4] = {};
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float4 x = *reinterpret_cast<const float4*>(&red[0][w][(lane & 7) * 4]);
                u[0] += x.x; u[1] += x.y; u[2] += x.z; u[3] += x.w;
            }
            u[0] = bt * (v4.x - u[0]);
            u[1] = bt * (v4.y - u[1]);
            u[2] = bt * (v4.z - u[2]);
            u[3] = bt * (v4.w - u[3]);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float kr = sk[b][r0 + i * GROUPS], kk[2] = {kr, kr};
                fma2(kk, u, S[i], S[i]);
                fma2(kk, u + 2, S[i] + 2, S[i] + 2);
            }
            if (last && tid < 8) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    const float4 y = *reinterpret_cast<const float4*>(&red[1][w][tid * 4]);
                    x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
                    s += redqk[w];
                }
                st_elem4(o, make_float4(fmaf(s, u[0], x.x), fmaf(s, u[1], x.y), fmaf(s, u[2], x.z), fmaf(s, u[3], x.w)));
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i)
        *reinterpret_cast<float4*>(sp + i * GROUPS * DV) = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
}

}  // namespace dn
