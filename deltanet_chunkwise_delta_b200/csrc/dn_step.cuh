// deltanet_step: the delta-rule recurrences for a few tokens per request on a cache of
// states, updated in place.
//
// Column b of k S, u, S and o depends only on column b of S, so a CTA takes 32 columns
// of one (request, head) and keeps its DK x 32 block of S in registers for all tokens:
// one read and one write of the state, which is nearly all the bytes there are.  B200: 256
// requests of 16 heads of 128 x 128 take 87 us, 95 % of the measured copy rate; one request
// alone 2.5 us, the latency of its chain of loads.  Each token after the first costs 0.5 us, its
// sums and barriers: four tokens of 33 requests (8 heads, 64 x 128, fp32) take 8.4 us, 35 %,
// four of 256 requests of 16 heads 148 us, 57 %.
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

// The rows of a write as they lie in memory, on their way kStepAhead - 1 writes ahead of the
// one worked on: fetched one write ahead, a write takes as long as memory does (four tokens of
// 256 requests 180 us, not 151).  A row's 16-byte pieces go one to a thread.
constexpr int kStepAhead = 8;
template <typename E, int DK, int GATE>
struct alignas(16) StepRows {
    E k[DK], q[DK], v[kStepCols];
    float g[GATE == 2 ? DK : 4], beta[4];
    static constexpr int kK = DK * sizeof(E) / 16, kV = kStepCols * sizeof(E) / 16, kG = GATE == 2 ? DK / 4 : GATE;
    static_assert(2 * kK + kV + kG + 1 <= DK, "a piece per thread");
};

enum StepKind { kStepOne, kStepTokens, kStepWrites };

// GATE: 0 none, 1 one log decay per token and head, 2 one per key channel.  DK threads: lane
// l & 7 of a warp has columns 4 (l & 7) .. + 3, each group of 8 lanes every fourth of a warp's
// 32 rows.
// kStepOne: a single token with a single write, the rule when decoding: no loop, registers for
// seven CTAs of 128 threads on an SM instead of four (256 requests of 16 heads: 87 us, not 108).
// kStepTokens: one write per token, known when compiled (four tokens of them 180 us, not 198).
template <typename E, int DK, int DV, int GATE, StepKind KIND>
__global__ void __launch_bounds__(DK, KIND == kStepOne ? 7 * 128 / DK : 1) k_step(StepParams p) {
    const int T = KIND == kStepOne ? 1 : p.T, nh = KIND == kStepWrites ? p.nh : 1;
    constexpr int RPT = 8, WARPS = DK / 32;
    __shared__ __align__(16) float sk[2][DK], sq[2][DK], sa[2][DK];
    __shared__ __align__(16) float red[2][WARPS][kStepCols];
    __shared__ float redqk[WARPS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cb = blockIdx.x % (DV / kStepCols);
    const int nh_i = blockIdx.x / (DV / kStepCols);
    const int h = nh_i % p.H, n = nh_i / p.H;
    // rows row0 + 4 i (four neighbours per access of a warp); a vector's entries for them lie
    // side by side in shared memory, from r0 on: entry e of it at `spot` of thread e
    const int row0 = warp * 32 + (lane >> 3), r0 = (tid >> 3) * RPT;
    const int spot = warp * 32 + (tid & 3) * 8 + (lane >> 2);
    const int c0 = cb * kStepCols + (lane & 7) * 4;

    E* o = static_cast<E*>(p.o) + n * p.o_sn + h * p.o_sh + c0;
    using Rows = StepRows<E, DK, GATE>;
    __shared__ Rows rows[KIND == kStepOne ? 1 : kStepAhead];
    const E* q = static_cast<const E*>(p.q) + n * p.q_sn + h * p.q_sh;
    const E* k = static_cast<const E*>(p.k) + n * p.k_sn + h * p.k_sh;
    const E* v = static_cast<const E*>(p.v) + n * p.v_sn + h * p.v_sh + cb * kStepCols;
    const float* beta = p.beta + n * p.b_sn + h * p.b_sh;
    const float* g = GATE ? p.g + n * p.g_sn + h * p.g_sh : nullptr;
    // this thread's piece: where it is, how far its next one, whether a write or a token on
    const char* src = nullptr;
    uint32_t dst = 0;
    int64_t src_step = 0;
    bool wide = true, by_token = false;
    int issued = 0, issued_j = 0;
    if (KIND != kStepOne) {
        auto piece = [&](const void* from, int64_t st, void* to) {
            src = static_cast<const char*>(from);
            src_step = st;
            dst = (uint32_t)__cvta_generic_to_shared(to);
        };
        int i = tid;
        if (i < Rows::kK) {
            piece(k + i * (16 / sizeof(E)), p.k_st * sizeof(E), rows[0].k + i * (16 / sizeof(E)));
        } else if ((i -= Rows::kK) < Rows::kK) {
            piece(q + i * (16 / sizeof(E)), p.q_st * sizeof(E), rows[0].q + i * (16 / sizeof(E)));
            by_token = true;
        } else if ((i -= Rows::kK) < Rows::kV) {
            piece(v + i * (16 / sizeof(E)), p.v_st * sizeof(E), rows[0].v + i * (16 / sizeof(E)));
        } else if ((i -= Rows::kV) < Rows::kG) {
            piece(g + i * 4, p.g_st * 4, rows[0].g + i * 4);
            by_token = true;
            wide = GATE == 2;
        } else if (i == Rows::kG) {
            piece(beta, p.b_st * 4, rows[0].beta);
            wide = false;
        }
    }
    const int writes = T * nh;
    auto issue = [&] {
        if (issued < writes && src) {
            const uint32_t to = dst + issued++ % kStepAhead * (int)sizeof(Rows);
            if (wide) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
            else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(src) : "memory");
            issued_j = issued_j == nh - 1 ? 0 : issued_j + 1;
            if (!by_token || issued_j == 0) src += src_step;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (KIND != kStepOne)
        for (int i = 0; i < kStepAhead; ++i) issue();
    const int64_t slot = step_slot(p.slots, p.M, n, p.err);
    if (slot < 0) {
        if (KIND != kStepOne) asm volatile("cp.async.wait_all;" ::: "memory");
        if (tid < 8)
            for (int t = 0; t < T; ++t, o += p.o_st) st_elem4(o, make_float4(0.f, 0.f, 0.f, 0.f));
        return;
    }
    float* sp = p.state + slot * p.s_sm + h * p.s_sh + (int64_t)row0 * DV + c0;
    float S[RPT][4];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(sp + i * 4 * DV);
        S[i][0] = x.x; S[i][1] = x.y; S[i][2] = x.z; S[i][3] = x.w;
    }
    // The next write's values: from memory, or where its rows have landed.
    float kn, qn = 0.f, gn = 0.f, bn;
    float4 vn;
    int at = 0;
    auto fetch = [&](bool first, bool last) {
        const Rows& r = rows[at];
        constexpr bool one = KIND == kStepOne;
        kn = ld_elem(one ? k + tid : r.k + tid);
        vn = ld_elem4((one ? v : r.v) + (lane & 7) * 4);
        bn = one ? *beta : r.beta[0];
        if (last) qn = ld_elem(one ? q + tid : r.q + tid);
        if (GATE && first) gn = (one ? g : r.g)[GATE == 2 ? tid : 0];
        at = at + 1 == kStepAhead ? 0 : at + 1;
    };
    if (KIND != kStepOne) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStepAhead - 1) : "memory");
        __syncthreads();
    }
    // a vector at four of this thread's rows
    auto take = [&](const float* mem, int i, float* f) {
        const float4 x = *reinterpret_cast<const float4*>(mem + r0 + i);
        f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
    };
    int b = 0;
    fetch(true, nh == 1);
    for (int t = 0; t < T; ++t, o += p.o_st) {
        for (int j = 0; j < nh; ++j, b ^= 1) {
            const bool first = j == 0, last = j == nh - 1;
            sk[b][spot] = kn;
            if (last) sq[b][spot] = qn;
            if (GATE == 2 && first) sa[b][spot] = expf(gn);
            const float4 v4 = vn;
            const float bt = bn;
            const float a = GATE == 1 && first ? expf(gn) : 1.f;
            if (KIND != kStepOne) asm volatile("cp.async.wait_group %0;" ::"n"(kStepAhead - 2) : "memory");
            __syncthreads();
            if (!last) fetch(false, j + 1 == nh - 1);
            else if (t + 1 < T) fetch(true, nh == 1);
            if (KIND != kStepOne) issue();
            // o = q (S + k^T u) = q S + (q k^T) u: q S in the same pass as k S
            float kS[4] = {}, qS[4] = {}, qk = 0.f, kv[4], qv[4], av[4];
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                if (i % 4 == 0) {
                    take(sk[b], i, kv);
                    if (last) take(sq[b], i, qv);
                    if (GATE == 2 && first) take(sa[b], i, av);
                }
                if (GATE && first) {
                    const float ar = GATE == 2 ? av[i % 4] : a, aa[2] = {ar, ar};
                    mul2(S[i], aa, S[i]);
                    mul2(S[i] + 2, aa, S[i] + 2);
                }
                const float kr = kv[i % 4], kk[2] = {kr, kr};
                fma2(kk, S[i], kS, kS);
                fma2(kk, S[i] + 2, kS + 2, kS + 2);
                if (last) {
                    const float qr = qv[i % 4], qq[2] = {qr, qr};
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
                if (i % 4 == 0) take(sk[b], i, kv);
                const float kr = kv[i % 4], kk[2] = {kr, kr};
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
        *reinterpret_cast<float4*>(sp + i * 4 * DV) = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
}

}  // namespace dn
