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

// ---- runs of tokens across warps and CTAs ------------------------------------------------
//
// A cluster of K CTAs takes 32 V channels of one batch row (or of the packed tokens) and
// walks the tokens in tiles of K * 8 * TS, each warp TS tokens of a tile.  A run of tokens
// maps the h before it to A h + H; a warp forms its run's (A, H) with the tokens in
// registers, warps exchange theirs through shared memory and CTAs through distributed
// shared memory, and each then knows the h before its run and finishes its tokens.  Every
// element is read once and written once.  Backward walks the tokens from the last one, with
// c = a_t delta_t (what reaches token t - 1) in the place of h.
//
// Packed input: the run's map is cut where a sequence starts (backward: ends).  Such a run
// passes H on whatever comes in, so that nothing of another sequence, NaN included, leaks:
// A = -1 marks it (products of decays are >= 0).
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kScanMaxCluster = 16;

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores x at the address of `p` (this CTA's shared memory) in the CTA of rank r.
__device__ __forceinline__ void st_cluster(float* p, unsigned r, float x) {
    uint32_t a = (uint32_t)__cvta_generic_to_shared(p), b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(r));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(b), "f"(x) : "memory");
}

// carry <- A carry + H (H alone where A is the mark)
template <bool PACKED>
__device__ __forceinline__ float run_map(float A, float H, float carry) {
    const float x = fmaf(A, carry, H);
    return PACKED && A < 0.f ? H : x;
}
// The product of two runs' decays.  Kept below infinity, so that a growing run still maps 0 to H.
template <bool PACKED>
__device__ __forceinline__ float run_prod(float A, float B) {
    const float x = fminf(A * B, 3.402823466e38f);
    return PACKED && (A < 0.f || B < 0.f) ? -1.f : x;
}

template <int V>
struct ScanSmem {
    float warp[2][kScanWarps][2][32 * V];       // (A, H) of each warp's run, by tile parity
    float cta[2][kScanMaxCluster][2][32 * V];   // (A, H) of each CTA's run
};

// Exchanges the warps' runs (A, H) of one tile: cin becomes what comes into this warp's run,
// carry what leaves the tile.  Every thread of the cluster calls it; `before_wait` runs while
// the other CTAs' runs are on their way.
template <int V, bool PACKED, typename F>
__device__ __forceinline__ void scan_exchange(ScanSmem<V>& sm, int par, int K, unsigned rank, const float* A,
                                              const float* H, float* carry, float* cin, F before_wait) {
    const int w = threadIdx.x >> 5, l = (threadIdx.x & 31) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        sm.warp[par][w][0][l + v] = A[v];
        sm.warp[par][w][1][l + v] = H[v];
    }
    __syncthreads();
    if (K == 1) {
        before_wait();
#pragma unroll
        for (int i = 0; i < kScanWarps; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (i == w) cin[v] = carry[v];
                carry[v] = run_map<PACKED>(sm.warp[par][i][0][l + v], sm.warp[par][i][1][l + v], carry[v]);
            }
        return;
    }
    // the run of the warps before this one, and of the whole CTA (last warp), which goes to every CTA
    float PA[V], PH[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        PA[v] = 1.f;
        PH[v] = 0.f;
        for (int i = 0; i < w; ++i) {
            const float a = sm.warp[par][i][0][l + v], h = sm.warp[par][i][1][l + v];
            PH[v] = run_map<PACKED>(a, h, PH[v]);
            PA[v] = run_prod<PACKED>(a, PA[v]);
        }
        if (w == kScanWarps - 1) {
            const float a = run_prod<PACKED>(A[v], PA[v]), h = run_map<PACKED>(A[v], H[v], PH[v]);
            for (int r = 0; r < K; ++r) {
                st_cluster(&sm.cta[par][rank][0][l + v], r, a);
                st_cluster(&sm.cta[par][rank][1][l + v], r, h);
            }
        }
    }
    cluster_arrive();
    before_wait();
    cluster_wait();
    for (int r = 0; r < K; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (r == (int)rank) cin[v] = carry[v];
            carry[v] = run_map<PACKED>(sm.cta[par][r][0][l + v], sm.cta[par][r][1][l + v], carry[v]);
        }
#pragma unroll
    for (int v = 0; v < V; ++v) cin[v] = run_map<PACKED>(PA[v], PH[v], cin[v]);
}

// The last n with cu[n] <= t, in 0 .. N - 1 whatever cu holds.
__device__ __forceinline__ int scan_owner(const int* cu, int N, int t) {
    int lo = 0, hi = N;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Packed input: state rows of sequences without tokens (forward: final = initial state;
// backward: d_initial = d_final), channel tile by channel tile.
template <int V>
__device__ __forceinline__ void scan_empty(const ScanParams& p, const float* src, int64_t src_sn, int c, int K,
                                           unsigned rank) {
    if (!p.fin) return;
    for (int n = rank * kScanWarps + (threadIdx.x >> 5); n < p.N; n += K * kScanWarps)
        if (p.cu[n] >= p.cu[n + 1] && c < p.D)
#pragma unroll
            for (int v = 0; v < V; ++v) p.fin[n * p.fin_sn + c + v] = src ? src[n * src_sn + c + v] : 0.f;
}

template <typename X, typename G, int V, int TS, bool PACKED>
__global__ void __launch_bounds__(kScanThreads, 2) k_scan_tiled(ScanParams p, int K) {
    __shared__ ScanSmem<V> sm;
    const unsigned rank = K > 1 ? cluster_rank() : 0;
    const int item = blockIdx.x / K, ct = (p.D + 32 * V - 1) / (32 * V);
    const int b = item / ct, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = (item % ct) * 32 * V + lane * V;
    const bool live = c < p.D;
    const X* x = static_cast<const X*>(p.x) + b * p.x_sb + c;
    const G* g = static_cast<const G*>(p.g) + b * p.g_sb + c;
    X* y = static_cast<X*>(p.y) + b * p.y_sb + c;
    if (PACKED) {
        scan_check_cu(p);
        scan_empty<V>(p, p.s0, p.s0_sn, c, K, rank);
    }
    float carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = !PACKED && live && p.s0 ? p.s0[b * p.s0_sn + c + v] : 0.f;

    typename RawVec<X, V>::T rx[TS];
    typename RawVec<G, V>::T rg[TS];
    const int step = K * kScanWarps * TS;
    int64_t t0 = ((int64_t)rank * kScanWarps + w) * TS;      // this warp's first token of the tile
    auto load = [&](int64_t t) {
#pragma unroll
        for (int j = 0; j < TS; ++j) {
            const bool in = live && t + j < p.T;
            rx[j] = in ? ld_raw<X, V>(x + (t + j) * p.x_st) : typename RawVec<X, V>::T{};
            rg[j] = in ? ld_raw<G, V>(g + (t + j) * p.g_st) : typename RawVec<G, V>::T{};
        }
    };
    load(t0);
    if (K > 1) {
        cluster_arrive();
        cluster_wait();
    }
    int par = 0;
    for (int64_t tile = 0; tile < p.T; tile += step, t0 += step, par ^= 1) {
        unsigned starts = 0, ends = 0;
        int owner = 0;
        if (PACKED) {
            const int t = (int)(t0 + (lane < TS ? lane : 0) < p.T ? t0 + (lane < TS ? lane : 0) : p.T - 1);
            owner = scan_owner(p.cu, p.N, t);
            const bool in = lane < TS && t0 + lane < p.T;
            starts = __ballot_sync(~0u, in && p.cu[owner] == t);
            ends = __ballot_sync(~0u, in && p.cu[owner + 1] == t + 1);
        }
        float hl[TS][V], Ap[TS][V], A[V], h[V];
        bool cut = false;
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = 1.f, h[v] = 0.f;
#pragma unroll
        for (int j = 0; j < TS; ++j) {
            float xv[V], gv[V];
            unpack(rx[j], xv);
            unpack(rg[j], gv);
            if (PACKED && (starts >> j & 1)) {
                cut = true;
                const int n = __shfl_sync(~0u, owner, j);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float s = live && p.s0 ? p.s0[n * p.s0_sn + c + v] : 0.f;
                    h[v] = fmaf(expf(gv[v]), s, xv[v]);
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float a = expf(gv[v]);
                    h[v] = fmaf(a, h[v], xv[v]);
                    A[v] = run_prod<false>(a, A[v]);
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                hl[j][v] = h[v];
                Ap[j][v] = PACKED && cut ? -1.f : A[v];
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = Ap[TS - 1][v];
        float cin[V];
        scan_exchange<V, PACKED>(sm, par, K, rank, A, h, carry, cin, [&] { load(t0 + step); });
#pragma unroll
        for (int j = 0; j < TS; ++j) {
            float o[V];
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = run_map<PACKED>(Ap[j][v], hl[j][v], cin[v]);
            if (live && t0 + j < p.T) st_vec<X, V>(y + (t0 + j) * p.y_st, o);
            if (PACKED && (ends >> j & 1)) {
                const int n = __shfl_sync(~0u, owner, j);
                if (p.fin && live)
#pragma unroll
                    for (int v = 0; v < V; ++v) p.fin[n * p.fin_sn + c + v] = o[v];
            }
        }
    }
    if (!PACKED && p.fin && live && rank == 0 && w == 0)
#pragma unroll
        for (int v = 0; v < V; ++v) p.fin[b * p.fin_sn + c + v] = carry[v];
}

template <typename X, typename G, int V, int TS, bool PACKED>
__global__ void __launch_bounds__(kScanThreads, 2) k_scan_bwd_tiled(ScanParams p, int K) {
    __shared__ ScanSmem<V> sm;
    const unsigned rank = K > 1 ? cluster_rank() : 0;
    const int item = blockIdx.x / K, ct = (p.D + 32 * V - 1) / (32 * V);
    const int b = item / ct, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = (item % ct) * 32 * V + lane * V;
    const bool live = c < p.D;
    const X* dh = static_cast<const X*>(p.x) + b * p.x_sb + c;
    const X* hp = static_cast<const X*>(p.h) + b * p.h_sb + c;
    const G* g = static_cast<const G*>(p.g) + b * p.g_sb + c;
    X* dx = static_cast<X*>(p.y) + b * p.y_sb + c;
    G* dg = static_cast<G*>(p.dg) + b * p.dg_sb + c;
    if (PACKED) {
        scan_check_cu(p);
        scan_empty<V>(p, p.sT, p.sT_sn, c, K, rank);
    }
    float carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = !PACKED && live && p.sT ? p.sT[b * p.sT_sn + c + v] : 0.f;

    typename RawVec<X, V>::T rd[TS], rh[TS];
    typename RawVec<G, V>::T rg[TS];
    const int step = K * kScanWarps * TS;
    // token of this warp's place j in the tile: t0 - j
    int64_t t0 = p.T - 1 - ((int64_t)rank * kScanWarps + w) * TS;
    auto load = [&](int64_t t) {
#pragma unroll
        for (int j = 0; j < TS; ++j) {
            const bool in = live && t - j >= 0, prev = live && t - j >= 1;
            rd[j] = in ? ld_raw<X, V>(dh + (t - j) * p.x_st) : typename RawVec<X, V>::T{};
            rg[j] = in ? ld_raw<G, V>(g + (t - j) * p.g_st) : typename RawVec<G, V>::T{};
            rh[j] = prev ? ld_raw<X, V>(hp + (t - j - 1) * p.h_st) : typename RawVec<X, V>::T{};
        }
    };
    load(t0);
    if (K > 1) {
        cluster_arrive();
        cluster_wait();
    }
    int par = 0;
    for (int64_t tile = 0; tile < p.T; tile += step, t0 -= step, par ^= 1) {
        unsigned starts = 0, ends = 0;
        int owner = 0;
        if (PACKED) {
            const bool in = lane < TS && t0 - lane >= 0;
            const int t = in ? (int)(t0 - lane) : 0;
            owner = scan_owner(p.cu, p.N, t);
            starts = __ballot_sync(~0u, in && p.cu[owner] == t);
            ends = __ballot_sync(~0u, in && p.cu[owner + 1] == t + 1);
        }
        float dl[TS][V], Ae[TS][V], m[TS][V], A[V], e[V];
        bool cut = false;
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = 1.f, e[v] = 0.f;
#pragma unroll
        for (int j = 0; j < TS; ++j) {
            float dv[V], gv[V], hv[V];
            unpack(rd[j], dv);
            unpack(rg[j], gv);
            unpack(rh[j], hv);
            if (PACKED && (ends >> j & 1)) {
                cut = true;
                const int n = __shfl_sync(~0u, owner, j);
#pragma unroll
                for (int v = 0; v < V; ++v) e[v] = live && p.sT ? p.sT[n * p.sT_sn + c + v] : 0.f;
            }
            if (PACKED ? (starts >> j & 1) : t0 - j == 0) {
                const int n = PACKED ? __shfl_sync(~0u, owner, j) : b;
#pragma unroll
                for (int v = 0; v < V; ++v) hv[v] = live && p.s0 ? p.s0[n * p.s0_sn + c + v] : 0.f;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float a = expf(gv[v]);
                const float d = dv[v] + e[v];
                dl[j][v] = d;
                Ae[j][v] = PACKED && cut ? -1.f : A[v];
                m[j][v] = a * hv[v];
                e[v] = a * d;
                A[v] = run_prod<false>(a, A[v]);
            }
        }
        if (PACKED && cut)
#pragma unroll
            for (int v = 0; v < V; ++v) A[v] = -1.f;
        float cin[V];
        scan_exchange<V, PACKED>(sm, par, K, rank, A, e, carry, cin, [&] { load(t0 - step); });
#pragma unroll
        for (int j = 0; j < TS; ++j) {
            float d[V], q[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                d[v] = run_map<PACKED>(Ae[j][v], dl[j][v], cin[v]);
                q[v] = d[v] * m[j][v];
            }
            if (live && t0 - j >= 0) {
                st_vec<X, V>(dx + (t0 - j) * p.y_st, d);
                st_vec<G, V>(dg + (t0 - j) * p.dg_st, q);
            }
            if (PACKED && (starts >> j & 1)) {
                const int n = __shfl_sync(~0u, owner, j);
                if (p.fin && live)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        p.fin[n * p.fin_sn + c + v] = expf(ld_elem(g + (t0 - j) * p.g_st + v)) * d[v];
            }
        }
    }
    if (!PACKED && p.fin && live && rank == 0 && w == 0)
#pragma unroll
        for (int v = 0; v < V; ++v) p.fin[b * p.fin_sn + c + v] = carry[v];
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
