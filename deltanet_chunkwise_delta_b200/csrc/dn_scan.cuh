// deltanet_scan_fwd / _bwd / _step: the gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t,
// channel by channel, and its gradients.
#pragma once

#include <type_traits>

#include "dn_common.cuh"
#include "dn_sm100.cuh"
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
    int stall;                   // > 0 (a test): a cluster's first CTA sends nothing at tile stall - 1
    unsigned long long wait_ns;  // a wait inside a cluster gives up after so long
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

// e^g as a power of two: one product and the hardware's 2^x (2 ulp), (4 + 2.4 |g|) 2^-24
// relative in all, where a token's step needs no more: a decay's error enters h with weight a.
__device__ __forceinline__ void scan_log2(float* g) {
    const float c[2] = {1.44269504f, 1.44269504f};
    mul2(g, c, g);
}
__device__ __forceinline__ float scan_pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float scan_decay(float g) { return scan_pow2(g * 1.44269504f); }

// ---- short sequences: a thread walks its channels, token after token ----------------------
//
// One thread per V channels of a sequence (2 where rows are made of pairs), the next kScanAhead
// tokens of its loads in registers.  Nothing is exchanged; what bounds it is the loads in
// flight, so it takes short rows, or so many that they fill the GPU.
constexpr int kScanAhead = 8, kScanWalkers = 128;

template <typename X, typename G, int V>
__global__ void __launch_bounds__(kScanWalkers) k_scan_serial(ScanParams p) {
    scan_check_cu(p);
    const int per = (p.D + kScanWalkers * V - 1) / (kScanWalkers * V);
    const int n = blockIdx.x / per, c = ((blockIdx.x % per) * kScanWalkers + threadIdx.x) * V;
    if (c >= p.D) return;
    int b, t0, t1;
    scan_range(p, n, b, t0, t1);
    const X* x = static_cast<const X*>(p.x) + b * p.x_sb + t0 * p.x_st + c;
    const G* g = static_cast<const G*>(p.g) + b * p.g_sb + t0 * p.g_st + c;
    X* y = static_cast<X*>(p.y) + b * p.y_sb + t0 * p.y_st + c;
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = p.s0 ? p.s0[n * p.s0_sn + c + v] : 0.f;
    for (int t = t0; t < t1; t += kScanAhead) {
        typename RawVec<X, V>::T rx[kScanAhead];
        typename RawVec<G, V>::T rg[kScanAhead];
#pragma unroll
        for (int j = 0; j < kScanAhead; ++j)
            if (t + j < t1) {
                rx[j] = ld_raw<X, V>(x + j * p.x_st);
                rg[j] = ld_raw<G, V>(g + j * p.g_st);
            }
#pragma unroll
        for (int j = 0; j < kScanAhead; ++j)
            if (t + j < t1) {
                float xv[V], a[V];
                unpack(rx[j], xv);
                unpack(rg[j], a);
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = fmaf(scan_decay(a[v]), h[v], xv[v]);
                st_vec<X, V>(y + j * p.y_st, h);
            }
        x += kScanAhead * p.x_st;
        g += kScanAhead * p.g_st;
        y += kScanAhead * p.y_st;
    }
    if (p.fin)
#pragma unroll
        for (int v = 0; v < V; ++v) p.fin[n * p.fin_sn + c + v] = h[v];
}

template <typename X, typename G, int V>
__global__ void __launch_bounds__(kScanWalkers) k_scan_bwd_serial(ScanParams p) {
    scan_check_cu(p);
    const int per = (p.D + kScanWalkers * V - 1) / (kScanWalkers * V);
    const int n = blockIdx.x / per, c = ((blockIdx.x % per) * kScanWalkers + threadIdx.x) * V;
    if (c >= p.D) return;
    int b, t0, t1;
    scan_range(p, n, b, t0, t1);
    const int64_t last = t1 - 1;
    const X* dh = static_cast<const X*>(p.x) + b * p.x_sb + last * p.x_st + c;
    const X* hp = static_cast<const X*>(p.h) + b * p.h_sb + (last - 1) * p.h_st + c;
    const G* g = static_cast<const G*>(p.g) + b * p.g_sb + last * p.g_st + c;
    X* dx = static_cast<X*>(p.y) + b * p.y_sb + last * p.y_st + c;
    G* dg = static_cast<G*>(p.dg) + b * p.dg_sb + last * p.dg_st + c;
    float e[V];                            // a_{t+1} delta_{t+1}
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = p.sT ? p.sT[n * p.sT_sn + c + v] : 0.f;
    for (int t = t1 - 1; t >= t0; t -= kScanAhead) {
        typename RawVec<X, V>::T rd[kScanAhead], rh[kScanAhead];
        typename RawVec<G, V>::T rg[kScanAhead];
#pragma unroll
        for (int j = 0; j < kScanAhead; ++j)
            if (t - j >= t0) {
                rd[j] = ld_raw<X, V>(dh - j * p.x_st);
                rg[j] = ld_raw<G, V>(g - j * p.g_st);
                if (t - j > t0) rh[j] = ld_raw<X, V>(hp - j * p.h_st);
            }
#pragma unroll
        for (int j = 0; j < kScanAhead; ++j)
            if (t - j >= t0) {
                float d[V], a[V], hv[V], q[V];
                unpack(rd[j], d);
                unpack(rg[j], a);
                if (t - j > t0) {
                    unpack(rh[j], hv);
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) hv[v] = p.s0 ? p.s0[n * p.s0_sn + c + v] : 0.f;
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    d[v] += e[v];
                    e[v] = scan_decay(a[v]) * d[v];
                    q[v] = e[v] * hv[v];
                }
                st_vec<X, V>(dx - j * p.y_st, d);
                st_vec<G, V>(dg - j * p.dg_st, q);
            }
        dh -= kScanAhead * p.x_st;
        hp -= kScanAhead * p.h_st;
        g -= kScanAhead * p.g_st;
        dx -= kScanAhead * p.y_st;
        dg -= kScanAhead * p.dg_st;
    }
    if (p.fin)
#pragma unroll
        for (int v = 0; v < V; ++v) p.fin[n * p.fin_sn + c + v] = e[v];
}

// ---- runs of tokens across warps and CTAs ------------------------------------------------
//
// A cluster of K CTAs takes 64 channels of one batch row (or of the packed tokens), two per
// lane, and walks the tokens in tiles of K * W * TS, each of W warps TS tokens of a tile.  A run of
// tokens maps the h before it to A h + H; a warp forms its run's (A, H), warps and CTAs
// exchange theirs, and each then knows the h before its run and finishes its tokens.  Every
// element is read once and written once.  Backward walks the tokens from the last one, with
// c = a_t delta_t (what reaches token t - 1) in the place of h.
//
// A is formed from the sum of its logarithms (run_factor): the product of a run's decays may
// pass what fp32 holds either way where h does not.
//
// Packed input: the run's map is cut where a sequence starts (backward: ends).  Such a run
// passes H on whatever comes in, so that nothing of another sequence, NaN included, leaks:
// a logarithm of NaN marks it, which its sums with others keep (where it is the decays' own,
// H is NaN as well).
//
// The tokens come through shared memory (cp.async; a warp reads only what it copied itself).
// The warps form the (A, H) of tile i + 1 before they finish tile i; one more warp joins the
// runs, sends the CTA's to the cluster's other CTAs (st.async on their mbarriers), waits for
// theirs and hands every warp the h before its run, all of it behind the finishing of the tile
// before.  A tile is finished by running its recurrence again from the h that comes in.  Its
// tokens and decays stay in registers until then (HELD, forward: seven warps and the joining
// one, 128 registers), or are read again (eight and one, 96 registers; the decays of an fp32 gate
// have taken its place in shared memory, of a bf16 gate the power is taken twice): fewer
// instructions and longer runs against one warp more.
//
// B200: forward of 8 x 2048 x 2048 (bf16, fp32 gates) 44 us, 93 % of the measured copy rate
// (256 CTAs: 108 SMs have two of them, 40 have one); of 65536 x 2048 in fp32 280 us, 88 %;
// backward of 65536 x 2048 (bf16, fp32 gates) 338 us, 85 %.  Packed forward of 222459 x 2048 in
// bf16 545 us, 76 %; without the 32 sequences' boundaries 500: a tile with one goes the long
// way in one warp, and the cluster waits for it.

template <bool HELD>
constexpr int kScanWarps = HELD ? 7 : 8;
template <bool HELD>
constexpr int kScanThreadsOf = (kScanWarps<HELD> + 1) * 32;
constexpr int kScanMaxCluster = 8;

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
// The product A of a run's decays from its logarithm l (base 2): A where fp32 holds it with room
// (|l| <= 126), else -2^(l/3), which stands for three steps c -> 2^(l/3) c.  They go the same way,
// so nothing overflows or vanishes ahead of A c, whatever finite c makes A c finite (one factor
// would end at 2^128, far from what a tiny c may grow by).  Below 2^-252 A c is less than 2^-124:
// 0.  NaN stays NaN.
__device__ __forceinline__ float run_factor(float l) {
    const bool near = fabsf(l) <= 126.f;
    const float r = scan_pow2(near ? l : l > 381.f ? 127.f : l * 0.333333343f);
    return near ? r : l < -252.f ? 0.f : -r;
}
// carry <- A carry + H (H alone where A is the mark).  FAR: f is the run_factor of A, not A.
template <bool PACKED, bool FAR>
__device__ __forceinline__ float run_map(float f, float H, float carry) {
    float x = carry;
    if (FAR && f < 0.f) x = f * (f * x), f = -f;
    x = fmaf(f, x, H);
    return PACKED && f != f ? H : x;
}

// Packed input: state rows of sequences without tokens (forward: final = initial state;
// backward: d_initial = d_final).
template <int W>
__device__ __forceinline__ void scan_empty(const ScanParams& p, const float* src, int64_t src_sn, int c, int K,
                                           unsigned rank) {
    if (!p.fin) return;
    for (int n = rank * W + (threadIdx.x >> 5); n < p.N; n += K * W)
        if (p.cu[n] >= p.cu[n + 1])
#pragma unroll
            for (int v = 0; v < 2; ++v)
                if (c + v < p.D) p.fin[n * p.fin_sn + c + v] = src ? src[n * src_sn + c + v] : 0.f;
}

constexpr int kScanStages = 3;

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
// the first n bytes from src, zeros after
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, int n) {
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Copies the tokens of one warp's run into shared memory, tile after tile: rows j = 0 .. TS - 1
// (token t + DIR * j; zeros outside 0 .. T - 1 and past channel D) of 64 channels from c0, 64
// elements a row.  16 bytes a lane where addresses allow (wide); else, with EVEN, a lane's own
// pair, without it the elements lane and lane + 32 (of bf16 through registers: the smallest
// asynchronous copy has 4 bytes).
template <typename E, int TS, int DIR, bool EVEN>
struct ScanSrc {
    static constexpr int kPer = 64 * sizeof(E) / 16;        // lanes of a row at 16 bytes each
    const E* base;                                          // a readable address
    const E* cur;                                           // this lane's first piece of the tile
    int64_t inc, tile;                                      // to the lane's next piece, to the next tile
    int row, left;                                          // its first row; bytes of the piece that exist
    bool wide;
    __device__ __forceinline__ ScanSrc(const E* p, int64_t st, int t, int step, int c0, int D, bool wide_) : wide(wide_) {
        const int lane = threadIdx.x & 31;
        constexpr int es = sizeof(E);
        row = wide ? lane / kPer : 0;
        const int c = c0 + (wide ? lane % kPer * (16 / es) : EVEN ? lane * 2 : lane);
        const int bytes = min(D - c, 64) * es;             // (a row may have more than 2^31)
        left = max(0, wide ? min(16, bytes) : EVEN ? min(2 * es, bytes) : bytes);
        base = p;
        cur = p + c + (t + DIR * row) * st;
        inc = DIR * st * (wide ? 32 / kPer : 1);
        tile = DIR * st * step;
    }
    // t: the tile's first token; inside: every row and channel of it exists
    __device__ __forceinline__ void copy(E* dst, int t, int T, bool inside) {
        constexpr int es = sizeof(E);
        const int lane = threadIdx.x & 31;
        const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
        const E* src = cur;
        if (wide) {
            if (inside) {
#pragma unroll
                for (int i = 0; i < TS * kPer / 32; ++i, src += inc) cp_async<16>(d + i * 512 + lane * 16, src);
            } else {
#pragma unroll
                for (int i = 0; i < TS * kPer / 32; ++i, src += inc) {
                    const bool in = (unsigned)(t + DIR * (row + i * (32 / kPer))) < (unsigned)T && left > 0;
                    cp_async<16>(d + i * 512 + lane * 16, in ? src : base, in ? left : 0);
                }
            }
        } else if constexpr (EVEN) {
#pragma unroll
            for (int j = 0; j < TS; ++j, src += inc) {
                const bool in = (unsigned)(t + DIR * j) < (unsigned)T && left > 0;
                cp_async<2 * es>(d + (j * 64 + lane * 2) * es, in ? src : base, in ? left : 0);
            }
        } else if constexpr (es == 4) {
#pragma unroll
            for (int j = 0; j < TS; ++j, src += inc) {
                const bool in = (unsigned)(t + DIR * j) < (unsigned)T;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool is = in && left > h * 32 * es;
                    cp_async<4>(d + (j * 64 + h * 32 + lane) * es, is ? src + h * 32 : base, is ? 4 : 0);
                }
            }
        } else {
            E f[TS][2];
#pragma unroll
            for (int j = 0; j < TS; ++j, src += inc)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    f[j][h] = (unsigned)(t + DIR * j) < (unsigned)T && left > h * 32 * es ? src[h * 32] : E(0.f);
#pragma unroll
            for (int j = 0; j < TS; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) dst[j * 64 + h * 32 + lane] = f[j][h];
        }
        cur += tile;
    }
};

// Two channels of a lane to global memory, as a pair or (EVEN false) as far as there are two.
template <typename E, bool EVEN>
__device__ __forceinline__ void scan_store(E* q, const float* f, bool second) {
    if constexpr (EVEN) {
        st_vec<E, 2>(q, f);
    } else {
        st_elem(q, f[0]);
        if (second) st_elem(q + 1, f[1]);
    }
}

// A warp's run of tile i + 1 is written after it has read what comes into that of tile i: one
// place.  The other CTAs may be a tile ahead: theirs go by tile parity.
template <int W, bool CL>
struct ScanRuns {
    float4 warp[W][32];                   // (A0, A1, H0, H1) of each warp's run; then, in its
                                          // first half, what comes into the run
    float2 logs[W][32];                   // the logarithms of A0, A1
    uint64_t full[2];                     // the cluster's runs of a tile have arrived
    // A where it is one factor, in a cluster together with the CTA's other runs; else negative
    static __device__ __forceinline__ float factor(float l) {
        return fabsf(l) > (CL ? 126.f / 8 : 126.f) ? -1.f : scan_pow2(l);
    }
    // h and the logarithms of one warp's run; cut: it passes on h alone
    __device__ __forceinline__ void put(int w, float* l, const float* h, bool cut) {
        const int lane = threadIdx.x & 31;
        if (cut) l[0] = l[1] = __uint_as_float(0x7fffffffu);
        logs[w][lane] = make_float2(l[0], l[1]);
        warp[w][lane] = make_float4(factor(l[0]), factor(l[1]), h[0], h[1]);
    }
    // a run with factors that run_map<.., true> takes
    __device__ __forceinline__ float4 farther(int w, float4 run) const {
        const float2 l = logs[w][threadIdx.x & 31];
        return make_float4(run_factor(l.x), run_factor(l.y), run.z, run.w);
    }
};

// the signs of a run's A among others' (NaN, the mark, has none)
__device__ __forceinline__ unsigned run_signs(unsigned signs, float4 run) {
    return signs | __float_as_uint(run.x) | __float_as_uint(run.y);
}
template <bool PACKED, bool FAR>
__device__ __forceinline__ void run_through(float4 r, float& c0, float& c1) {
    c0 = run_map<PACKED, FAR>(r.x, r.z, c0);
    c1 = run_map<PACKED, FAR>(r.y, r.w, c1);
}

__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }
constexpr int kBarRuns = 1, kBarCin = 2;   // named barriers: runs of a tile formed, h before them known

// Waits for a phase that other CTAs of the cluster complete and acquires what they sent (a
// fence in its place would also wait for this warp's own sends to land: 0.6 us a tile).  Gives
// up after limit_ns.
__device__ __forceinline__ bool cluster_mbar_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
    uint64_t t0 = 0;
    for (int i = 0;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(sm100::saddr(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if (i == 255) t0 = sm100::globaltimer();
        if (i > 255 && sm100::globaltimer() - t0 > limit_ns) return false;
    }
}

// The last warp: tile after tile, the runs of this CTA joined and exchanged.  carry: what comes
// into the first tile, in the end what leaves the last one.
//
// A wait that gives up ends the CTA's part in the exchange: it arrives on no barrier whose phase
// may be open and sends nothing more, so that the others give up in turn, a tile later at most.
// Its warps get NaN for what comes into their runs from that tile on; sequences that start in
// them are right.  Returns the tile, or -1.
template <bool PACKED, bool CL, int W>
__device__ __forceinline__ int scan_join(ScanRuns<W, CL>& sm, float4* cta, int tiles, int K, unsigned rank,
                                         float* carry, const ScanParams& p) {
    const int lane = threadIdx.x & 31;
    int gave = -1;
    for (int i = 0; i < tiles; ++i) {
        const int par = i & 1;
        bar_sync(kBarRuns, (W + 1) * 32);
        float4 run[W];
        unsigned signs = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) signs = run_signs(signs, run[w] = sm.warp[w][lane]);
        const bool far = (int)signs < 0;
        if constexpr (!CL) {
            auto through = [&](auto any) {
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float4 r = decltype(any)::value ? sm.farther(w, run[w]) : run[w];
                    *reinterpret_cast<float2*>(&sm.warp[w][lane]) = make_float2(carry[0], carry[1]);
                    run_through<PACKED, decltype(any)::value>(r, carry[0], carry[1]);
                }
            };
            if (far) through(std::true_type());
            else through(std::false_type());
        } else if (gave < 0) {
            // the runs ahead of each warp's as one map.  The product of their factors where that is
            // one factor as well; else from the sum of their logarithms, which the chain over the
            // warps would wait for (in every tile: 65536 x 512 a tenth longer).
            float4 pre[W], all = make_float4(1.f, 1.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                pre[w] = all;
                all.x *= run[w].x;
                all.y *= run[w].y;
                run_through<PACKED, false>(run[w], all.z, all.w);
            }
            if (far) {
                all = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    pre[w] = make_float4(run_factor(all.x), run_factor(all.y), all.z, all.w);
                    const float4 r = sm.farther(w, sm.warp[w][lane]);
                    all.x += sm.logs[w][lane].x;
                    all.y += sm.logs[w][lane].y;
                    run_through<PACKED, true>(r, all.z, all.w);
                }
                all.x = run_factor(all.x);
                all.y = run_factor(all.y);
            }
            if (lane == 0) sm100::mbar_expect_tx(&sm.full[par], K * 512);
            const uint32_t dst = sm100::saddr(cta + (par * K + rank) * 32 + lane), bar = sm100::saddr(&sm.full[par]);
            const int to = rank == 0 && p.stall == i + 1 ? 0 : K;
            for (int r = 0; r < to; ++r) {
                uint32_t d, m;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(dst), "r"(r));
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(m) : "r"(bar), "r"(r));
                asm volatile(
                    "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(d),
                    "r"(__float_as_uint(all.x)), "r"(__float_as_uint(all.y)), "r"(__float_as_uint(all.z)),
                    "r"(__float_as_uint(all.w)), "r"(m)
                    : "memory");
            }
            if (!__all_sync(~0u, cluster_mbar_wait(&sm.full[par], i >> 1 & 1, p.wait_ns))) {
                gave = i;
                // what the others may have sent for the next tile (for no later one) lands on its barrier
                if (lane == 0 && i + 1 < tiles) sm100::mbar_expect_tx(&sm.full[par ^ 1], K * 512);
            } else {
                float c0 = 0.f, c1 = 0.f;
                const float before[2] = {carry[0], carry[1]};
                signs = 0;
                for (int r = 0; r < K; ++r) {
                    if (r == (int)rank) c0 = carry[0], c1 = carry[1];
                    const float4 run = cta[(par * K + r) * 32 + lane];
                    signs = run_signs(signs, run);
                    run_through<PACKED, false>(run, carry[0], carry[1]);
                }
                if ((int)signs < 0) {
                    carry[0] = before[0], carry[1] = before[1];
                    for (int r = 0; r < K; ++r) {
                        if (r == (int)rank) c0 = carry[0], c1 = carry[1];
                        run_through<PACKED, true>(cta[(par * K + r) * 32 + lane], carry[0], carry[1]);
                    }
                }
                auto into = [&](auto any) {
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        float x0 = c0, x1 = c1;
                        run_through<PACKED, decltype(any)::value>(pre[w], x0, x1);
                        *reinterpret_cast<float2*>(&sm.warp[w][lane]) = make_float2(x0, x1);
                    }
                };
                if (far) into(std::true_type());
                else into(std::false_type());
            }
        }
        if (CL && gave >= 0)
#pragma unroll
            for (int w = 0; w < W; ++w)
                *reinterpret_cast<float2*>(&sm.warp[w][lane]) =
                    make_float2(__uint_as_float(0x7fffffffu), __uint_as_float(0x7fffffffu));
        bar_arrive(kBarCin, (W + 1) * 32);
    }
    if (gave >= 0 && lane == 0) *p.err = kErrTimeout;
    return gave;
}

// Before and after the work of a CTA of a cluster: barriers of the exchange ready everywhere,
// nobody's memory gone while another CTA may still write to it.
template <bool CL, int W>
__device__ __forceinline__ void scan_enter(ScanRuns<W, CL>& sm) {
    if (CL && threadIdx.x == 0) {
        sm100::mbar_init(&sm.full[0], 1);
        sm100::mbar_init(&sm.full[1], 1);
        sm100::mbar_fence_init();
    }
    __syncthreads();
    if (CL) {
        cluster_arrive();
        cluster_wait();
    }
}
template <bool CL>
__device__ __forceinline__ void scan_leave() {
    if (CL) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }
}
// The joining warp's: where it gave up, the others' sends of that tile and the next, all of them
// under way by now, are waited for (200 ms each where one was never sent).
template <bool CL, int W>
__device__ __forceinline__ void scan_leave(ScanRuns<W, CL>& sm, int gave, int tiles) {
    scan_leave<CL>();
    if (CL && gave >= 0)
        for (int i = gave; i < min(gave + 2, tiles); ++i) sm100::mbar_drain(&sm.full[i & 1], i >> 1 & 1);
}

// The last n with cu[n] <= t, looked for outwards from `near`; in 0 .. N - 1 whatever cu holds.
__device__ __forceinline__ int scan_owner_near(const int* cu, int N, int t, int near) {
    int lo = near, hi = near;
    if (cu[near] <= t) {
        for (int d = 1; (hi = min(near + d, N)) < N && cu[hi] <= t; d *= 2) lo = hi;
    } else {
        for (int d = 1; (lo = max(near - d, 0)) > 0 && cu[lo] > t; d *= 2) hi = lo;
    }
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Packed input: which of a warp's tokens start or end a sequence.  Tiles come in the order of
// the walk, and those short of the far end (`edge`) of the last sequence looked up, n, need no
// search.
template <int TS, int DIR>
struct ScanSeq {
    int edge = DIR > 0 ? 0 : 0x7fffffff, n = 0, own = 0;
    unsigned starts = 0, ends = 0;
    // the sequence of this lane's token (lanes past the last one: of the last) of the tile at t0
    __device__ __forceinline__ int owner(const ScanParams& p, int t0) const {
        const int lane = threadIdx.x & 31, t = t0 + DIR * (lane < TS ? lane : TS - 1);
        return scan_owner_near(p.cu, p.N, t < 0 ? 0 : t < p.T ? t : p.T - 1, n);
    }
    // s: the states that sequences begin with, in the order of the walk (or null): the next
    // one's is asked for here, long before it is needed
    __device__ __forceinline__ void find(const ScanParams& p, int t0, const float* s, int64_t sn, int c) {
        starts = ends = 0;
        if (DIR > 0 ? t0 + TS < edge : t0 - (TS - 1) > edge) return;
        const int lane = threadIdx.x & 31, t = t0 + DIR * lane;
        own = owner(p, t0);
        const bool in = lane < TS && t >= 0 && t < p.T;
        const int first = p.cu[own], e = p.cu[own + 1];
        starts = __ballot_sync(~0u, in && first == t);
        ends = __ballot_sync(~0u, in && e == t + 1);
        edge = __shfl_sync(~0u, DIR > 0 ? e : first, TS - 1);
        n = __shfl_sync(~0u, own, TS - 1);
        const int next = n + DIR;
        if (s && next >= 0 && next < p.N && c < p.D) asm volatile("prefetch.global.L2 [%0];" ::"l"(s + next * sn + c));
    }
};

template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Where they begin in shared memory, past a multiple of 128 bytes.  Forward on one: at 16 its
// copies and reads take longer (8 x 2048 x 2048 51 us, not 45, packed 222459 x 2048 597, not 551,
// 65536 x 512 118, not 102).  Backward at 16: long wide rows' five streams then come through
// faster than at 0 (65536 x 2048 338 and 360 us, 2 x 8192 x 2048 88 and 96; 32768 x 1024, the
// other way, 154 and 125).
template <bool BWD>
constexpr int kScanPlace = BWD ? 16 : 0;

// The tokens on their way, a warp's rows together.
template <typename X, typename G, int TS, bool BWD, int W>
struct ScanStage {
    G g[kScanStages][W][TS][64];
    X x[kScanStages][W][TS][64];
    X h[BWD ? kScanStages : 1][BWD ? W : 1][BWD ? TS : 1][64];
};

template <typename X, typename G, int TS, bool PACKED, bool CL, bool EVEN, bool HELD>
__global__ void __launch_bounds__(kScanThreadsOf<HELD>, 2) k_scan_piped(ScanParams p, int K, int wide) {
    extern __shared__ __align__(128) unsigned char dyn[];
    constexpr int W = kScanWarps<HELD>;
    using Stage = ScanStage<X, G, TS, false, W>;       // then [2][K][32] float4: the CTAs' runs
    Stage& st = *reinterpret_cast<Stage*>(dyn + kScanPlace<false>);
    __shared__ ScanRuns<W, CL> sm;
    if (!CL) K = 1;
    const unsigned rank = CL ? cluster_rank() : 0;
    const int item = blockIdx.x / K, ct = (p.D + 63) / 64;
    const int b = item / ct, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = (item % ct) * 64, c = c0 + lane * 2;
    const bool live = c < p.D, live1 = EVEN || c + 1 < p.D, whole = c0 + 64 <= p.D;
    const int step = K * W * TS;
    const int tiles = (int)(((int64_t)p.T + step - 1) / step);
    int t0 = ((int)rank * W + w) * TS;              // this warp's first token of tile i
    ScanSrc<X, TS, 1, EVEN> xs(static_cast<const X*>(p.x) + b * p.x_sb, p.x_st, t0, step, c0, p.D, wide & 1);
    ScanSrc<G, TS, 1, EVEN> gs(static_cast<const G*>(p.g) + b * p.g_sb, p.g_st, t0, step, c0, p.D, wide & 2);
    X* y = static_cast<X*>(p.y) + b * p.y_sb + c + t0 * p.y_st;
    const int64_t y_tile = (int64_t)step * p.y_st;
    auto load = [&](int t, int s) {
        const bool inside = whole && (unsigned)t + TS <= (unsigned)p.T;
        xs.copy(&st.x[s][w][0][0], t, p.T, inside);
        gs.copy(&st.g[s][w][0][0], t, p.T, inside);
        cp_async_commit();
    };
    if (w < W)
#pragma unroll
        for (int s = 0; s < kScanStages; ++s) load(t0 + s * step, s);
    if (PACKED) {
        scan_check_cu(p);
        if (w < W) scan_empty<W>(p, p.s0, p.s0_sn, c, K, rank);
    }
    scan_enter<CL, W>(sm);
    float cin[2], carry[2] = {0.f, 0.f};
    if (!PACKED && live && p.s0) {
        carry[0] = p.s0[b * p.s0_sn + c];
        if (live1) carry[1] = p.s0[b * p.s0_sn + c + 1];
    }
    if (w == W) {
        const int gave = scan_join<PACKED, CL, W>(sm, reinterpret_cast<float4*>(&st + 1), tiles, K, rank, carry, p);
        scan_leave<CL, W>(sm, gave, tiles);
        return;
    }
    auto initial = [&](int n, float* s) {      // the start state of sequence n
        s[0] = live && p.s0 ? p.s0[n * p.s0_sn + c] : 0.f;
        s[1] = live && live1 && p.s0 ? p.s0[n * p.s0_sn + c + 1] : 0.f;
    };
    // the run of this warp's tokens of one tile
    using GR = typename RawVec<G, 2>::T;
    struct Held {                              // the tokens of a run
        typename RawVec<X, 2>::T x[TS];
        float a[TS][2];
    };
    // all of a run's loads ahead of the first store, which they could not pass
    auto read = [&](int s, typename RawVec<X, 2>::T* rx, GR* rg) {
#pragma unroll
        for (int j = 0; j < TS; ++j) {
            rx[j] = ld_raw<X, 2>(&st.x[s][w][j][lane * 2]);
            rg[j] = ld_raw<G, 2>(&st.g[s][w][j][lane * 2]);
        }
    };
    auto form = [&](int s, unsigned starts, int own, Held& hd) {
        float h[2] = {0.f, 0.f}, L[2] = {0.f, 0.f};
        GR rg[TS];
        read(s, hd.x, rg);
#pragma unroll
        for (int j = 0; j < TS; ++j) {
            float xv[2], a[2];
            unpack(hd.x[j], xv);
            unpack(rg[j], a);
            scan_log2(a);
            add2(L, a, L);
            a[0] = scan_pow2(a[0]);
            a[1] = scan_pow2(a[1]);
            if constexpr (HELD) hd.a[j][0] = a[0], hd.a[j][1] = a[1];
            else if constexpr (sizeof(G) == 4) st_vec<G, 2>(&st.g[s][w][j][lane * 2], a);
            if (PACKED && (starts >> j & 1)) initial(__shfl_sync(~0u, own, j), h);
            fma2(a, h, xv, h);
        }
        sm.put(w, L, h, PACKED && starts);
    };
    // the same tokens again from what comes in, to the output
    auto finish = [&](int t, int s, Held& hd, unsigned starts, unsigned ends, int own) {
        GR rg[TS];
        if (!HELD) read(s, hd.x, rg);
        const int left = min(TS, p.T - t);
        X* o = y;
#pragma unroll
        for (int j = 0; j < TS; ++j, o += p.y_st) {
            float xv[2], a[2];
            unpack(hd.x[j], xv);
            if constexpr (HELD) {
                a[0] = hd.a[j][0];
                a[1] = hd.a[j][1];
            } else {
                unpack(rg[j], a);
                if constexpr (sizeof(G) == 2) {
                    scan_log2(a);
                    a[0] = scan_pow2(a[0]);
                    a[1] = scan_pow2(a[1]);
                }
            }
            if (PACKED && (starts >> j & 1)) initial(__shfl_sync(~0u, own, j), cin);
            fma2(a, cin, xv, cin);
            if (live && j < left) scan_store<X, EVEN>(o, cin, live1);
            if (PACKED && (ends >> j & 1)) {
                float* f = p.fin + __shfl_sync(~0u, own, j) * p.fin_sn + c;
                if (live && p.fin) {
                    f[0] = cin[0];
                    if (live1) f[1] = cin[1];
                }
            }
        }
        // the places past the last token hold a = 1, x = 0: they leave h as it is
        if (!PACKED && left > 0 && left >= p.T - t && live && p.fin) {
            p.fin[b * p.fin_sn + c] = cin[0];
            if (live1) p.fin[b * p.fin_sn + c + 1] = cin[1];
        }
    };
    ScanSeq<TS, 1> seq;
    auto next = [&](int t, int s, Held& hd) {   // the run of a tile that has landed
        __syncwarp();
        unsigned cut = 0;
        if (PACKED) {
            seq.find(p, t, p.s0, p.s0_sn, c);
            cut = seq.starts;
        }
        if (PACKED && cut) form(s, cut, seq.own, hd);
        else form(s, 0u, 0, hd);
        bar_arrive(kBarRuns, kScanThreadsOf<HELD>);
        if (HELD) {                              // its place is free
            __syncwarp();
            load(t + kScanStages * step, s);
        }
    };
    Held even, odd;
    int s = 0;
    cp_async_wait<kScanStages - 1>();
    next(t0, 0, even);
    auto tile = [&](int i, Held& now, Held& then) {
        bar_sync(kBarCin, kScanThreadsOf<HELD>);
        const float2 in = *reinterpret_cast<const float2*>(&sm.warp[w][lane]);
        cin[0] = in.x;
        cin[1] = in.y;
        const unsigned starts = seq.starts, ends = seq.ends;
        const int own = seq.own, s1 = s + 1 == kScanStages ? 0 : s + 1;
        if (i + 1 < tiles) {
            cp_async_wait<HELD ? kScanStages - 1 : kScanStages - 2>();
            next(t0 + step, s1, then);
        }
        if (PACKED && (starts | ends)) finish(t0, s, now, starts, ends, HELD ? own : seq.owner(p, t0));   // (registers, or a search)
        else finish(t0, s, now, 0u, 0u, 0);
        if (!HELD) {
            __syncwarp();
            load(t0 + kScanStages * step, s);
        }
        s = s1;
        t0 += step;
        y += y_tile;
    };
    if constexpr (HELD) {
        for (int i = 0; i < tiles; i += 2) {
            tile(i, even, odd);
            if (i + 1 < tiles) tile(i + 1, odd, even);
        }
    } else {
        for (int i = 0; i < tiles; ++i) tile(i, even, odd);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    scan_leave<CL>();
}

template <typename X, typename G, int TS, bool PACKED, bool CL, bool EVEN>
__global__ void __launch_bounds__(kScanThreadsOf<false>, 2) k_scan_bwd_piped(ScanParams p, int K, int wide) {
    extern __shared__ __align__(128) unsigned char dyn[];
    constexpr int W = kScanWarps<false>;
    using Stage = ScanStage<X, G, TS, true, W>;       // then [2][K][32] float4: the CTAs' runs
    Stage& st = *reinterpret_cast<Stage*>(dyn + kScanPlace<true>);
    __shared__ ScanRuns<W, CL> sm;
    if (!CL) K = 1;
    const unsigned rank = CL ? cluster_rank() : 0;
    const int item = blockIdx.x / K, ct = (p.D + 63) / 64;
    const int b = item / ct, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = (item % ct) * 64, c = c0 + lane * 2;
    const bool live = c < p.D, live1 = EVEN || c + 1 < p.D, whole = c0 + 64 <= p.D;
    const int step = K * W * TS;
    const int tiles = (int)(((int64_t)p.T + step - 1) / step);
    int t0 = p.T - 1 - ((int)rank * W + w) * TS;    // token of place j of tile i: t0 - j
    ScanSrc<X, TS, -1, EVEN> ds(static_cast<const X*>(p.x) + b * p.x_sb, p.x_st, t0, step, c0, p.D, wide & 1);
    ScanSrc<G, TS, -1, EVEN> gs(static_cast<const G*>(p.g) + b * p.g_sb, p.g_st, t0, step, c0, p.D, wide & 2);
    ScanSrc<X, TS, -1, EVEN> hs(static_cast<const X*>(p.h) + b * p.h_sb, p.h_st, t0 - 1, step, c0, p.D, wide & 4);
    X* dx = static_cast<X*>(p.y) + b * p.y_sb + c + t0 * p.y_st;
    G* dg = static_cast<G*>(p.dg) + b * p.dg_sb + c + t0 * p.dg_st;
    const int64_t dx_tile = (int64_t)step * p.y_st, dg_tile = (int64_t)step * p.dg_st;
    auto load = [&](int t, int s) {
        const bool inside = whole && t >= TS - 1;
        ds.copy(&st.x[s][w][0][0], t, p.T, inside);
        gs.copy(&st.g[s][w][0][0], t, p.T, inside);
        hs.copy(&st.h[s][w][0][0], t - 1, p.T, inside && t >= TS);
        cp_async_commit();
    };
    if (w < W)
#pragma unroll
        for (int s = 0; s < kScanStages; ++s) load(t0 - s * step, s);
    if (PACKED) {
        scan_check_cu(p);
        if (w < W) scan_empty<W>(p, p.sT, p.sT_sn, c, K, rank);
    }
    scan_enter<CL, W>(sm);
    float cin[2], carry[2] = {0.f, 0.f};
    if (!PACKED && live && p.sT) {
        carry[0] = p.sT[b * p.sT_sn + c];
        if (live1) carry[1] = p.sT[b * p.sT_sn + c + 1];
    }
    if (w == W) {
        const int gave = scan_join<PACKED, CL, W>(sm, reinterpret_cast<float4*>(&st + 1), tiles, K, rank, carry, p);
        scan_leave<CL, W>(sm, gave, tiles);
        return;
    }
    auto state = [&](const float* src, int64_t sn, int n, float* s) {
        s[0] = live && src ? src[n * sn + c] : 0.f;
        s[1] = live && live1 && src ? src[n * sn + c + 1] : 0.f;
    };
    using XR = typename RawVec<X, 2>::T;
    using GR = typename RawVec<G, 2>::T;
    auto read = [&](int s, XR* rd, GR* rg) {
#pragma unroll
        for (int j = 0; j < TS; ++j) {
            rd[j] = ld_raw<X, 2>(&st.x[s][w][j][lane * 2]);
            rg[j] = ld_raw<G, 2>(&st.g[s][w][j][lane * 2]);
        }
    };
    auto read_h = [&](int s, XR* rh) {
#pragma unroll
        for (int j = 0; j < TS; ++j) rh[j] = ld_raw<X, 2>(&st.h[s][w][j][lane * 2]);
    };
    auto form = [&](int s, unsigned ends, int own) {
        float e[2] = {0.f, 0.f}, L[2] = {0.f, 0.f};
        XR rd[TS];
        GR rg[TS];
        read(s, rd, rg);
#pragma unroll
        for (int j = 0; j < TS; ++j) {
            float dv[2], a[2];
            unpack(rd[j], dv);
            unpack(rg[j], a);
            scan_log2(a);
            add2(L, a, L);
            a[0] = scan_pow2(a[0]);
            a[1] = scan_pow2(a[1]);
            if constexpr (sizeof(G) == 4) st_vec<G, 2>(&st.g[s][w][j][lane * 2], a);
            if (PACKED && (ends >> j & 1)) state(p.sT, p.sT_sn, __shfl_sync(~0u, own, j), e);
            add2(dv, e, e);
            mul2(a, e, e);
        }
        sm.put(w, L, e, PACKED && ends);
    };
    auto finish = [&](int t, int s, unsigned starts, unsigned ends, int own) {
        XR rd[TS], rh[TS];
        GR rg[TS];
        read(s, rd, rg);
        read_h(s, rh);
        // places up to `left` hold tokens; dense: place left - 1 of the last tile is token 0
        const int left = max(0, min(TS, t + 1));
        const bool at0 = !PACKED && left > 0 && t < TS;
        X* ox = dx;
        G* og = dg;
#pragma unroll
        for (int j = 0; j < TS; ++j, ox -= p.y_st, og -= p.dg_st) {
            float dv[2], a[2], hv[2];
            unpack(rd[j], dv);
            unpack(rh[j], hv);
            unpack(rg[j], a);
            if constexpr (sizeof(G) == 2) {
                scan_log2(a);
                a[0] = scan_pow2(a[0]);
                a[1] = scan_pow2(a[1]);
            }
            int n = b;
            if (PACKED && ((starts | ends) >> j & 1)) n = __shfl_sync(~0u, own, j);
            if (PACKED && (ends >> j & 1)) state(p.sT, p.sT_sn, n, cin);
            if (PACKED ? (starts >> j & 1) : at0 && j == left - 1) state(p.s0, p.s0_sn, n, hv);
            float d[2], q[2];
            add2(dv, cin, d);
            mul2(a, d, cin);
            mul2(cin, hv, q);
            if (live && j < left) {
                scan_store<X, EVEN>(ox, d, live1);
                scan_store<G, EVEN>(og, q, live1);
            }
            if (PACKED && (starts >> j & 1) && live && p.fin) {
                p.fin[n * p.fin_sn + c] = cin[0];
                if (live1) p.fin[n * p.fin_sn + c + 1] = cin[1];
            }
        }
        // the places past token 0 hold a = 1, d = 0: they leave what comes in as it is
        if (at0 && live && p.fin) {
            p.fin[b * p.fin_sn + c] = cin[0];
            if (live1) p.fin[b * p.fin_sn + c + 1] = cin[1];
        }
    };
    ScanSeq<TS, -1> seq;
    auto next = [&](int t, int s) {            // the run of a tile that has landed
        __syncwarp();
        unsigned cut = 0;
        if (PACKED) {
            seq.find(p, t, p.sT, p.sT_sn, c);
            cut = seq.ends;
        }
        if (PACKED && cut) form(s, cut, seq.own);
        else form(s, 0u, 0);
        bar_arrive(kBarRuns, kScanThreadsOf<false>);
    };
    int s = 0;
    cp_async_wait<kScanStages - 1>();
    next(t0, 0);
    for (int i = 0; i < tiles; ++i) {
        bar_sync(kBarCin, kScanThreadsOf<false>);
        const float2 in = *reinterpret_cast<const float2*>(&sm.warp[w][lane]);
        cin[0] = in.x;
        cin[1] = in.y;
        const unsigned starts = seq.starts, ends = seq.ends;
        const int s1 = s + 1 == kScanStages ? 0 : s + 1;
        if (i + 1 < tiles) {
            cp_async_wait<kScanStages - 2>();
            next(t0 - step, s1);
        }
        if (PACKED && (starts | ends)) finish(t0, s, starts, ends, seq.owner(p, t0));    // (registers, or a search)
        else finish(t0, s, 0u, 0u, 0);
        __syncwarp();
        load(t0 - kScanStages * step, s);
        s = s1;
        t0 -= step;
        dx -= dx_tile;
        dg -= dg_tile;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    scan_leave<CL>();
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

// One thread per V channels of a request, V = 4 where rows are made of such pieces.
template <typename X, typename G, int V>
__global__ void __launch_bounds__(kScanThreads) k_scan_step(ScanStepParams p) {
    const int per = (p.D + kScanThreads * V - 1) / (kScanThreads * V);
    const int n = blockIdx.x / per, c = ((blockIdx.x % per) * kScanThreads + threadIdx.x) * V;
    const int64_t slot = step_slot(p.slots, p.M, n, p.err);
    if (c >= p.D) return;
    auto load = [](const auto* q, float* f) {
        if constexpr (V == 4) *reinterpret_cast<float4*>(f) = ld_elem4(q);
        else f[0] = ld_elem(q);
    };
    auto store = [](auto* q, const float* f) {
        if constexpr (V == 4) st_elem4(q, make_float4(f[0], f[1], f[2], f[3]));
        else st_elem(q, f[0]);
    };
    X* y = static_cast<X*>(p.y) + n * p.y_sn + c;
    alignas(16) float h[V] = {}, xv[V], a[V];
    if (slot < 0) {
        for (int t = 0; t < p.T; ++t) store(y + t * p.y_st, h);
        return;
    }
    const X* x = static_cast<const X*>(p.x) + n * p.x_sn + c;
    const G* g = static_cast<const G*>(p.g) + n * p.g_sn + c;
    float* s = p.state + slot * p.s_sm + c;
    load(s, h);
    for (int t = 0; t < p.T; ++t) {
        load(x + t * p.x_st, xv);
        load(g + t * p.g_st, a);
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = fmaf(expf(a[v]), h[v], xv[v]);
        store(y + t * p.y_st, h);
    }
    store(s, h);
}

}  // namespace dn
