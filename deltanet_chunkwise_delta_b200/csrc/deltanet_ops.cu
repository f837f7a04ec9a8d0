// Host side of the operators around the delta-rule kernels (include/deltanet.h):
// deltanet_step and deltanet_scan_*.  Argument checks and launches only.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "../../include/deltanet.h"
#include "dn_host.h"
#include "dn_scan.cuh"
#include "dn_step.cuh"

using namespace dn;

namespace {

// [B, T, H] fp32 scalars per token and head, any non-negative strides.
bool scalars_ok(const dn_tensor* t, const int64_t* dims) {
    if (!shape_eq(t, 3, dims) || t->dtype != DN_F32) return false;
    for (int i = 0; i < 3; ++i)
        if (t->stride[i] < 0) return false;
    return numel(t) == 0 || (t->data && reinterpret_cast<uintptr_t>(t->data) % 4 == 0);
}

template <typename E, int DK, int DV, StepKind KIND>
void launch_step(const StepParams& p, int gate, unsigned grid, cudaStream_t s) {
    if (gate == 0) k_step<E, DK, DV, 0, KIND><<<grid, DK, 0, s>>>(p);
    else if (gate == 1) k_step<E, DK, DV, 1, KIND><<<grid, DK, 0, s>>>(p);
    else k_step<E, DK, DV, 2, KIND><<<grid, DK, 0, s>>>(p);
}

template <typename E, int DK, int DV>
void launch_step(const StepParams& p, int gate, unsigned grid, cudaStream_t s) {
    if (p.nh > 1) launch_step<E, DK, DV, kStepWrites>(p, gate, grid, s);
    else if (p.T > 1) launch_step<E, DK, DV, kStepTokens>(p, gate, grid, s);
    else launch_step<E, DK, DV, kStepOne>(p, gate, grid, s);
}

template <typename E>
void launch_step(const StepParams& p, int64_t dk, int64_t dv, int gate, unsigned grid, cudaStream_t s) {
    if (dk == 128 && dv == 128) launch_step<E, 128, 128>(p, gate, grid, s);
    else if (dk == 128) launch_step<E, 128, 64>(p, gate, grid, s);
    else if (dv == 128) launch_step<E, 64, 128>(p, gate, grid, s);
    else launch_step<E, 64, 64>(p, gate, grid, s);
}

// The state cache and slot indices of the step entry points; M rows.  Every CTA looks a slot up
// among those before it (step_slot): with 2^20 requests that is 2^39 reads for every row of CTAs,
// and with a hundred times as many it would hold the GPU for an hour.
constexpr int64_t kMaxSlots = int64_t(1) << 20;
dn_status cache_check(const dn_tensor* state, const dn_tensor* slots, int64_t N) {
    if (slots && N > kMaxSlots) return DN_ERR_INVALID_ARG;
    if (slots ? !index_ok(slots, 0) || slots->shape[0] != N : state->shape[0] != N) return DN_ERR_INVALID_ARG;
    return state->shape[0] <= kMax31 ? DN_OK : DN_ERR_INVALID_ARG;
}

// Kernel choice by the dtypes of x and g: f(X(), G()).
template <typename F>
void by_types(int32_t x, int32_t g, F f) {
    if (x == DN_F32) f(float(), float());
    else if (g == DN_F32) f(__nv_bfloat16(), float());
    else f(__nv_bfloat16(), __nv_bfloat16());
}

constexpr int64_t kMaxSize = kMax31 - 16384;

// Shapes of deltanet_scan_fwd / _bwd: x [B, T, D] (x: its dtype and shape lead), g, the state
// tensors, the packed boundaries.  Sets N.
dn_status scan_shapes(const dn_tensor* x, const dn_tensor* g, const dn_tensor* cu, int64_t& N) {
    if (!x || !g || x->ndim != 3) return DN_ERR_INVALID_ARG;
    const int64_t B = x->shape[0], T = x->shape[1], D = x->shape[2];
    if (B < 0 || T < 0 || D < 1 || D > kMax31 || T > kMax31 || B > kMax31) return DN_ERR_INVALID_ARG;
    if (T > 0 && B > kMax31 / T) return DN_ERR_INVALID_ARG;
    // the kernels' token counters run past T by a few tiles, their channels past D by a CTA's
    if (T > kMaxSize || D > kMaxSize) return DN_ERR_INVALID_ARG;
    const int64_t dims[3] = {B, T, D};
    if (!view_ok(x, 3, dims, kF32 | kBf16)) return DN_ERR_INVALID_ARG;
    if (!view_ok(g, 3, dims, x->dtype == DN_F32 ? kF32 : kF32 | kBf16)) return DN_ERR_INVALID_ARG;
    N = B;
    if (cu) {
        if (!index_ok(cu, 1) || B != 1) return DN_ERR_INVALID_ARG;
        N = cu->shape[0] - 1;
        if (N >= (int64_t(1) << 24) || (N == 0 && T > 0)) return DN_ERR_INVALID_ARG;   // (tokens of no sequence)
    }
    if (N > 0 && (D + kScanWalkers - 1) / kScanWalkers > kMax31 / N) return DN_ERR_INVALID_ARG;   // a grid's CTAs
    return DN_OK;
}

dn_status scan_common(ScanParams& p, const dn_tensor* x, const dn_tensor* g, const dn_tensor* cu, int64_t N,
                      cudaStream_t stream) {
    int dev = 0, sms = 0;
    dn_status st = dn_device_check(dev, sms);
    if (st != DN_OK) return st;
    std::memset(&p, 0, sizeof p);
    p.x = x->data; p.x_sb = x->stride[0]; p.x_st = x->stride[1];
    p.g = g->data; p.g_sb = g->stride[0]; p.g_st = g->stride[1];
    p.B = (int)x->shape[0]; p.T = (int)x->shape[1]; p.D = (int)x->shape[2]; p.N = (int)N;
    dn_wait_settings(&p.wait_ns, &p.stall);
    if (!p.wait_ns) p.wait_ns = sm100::kDefaultWaitNs;
    if (!cu) return DN_OK;
    p.cu = static_cast<const int*>(cu->data);
    return dn_stream_flag(dev, stream, &p.err);
}

// Pairs of channels can move as one access: even D, strides and addresses.
bool scan_pairs(const ScanParams& p, int32_t x, int32_t g, bool bwd) {
    auto ok = [](const void* a, int64_t sb, int64_t st, int32_t dt) {
        return reinterpret_cast<uintptr_t>(a) % (2 * elem_size(dt)) == 0 && sb % 2 == 0 && st % 2 == 0;
    };
    return p.D % 2 == 0 && ok(p.x, p.x_sb, p.x_st, x) && ok(p.g, p.g_sb, p.g_st, g) &&
           ok(p.y, p.y_sb, p.y_st, x) && (!bwd || (ok(p.h, p.h_sb, p.h_st, x) && ok(p.dg, p.dg_sb, p.dg_st, g)));
}

// CTAs per cluster: enough for most SMs, and on to one and a third of them where a row is
// split anyway (a cluster's CTAs often sit two to an SM), each with one and a half tiles or
// more.  Measured with 1, 2, 4, 8 (forward, bf16, fp32 gates): 16 channel tiles of 32768 tokens
// 334, 180, 95, 69 us; 32 of 16384 172, 93, 52, 50; 64 of 512 8.3, 8.7, 8.0, 10.9; 256 of
// 2048 44, 51, 59, 85; 128 of 1024 15, 17, 23, 28 us.
int scan_cluster(int64_t items, int64_t T, int tokens, int sms) {
    int K = 1;
    while (K < kScanMaxCluster && (items * K < sms * 5 / 6 || (K > 1 && items * K < sms * 4 / 3)) &&
           (int64_t)K * tokens * 3 <= T)
        K *= 2;
    return K;
}

template <typename Kern, typename... A>
dn_status scan_launch(Kern* kern, int64_t items, int K, int threads, int smem, int most, cudaStream_t stream,
                      const ScanParams& p, A... a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * K));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)K;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = K > 1 ? 1 : 0;
    // the same limit in every call: calls on several host threads share the kernel's attribute
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
        return DN_ERR_CUDA;
    return cudaLaunchKernelEx(&cfg, kern, p, K, a...) == cudaSuccess ? DN_OK : DN_ERR_CUDA;
}

// Up to so many tokens a thread walks its channels, and up to the larger number where that
// fills the GPU (four CTAs of walkers on an SM).  2048 channels, bf16 with fp32 gates, walkers
// against tiles: 32 tokens of 512 rows 45 and 158 us, 128 of 128 rows 45 and 62, 192 of 85 rows
// 48 and 55, 512 of 32 rows 85 and 49; backward 32 of 512 80 and 240, 512 of 128 343 and 302.
constexpr int kScanSerialT = 16, kScanSerialManyT = 192;

// 16-byte copies: bit 0 for x, 1 for g, 2 for h.
int scan_wide(const ScanParams& p, int32_t x, int32_t g) {
    auto ok = [](const void* a, int64_t sb, int64_t st, int32_t dt) {
        const int64_t es = elem_size(dt);
        return aligned16(a) && sb * es % 16 == 0 && st * es % 16 == 0;
    };
    return (ok(p.x, p.x_sb, p.x_st, x) ? 1 : 0) | (ok(p.g, p.g_sb, p.g_st, g) ? 2 : 0) |
           (p.h && ok(p.h, p.h_sb, p.h_st, x) ? 4 : 0);
}

template <typename X, typename G, bool PACKED, bool BWD, bool EVEN>
dn_status scan_tiled(ScanParams& p, int dev, int sms, cudaStream_t stream) {
    const int64_t items = (int64_t)(PACKED ? 1 : p.B) * ((p.D + 63) / 64);
    // Held runs where the instructions bound the tiles, and tokens per run as many as registers
    // or two CTAs' shared memory allow.  Held and read twice: rows of one CTA, 8 x 2048 x 2048,
    // bf16 gates 35 and 38 us, fp32 gates 45 and 45, all fp32 66 and 64; clusters of 8, 65536 x
    // 2048 all fp32 278 and 303, 222459 x 2048 packed all bf16 547 and 634 us.  Backward reads
    // twice (held: 65536 x 2048 339 us, not 335, 8 x 2048 x 2048 93, not 90).
    constexpr bool H1 = !BWD && sizeof(G) == 2, HK = !BWD;
    constexpr int T1 = sizeof(X) == 4 ? 4 : 8, TK = T1 + (HK && EVEN ? 4 : 0);
    constexpr int W1 = kScanWarps<H1>, WK = kScanWarps<HK>;
    constexpr int stage = kScanPlace<BWD> + (int)sizeof(ScanStage<X, G, T1, BWD, W1>);
    constexpr int part = kScanPlace<BWD> + (int)sizeof(ScanStage<X, G, TK, BWD, WK>);
    static_assert(2 * (stage + sizeof(ScanRuns<W1, false>) + 128 + 1024) <= 228 * 1024 &&
                  2 * (part + 8192 + sizeof(ScanRuns<WK, true>) + 128 + 1024) <= 228 * 1024, "two CTAs on an SM, clusters of 8");
    const int K = scan_cluster(items, p.T, WK * TK, sms);
    const int wide = scan_wide(p, sizeof(X) == 4 ? DN_F32 : DN_BF16, sizeof(G) == 4 ? DN_F32 : DN_BF16);
    if (items > kMax31 / K) return DN_ERR_INVALID_ARG;
    auto go = [&](auto* kern, int threads, int smem, int most) { return scan_launch(kern, items, K, threads, smem, most, stream, p, wide); };
    if (K > 1) {
        // a wait inside a cluster that gives up is reported (packed input has its word)
        const dn_status st = p.err ? DN_OK : dn_stream_flag(dev, stream, &p.err);
        if (st != DN_OK) return st;
        constexpr int th = kScanThreadsOf<HK>;
        const int smem = part + K * 1024, most = part + kScanMaxCluster * 1024;
        if constexpr (BWD) return go(k_scan_bwd_piped<X, G, TK, PACKED, true, EVEN>, th, smem, most);
        else return go(k_scan_piped<X, G, TK, PACKED, true, EVEN, HK>, th, smem, most);
    }
    constexpr int th = kScanThreadsOf<H1>;
    if constexpr (BWD) return go(k_scan_bwd_piped<X, G, T1, PACKED, false, EVEN>, th, stage, stage);
    else return go(k_scan_piped<X, G, T1, PACKED, false, EVEN, H1>, th, stage, stage);
}

template <bool BWD>
dn_status scan_run(ScanParams& p, int32_t x, int32_t g, cudaStream_t stream) {
    int dev = 0, sms = 0;
    dn_status st = dn_device_check(dev, sms);
    if (st != DN_OK) return st;
    by_types(x, g, [&](auto xt, auto gt) {
        using X = decltype(xt);
        using G = decltype(gt);
        const bool even = scan_pairs(p, x, g, BWD);
        const int V = even ? 2 : 1;
        const int64_t walkers = (int64_t)p.N * ((p.D + kScanWalkers * V - 1) / (kScanWalkers * V));
        if (p.T <= kScanSerialT || (p.T <= kScanSerialManyT && walkers >= 4 * sms)) {
            const unsigned grid = (unsigned)walkers;
            if constexpr (BWD) {
                if (even) k_scan_bwd_serial<X, G, 2><<<grid, kScanWalkers, 0, stream>>>(p);
                else k_scan_bwd_serial<X, G, 1><<<grid, kScanWalkers, 0, stream>>>(p);
            } else {
                if (even) k_scan_serial<X, G, 2><<<grid, kScanWalkers, 0, stream>>>(p);
                else k_scan_serial<X, G, 1><<<grid, kScanWalkers, 0, stream>>>(p);
            }
        } else if (even) {
            st = p.cu ? scan_tiled<X, G, true, BWD, true>(p, dev, sms, stream) : scan_tiled<X, G, false, BWD, true>(p, dev, sms, stream);
        } else {
            st = p.cu ? scan_tiled<X, G, true, BWD, false>(p, dev, sms, stream) : scan_tiled<X, G, false, BWD, false>(p, dev, sms, stream);
        }
    });
    return st == DN_OK ? launched(1) : st;
}

template <typename P>
void set_state(const dn_tensor* t, P*& ptr, int64_t& stride) {
    if (t && numel(t)) {
        ptr = static_cast<P*>(t->data);
        stride = t->stride[0];
    }
}

}  // namespace

extern "C" {

dn_status deltanet_step(const dn_tensor* q, const dn_tensor* k, const dn_tensor* v, const dn_tensor* beta,
                        const dn_tensor* g, int n_h, dn_tensor* state, const dn_tensor* slot_idx,
                        dn_tensor* out, void* stream_ptr) {
    if (!q || !k || !v || !beta || !state || !out) return DN_ERR_INVALID_ARG;
    if (q->ndim != 4 || v->ndim != 4 || state->ndim != 4 || n_h < 1 || n_h > 1024) return DN_ERR_INVALID_ARG;
    const int64_t N = q->shape[0], T = q->shape[1], H = q->shape[2], dk = q->shape[3], dv = v->shape[3];
    if (N < 0 || T < 0 || H < 0 || dk < 1 || dv < 1) return DN_ERR_INVALID_ARG;
    if (N > kMax31 || T > kMax31 / n_h || H >= 65536) return DN_ERR_INVALID_ARG;
    if (T > 0 && N > kMax31 / (T * n_h)) return DN_ERR_INVALID_ARG;
    const int64_t Tw = T * n_h, M = state->shape[0];
    const int64_t kd[4] = {N, Tw, H, dk}, vd[4] = {N, Tw, H, dv}, od[4] = {N, T, H, dv}, bd[3] = {N, Tw, H};
    const int64_t sd[4] = {M, H, dk, dv}, gd[4] = {N, T, H, dk};
    const int32_t dt = q->dtype;
    if (dt != DN_BF16 && dt != DN_F32) return DN_ERR_INVALID_ARG;
    if (!shape_eq(k, 4, kd) || !shape_eq(v, 4, vd) || !shape_eq(out, 4, od) || k->dtype != dt ||
        v->dtype != dt || out->dtype != dt)
        return DN_ERR_INVALID_ARG;
    if (!token_tensor_ok(q) || !token_tensor_ok(k) || !token_tensor_ok(v) || !token_tensor_ok(out))
        return DN_ERR_INVALID_ARG;
    if (!scalars_ok(beta, bd)) return DN_ERR_INVALID_ARG;
    int gate = 0;
    if (g) {
        gate = g->ndim == 4 ? 2 : 1;
        if (gate == 1 ? !scalars_ok(g, gd)
                      : !shape_eq(g, 4, gd) || g->dtype != DN_F32 || !token_tensor_ok(g))
            return DN_ERR_INVALID_ARG;
    }
    if (M < 0 || !shape_eq(state, 4, sd) || !state_tensor_ok(state, dv)) return DN_ERR_INVALID_ARG;
    dn_status st = cache_check(state, slot_idx, N);
    if (st != DN_OK) return st;
    if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return DN_ERR_UNSUPPORTED;
    if ((st = alias_check({out, state}, {q, k, v, beta, g, slot_idx})) != DN_OK) return st;
    const int64_t ctas = dv / kStepCols;
    if (H > 0 && N > kMax31 / (H * ctas)) return DN_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if ((st = dn_device_check(dev, sms)) != DN_OK) return st;
    if (N == 0 || T == 0 || H == 0) return DN_OK;

    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    StepParams p;
    std::memset(&p, 0, sizeof p);
    p.q = q->data; p.q_sn = q->stride[0]; p.q_st = q->stride[1]; p.q_sh = q->stride[2];
    p.k = k->data; p.k_sn = k->stride[0]; p.k_st = k->stride[1]; p.k_sh = k->stride[2];
    p.v = v->data; p.v_sn = v->stride[0]; p.v_st = v->stride[1]; p.v_sh = v->stride[2];
    p.o = out->data; p.o_sn = out->stride[0]; p.o_st = out->stride[1]; p.o_sh = out->stride[2];
    p.beta = static_cast<const float*>(beta->data);
    p.b_sn = beta->stride[0]; p.b_st = beta->stride[1]; p.b_sh = beta->stride[2];
    if (g) {
        p.g = static_cast<const float*>(g->data);
        p.g_sn = g->stride[0]; p.g_st = g->stride[1]; p.g_sh = g->stride[2];
    }
    p.state = static_cast<float*>(state->data);
    p.s_sm = state->stride[0]; p.s_sh = state->stride[1];
    p.M = M;
    p.N = (int)N; p.T = (int)T; p.H = (int)H; p.nh = n_h;
    if (slot_idx) {
        p.slots = static_cast<const int*>(slot_idx->data);
        if ((st = dn_stream_flag(dev, stream, &p.err)) != DN_OK) return st;
    }
    const unsigned grid = (unsigned)(N * H * ctas);
    if (dt == DN_F32) launch_step<float>(p, dk, dv, gate, grid, stream);
    else launch_step<__nv_bfloat16>(p, dk, dv, gate, grid, stream);
    return launched(1);
}

dn_status deltanet_scan_fwd(const dn_tensor* x, const dn_tensor* g, const dn_tensor* initial_state,
                            const dn_tensor* cu_seqlens, dn_tensor* out, dn_tensor* final_state,
                            void* stream_ptr) {
    int64_t N = 0;
    dn_status st = scan_shapes(x, g, cu_seqlens, N);
    if (st != DN_OK) return st;
    const int64_t D = x->shape[2], sd[2] = {N, D};
    if (!out || !view_ok(out, 3, x->shape, 1 << x->dtype)) return DN_ERR_INVALID_ARG;
    if (initial_state && !view_ok(initial_state, 2, sd, kF32)) return DN_ERR_INVALID_ARG;
    if (final_state && !view_ok(final_state, 2, sd, kF32)) return DN_ERR_INVALID_ARG;
    if ((st = alias_check({out, final_state}, {x, g, initial_state, cu_seqlens})) != DN_OK) return st;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    ScanParams p;
    if ((st = scan_common(p, x, g, cu_seqlens, N, stream)) != DN_OK) return st;
    if (N == 0) return DN_OK;
    p.y = out->data; p.y_sb = out->stride[0]; p.y_st = out->stride[1];
    set_state(initial_state, p.s0, p.s0_sn);
    set_state(final_state, p.fin, p.fin_sn);
    return scan_run<false>(p, x->dtype, g->dtype, stream);
}

dn_status deltanet_scan_bwd(const dn_tensor* g, const dn_tensor* out, const dn_tensor* initial_state,
                            const dn_tensor* cu_seqlens, const dn_tensor* d_out,
                            const dn_tensor* d_final_state, dn_tensor* d_x, dn_tensor* d_g,
                            dn_tensor* d_initial_state, void* stream_ptr) {
    int64_t N = 0;
    dn_status st = scan_shapes(out, g, cu_seqlens, N);
    if (st != DN_OK) return st;
    const int64_t D = out->shape[2], sd[2] = {N, D};
    const int xt = 1 << out->dtype;
    if (!d_out || !view_ok(d_out, 3, out->shape, xt) || !d_x || !view_ok(d_x, 3, out->shape, xt) || !d_g ||
        !view_ok(d_g, 3, out->shape, 1 << g->dtype))
        return DN_ERR_INVALID_ARG;
    for (const dn_tensor* t : {initial_state, d_final_state, (const dn_tensor*)d_initial_state})
        if (t && !view_ok(t, 2, sd, kF32)) return DN_ERR_INVALID_ARG;
    if ((st = alias_check({d_x, d_g, d_initial_state},
                          {g, out, initial_state, cu_seqlens, d_out, d_final_state})) != DN_OK)
        return st;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    ScanParams p;
    if ((st = scan_common(p, d_out, g, cu_seqlens, N, stream)) != DN_OK) return st;
    if (N == 0) return DN_OK;
    p.h = out->data; p.h_sb = out->stride[0]; p.h_st = out->stride[1];
    p.y = d_x->data; p.y_sb = d_x->stride[0]; p.y_st = d_x->stride[1];
    p.dg = d_g->data; p.dg_sb = d_g->stride[0]; p.dg_st = d_g->stride[1];
    set_state(initial_state, p.s0, p.s0_sn);
    set_state(d_final_state, p.sT, p.sT_sn);
    set_state(d_initial_state, p.fin, p.fin_sn);
    return scan_run<true>(p, out->dtype, g->dtype, stream);
}

dn_status deltanet_scan_step(const dn_tensor* x, const dn_tensor* g, dn_tensor* state,
                             const dn_tensor* slot_idx, dn_tensor* out, void* stream_ptr) {
    int64_t N = 0;
    dn_status st = scan_shapes(x, g, nullptr, N);
    if (st != DN_OK) return st;
    if (!state || state->ndim != 2 || state->shape[0] < 0) return DN_ERR_INVALID_ARG;
    const int64_t T = x->shape[1], D = x->shape[2], sd[2] = {state->shape[0], D};
    if (!out || !view_ok(out, 3, x->shape, 1 << x->dtype) || !view_ok(state, 2, sd, kF32))
        return DN_ERR_INVALID_ARG;
    if ((st = cache_check(state, slot_idx, N)) != DN_OK) return st;
    if ((st = alias_check({out, state}, {x, g, slot_idx})) != DN_OK) return st;
    int dev = 0, sms = 0;
    if ((st = dn_device_check(dev, sms)) != DN_OK) return st;
    if (N == 0 || T == 0) return DN_OK;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    ScanStepParams p;
    std::memset(&p, 0, sizeof p);
    p.x = x->data; p.x_sn = x->stride[0]; p.x_st = x->stride[1];
    p.g = g->data; p.g_sn = g->stride[0]; p.g_st = g->stride[1];
    p.y = out->data; p.y_sn = out->stride[0]; p.y_st = out->stride[1];
    p.state = static_cast<float*>(state->data);
    p.s_sm = state->stride[0];
    p.M = state->shape[0];
    p.N = (int)N; p.T = (int)T; p.D = (int)D;
    if (slot_idx) {
        p.slots = static_cast<const int*>(slot_idx->data);
        if ((st = dn_stream_flag(dev, stream, &p.err)) != DN_OK) return st;
    }
    auto fours = [](const void* q, int64_t sn, int64_t st, int32_t dt) {
        return reinterpret_cast<uintptr_t>(q) % (4 * elem_size(dt)) == 0 && sn % 4 == 0 && st % 4 == 0;
    };
    const int V = D % 4 == 0 && fours(p.x, p.x_sn, p.x_st, x->dtype) && fours(p.g, p.g_sn, p.g_st, g->dtype) &&
                  fours(p.y, p.y_sn, p.y_st, x->dtype) && fours(p.state, p.s_sm, 0, DN_F32) ? 4 : 1;
    const unsigned grid = (unsigned)(N * ((D + kScanThreads * V - 1) / (kScanThreads * V)));
    by_types(x->dtype, g->dtype, [&](auto xt, auto gt) {
        if (V == 4) k_scan_step<decltype(xt), decltype(gt), 4><<<grid, kScanThreads, 0, stream>>>(p);
        else k_scan_step<decltype(xt), decltype(gt), 1><<<grid, kScanThreads, 0, stream>>>(p);
    });
    return launched(1);
}

}  // extern "C"
