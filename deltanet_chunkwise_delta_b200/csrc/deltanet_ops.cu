// Host side of the operators around the delta-rule kernels (include/deltanet.h):
// deltanet_step, deltanet_scan_* and deltanet_norm_*.  Argument checks and launches only.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "../../include/deltanet.h"
#include "dn_host.h"
#include "dn_norm.cuh"
#include "dn_scan.cuh"
#include "dn_step.cuh"

using namespace dn;

namespace {

constexpr int64_t kMax31 = (int64_t(1) << 31) - 1;

// A tensor of the given shape: a dtype of the mask, last stride 1, non-negative strides,
// data aligned to its element (any address where it has no elements).
constexpr int kF32 = 1 << DN_F32, kBf16 = 1 << DN_BF16;
bool view_ok(const dn_tensor* t, int ndim, const int64_t* dims, int dtypes) {
    if (!shape_eq(t, ndim, dims) || t->dtype < 0 || t->dtype > 2 || !(dtypes >> t->dtype & 1)) return false;
    for (int i = 0; i < ndim; ++i)
        if (t->stride[i] < 0) return false;
    if (t->shape[ndim - 1] > 1 && t->stride[ndim - 1] != 1) return false;
    if (numel(t) == 0) return true;
    return t->data && reinterpret_cast<uintptr_t>(t->data) % elem_size(t->dtype) == 0;
}

// No two elements of an output share an address.
bool distinct(const dn_tensor* t) {
    if (numel(t) == 0) return true;
    int order[4];
    for (int i = 0; i < t->ndim; ++i) order[i] = i;
    std::sort(order, order + t->ndim, [&](int a, int b) { return t->stride[a] < t->stride[b]; });
    int64_t extent = 1;
    for (int i = 0; i < t->ndim; ++i) {
        const int o = order[i];
        if (t->shape[o] == 1) continue;
        if (t->stride[o] < extent) return false;
        extent += t->stride[o] * (t->shape[o] - 1);
    }
    return true;
}

// Rows side by side in one buffer: equal shapes and strides, and the two rows apart within
// the smallest row pitch, which divides the larger ones.
bool interleaved(const dn_tensor* a, const dn_tensor* b) {
    if (a->ndim != b->ndim || a->ndim < 2) return false;
    const int64_t es = elem_size(a->dtype);
    if (es != elem_size(b->dtype)) return false;
    int64_t pitch = 0;
    for (int i = 0; i < a->ndim; ++i) {
        if (a->shape[i] != b->shape[i]) return false;
        if (i == a->ndim - 1 || a->shape[i] == 1) continue;
        if (a->stride[i] != b->stride[i] || a->stride[i] < 1) return false;
        pitch = pitch ? std::min(pitch, a->stride[i]) : a->stride[i];
    }
    if (!pitch) return false;
    for (int i = 0; i + 1 < a->ndim; ++i)
        if (a->shape[i] > 1 && a->stride[i] % pitch) return false;
    const int64_t S = pitch * es, L = a->shape[a->ndim - 1] * es;
    int64_t off = (int64_t)(reinterpret_cast<uintptr_t>(b->data) - reinterpret_cast<uintptr_t>(a->data)) % S;
    if (off < 0) off += S;
    return off >= L && off + L <= S;
}

bool clash(const dn_tensor* a, const dn_tensor* b) { return overlap(a, b) && !interleaved(a, b); }

// DN_ERR_INVALID_ARG for an output whose own elements overlap, DN_ERR_ALIAS for one that
// overlaps an input or another output (null entries are skipped).
dn_status alias_check(std::initializer_list<const dn_tensor*> outs, std::initializer_list<const dn_tensor*> ins) {
    for (const dn_tensor* o : outs)
        if (o && !distinct(o)) return DN_ERR_INVALID_ARG;
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        if (!*o) continue;
        for (const dn_tensor* in : ins)
            if (in && clash(*o, in)) return DN_ERR_ALIAS;
        for (auto o2 = o + 1; o2 != outs.end(); ++o2)
            if (*o2 && clash(*o, *o2)) return DN_ERR_ALIAS;
    }
    return DN_OK;
}

bool index_ok(const dn_tensor* t, int64_t min_len) {
    return t->ndim == 1 && t->dtype == DN_I32 && t->shape[0] >= min_len &&
           (t->shape[0] <= 1 || t->stride[0] == 1) && (t->shape[0] == 0 || t->data) &&
           reinterpret_cast<uintptr_t>(t->data) % 4 == 0;
}

// [B, T, H] fp32 scalars per token and head, any non-negative strides.
bool scalars_ok(const dn_tensor* t, const int64_t* dims) {
    if (!shape_eq(t, 3, dims) || t->dtype != DN_F32) return false;
    for (int i = 0; i < 3; ++i)
        if (t->stride[i] < 0) return false;
    return numel(t) == 0 || (t->data && reinterpret_cast<uintptr_t>(t->data) % 4 == 0);
}

dn_status launched(int n) {
    if (cudaGetLastError() != cudaSuccess) return DN_ERR_CUDA;
    dn_note_launches(n);
    return DN_OK;
}

template <typename E, int DK, int DV>
void launch_step(const StepParams& p, int gate, unsigned grid, cudaStream_t s) {
    if (gate == 0) k_step<E, DK, DV, 0><<<grid, kStepThreads, 0, s>>>(p);
    else if (gate == 1) k_step<E, DK, DV, 1><<<grid, kStepThreads, 0, s>>>(p);
    else k_step<E, DK, DV, 2><<<grid, kStepThreads, 0, s>>>(p);
}

template <typename E>
void launch_step(const StepParams& p, int64_t dk, int64_t dv, int gate, unsigned grid, cudaStream_t s) {
    if (dk == 128 && dv == 128) launch_step<E, 128, 128>(p, gate, grid, s);
    else if (dk == 128) launch_step<E, 128, 64>(p, gate, grid, s);
    else if (dv == 128) launch_step<E, 64, 128>(p, gate, grid, s);
    else launch_step<E, 64, 64>(p, gate, grid, s);
}

// The state cache and slot indices of the step entry points; M rows.
dn_status cache_check(const dn_tensor* state, const dn_tensor* slots, int64_t N) {
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

// Shapes of deltanet_scan_fwd / _bwd: x [B, T, D] (x: its dtype and shape lead), g, the state
// tensors, the packed boundaries.  Sets N.
dn_status scan_shapes(const dn_tensor* x, const dn_tensor* g, const dn_tensor* cu, int64_t& N) {
    if (!x || !g || x->ndim != 3) return DN_ERR_INVALID_ARG;
    const int64_t B = x->shape[0], T = x->shape[1], D = x->shape[2];
    if (B < 0 || T < 0 || D < 1 || D > kMax31 || T > kMax31 || B > kMax31) return DN_ERR_INVALID_ARG;
    if (T > 0 && B > kMax31 / T) return DN_ERR_INVALID_ARG;
    if (T > kMax31 - 4096) return DN_ERR_INVALID_ARG;   // the kernels' token counters run past T by a few tiles
    const int64_t dims[3] = {B, T, D};
    if (!view_ok(x, 3, dims, kF32 | kBf16)) return DN_ERR_INVALID_ARG;
    if (!view_ok(g, 3, dims, x->dtype == DN_F32 ? kF32 : kF32 | kBf16)) return DN_ERR_INVALID_ARG;
    N = B;
    if (cu) {
        if (!index_ok(cu, 1) || B != 1) return DN_ERR_INVALID_ARG;
        N = cu->shape[0] - 1;
        if (N >= (int64_t(1) << 24)) return DN_ERR_INVALID_ARG;
    }
    if (N > 0 && (D + kScanThreads - 1) / kScanThreads > kMax31 / N) return DN_ERR_INVALID_ARG;
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
    // packed input reports its boundaries through the error word; without it only a wait
    // inside a cluster that gave up would, and a capture that finds none goes on without
    st = dn_stream_flag(dev, stream, &p.err);
    if (!cu) return DN_OK;
    p.cu = static_cast<const int*>(cu->data);
    return st;
}

// Pairs of channels can move as one access: even D, strides and addresses.
bool scan_pairs(const ScanParams& p, int32_t x, int32_t g, bool bwd) {
    auto ok = [](const void* a, int64_t sb, int64_t st, int32_t dt) {
        return reinterpret_cast<uintptr_t>(a) % (2 * elem_size(dt)) == 0 && sb % 2 == 0 && st % 2 == 0;
    };
    return p.D % 2 == 0 && ok(p.x, p.x_sb, p.x_st, x) && ok(p.g, p.g_sb, p.g_st, g) &&
           ok(p.y, p.y_sb, p.y_st, x) && (!bwd || (ok(p.h, p.h_sb, p.h_st, x) && ok(p.dg, p.dg_sb, p.dg_st, g)));
}

// CTAs per cluster: about one and a half CTAs on every SM, while each has tokens.  A cluster
// costs a start and an exchange per tile, idle SMs cost more: 64 channel tiles of 8192 tokens
// take 108, 72, 61 and 67 us with 1, 2, 4 and 8; 256 of 2048 tokens 52, 60, 68 and 90 us.
int scan_cluster(int64_t items, int64_t T, int tokens, int sms) {
    int K = 1;
    while (K < kScanMaxCluster && items * K < sms + sms / 2 && (int64_t)K * tokens < T) K *= 2;
    return K;
}

template <typename Kern, typename... A>
dn_status scan_launch(Kern* kern, int64_t items, int K, int threads, int smem, cudaStream_t stream,
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
    if (smem > 0 && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return DN_ERR_CUDA;
    return cudaLaunchKernelEx(&cfg, kern, p, K, a...) == cudaSuccess ? DN_OK : DN_ERR_CUDA;
}

constexpr int kScanTs = 8;         // tokens of a warp's run (one channel a lane)
constexpr int kScanSerialT = 32;   // up to so many tokens, one thread walks a channel

// 16-byte copies: bit 0 for x, 1 for g, 2 for h.
int scan_wide(const ScanParams& p, int32_t x, int32_t g) {
    auto ok = [](const void* a, int64_t sb, int64_t st, int32_t dt) {
        const int64_t es = elem_size(dt);
        return aligned16(a) && sb * es % 16 == 0 && st * es % 16 == 0;
    };
    return (ok(p.x, p.x_sb, p.x_st, x) ? 1 : 0) | (ok(p.g, p.g_sb, p.g_st, g) ? 2 : 0) |
           (p.h && ok(p.h, p.h_sb, p.h_st, x) ? 4 : 0);
}

template <typename X, typename G, int V, bool PACKED, bool BWD>
dn_status scan_tiled(const ScanParams& p, int sms, cudaStream_t stream) {
    const int64_t items = (int64_t)(PACKED ? 1 : p.B) * ((p.D + 32 * V - 1) / (32 * V));
    if constexpr (V == 2) {
        // tokens of a warp's run: as many as leave room for two CTAs on an SM
        constexpr int TS = sizeof(X) == 4 ? 4 : sizeof(G) == 2 && !BWD ? 16 : 8;
        constexpr int smem = (int)sizeof(ScanStage<X, G, TS, BWD>);
        const int K = scan_cluster(items, p.T, kScanWarps * TS, sms);
        const int wide = scan_wide(p, sizeof(X) == 4 ? DN_F32 : DN_BF16, sizeof(G) == 4 ? DN_F32 : DN_BF16);
        if (items > kMax31 / K) return DN_ERR_INVALID_ARG;
        auto go = [&](auto* kern) { return scan_launch(kern, items, K, kScanPipedThreads, smem, stream, p, wide); };
        if constexpr (BWD) return K > 1 ? go(k_scan_bwd_piped<X, G, TS, PACKED, true>) : go(k_scan_bwd_piped<X, G, TS, PACKED, false>);
        else return K > 1 ? go(k_scan_piped<X, G, TS, PACKED, true>) : go(k_scan_piped<X, G, TS, PACKED, false>);
    } else {
        const int K = scan_cluster(items, p.T, kScanWarps * kScanTs, sms);
        if (items > kMax31 / K) return DN_ERR_INVALID_ARG;
        if constexpr (BWD) return scan_launch(k_scan_bwd_tiled<X, G, V, kScanTs, PACKED>, items, K, kScanThreads, 0, stream, p);
        else return scan_launch(k_scan_tiled<X, G, V, kScanTs, PACKED>, items, K, kScanThreads, 0, stream, p);
    }
}

template <bool BWD>
dn_status scan_run(const ScanParams& p, int32_t x, int32_t g, cudaStream_t stream) {
    int dev = 0, sms = 0;
    dn_status st = dn_device_check(dev, sms);
    if (st != DN_OK) return st;
    by_types(x, g, [&](auto xt, auto gt) {
        using X = decltype(xt);
        using G = decltype(gt);
        if (p.T <= kScanSerialT) {
            const unsigned grid = (unsigned)((int64_t)p.N * ((p.D + kScanThreads - 1) / kScanThreads));
            if constexpr (BWD) k_scan_bwd_serial<X, G><<<grid, kScanThreads, 0, stream>>>(p);
            else k_scan_serial<X, G><<<grid, kScanThreads, 0, stream>>>(p);
        } else if (scan_pairs(p, x, g, BWD)) {
            st = p.cu ? scan_tiled<X, G, 2, true, BWD>(p, sms, stream) : scan_tiled<X, G, 2, false, BWD>(p, sms, stream);
        } else {
            st = p.cu ? scan_tiled<X, G, 1, true, BWD>(p, sms, stream) : scan_tiled<X, G, 1, false, BWD>(p, sms, stream);
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

bool param_ok(const dn_tensor* t, int64_t d, int dtypes) { return view_ok(t, 1, &d, dtypes); }

ParamVec param(const dn_tensor* t) {
    ParamVec v;
    v.p = t ? t->data : nullptr;
    v.bf16 = t && t->dtype == DN_BF16;
    return v;
}

RowRef row_ref(const dn_tensor* t) {
    RowRef r = {nullptr, 0, 0, 0};
    if (!t) return r;
    r.p = t->data;
    r.s0 = t->stride[0];
    r.s1 = t->ndim > 2 ? t->stride[1] : 0;
    r.s2 = t->ndim > 3 ? t->stride[2] : 0;
    return r;
}

// The arguments that deltanet_norm_fwd and _bwd share.
dn_status norm_check(const dn_tensor* y, const dn_tensor* w, const dn_tensor* gate, int act, const dn_tensor* res,
                     const dn_tensor* sc, const dn_tensor* nw, float eps, NormParams& p) {
    if (!y || y->ndim < 2 || y->ndim > 4) return DN_ERR_INVALID_ARG;
    if (!w && !gate && !res) return DN_ERR_INVALID_ARG;
    if ((sc || nw) && !res) return DN_ERR_INVALID_ARG;
    if (act != DN_ACT_SILU && act != DN_ACT_SIGMOID) return DN_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || std::isinf(eps)) return DN_ERR_INVALID_ARG;
    const int64_t d = y->shape[y->ndim - 1];
    int64_t rows = 1;
    if (d < 1) return DN_ERR_INVALID_ARG;
    for (int i = 0; i + 1 < y->ndim; ++i) {
        if (y->shape[i] < 0 || y->shape[i] > kMax31) return DN_ERR_INVALID_ARG;
        rows *= y->shape[i];
        if (rows > kMax31) return DN_ERR_INVALID_ARG;
    }
    if (!view_ok(y, y->ndim, y->shape, kF32 | kBf16)) return DN_ERR_INVALID_ARG;
    const int yt = 1 << y->dtype;
    if (gate && !view_ok(gate, y->ndim, y->shape, yt)) return DN_ERR_INVALID_ARG;
    if (res && !view_ok(res, y->ndim, y->shape, yt | kF32)) return DN_ERR_INVALID_ARG;
    for (const dn_tensor* t : {w, sc, nw})
        if (t && !param_ok(t, d, kF32 | kBf16)) return DN_ERR_INVALID_ARG;
    if (d > kNormMaxD) return DN_ERR_UNSUPPORTED;
    std::memset(&p, 0, sizeof p);
    p.y = row_ref(y);
    p.gate = row_ref(gate);
    p.res = row_ref(res);
    p.w = param(w);
    p.sc = param(sc);
    p.nw = param(nw);
    p.act = act;
    p.eps = eps;
    p.rows = rows;
    p.d = (int)d;
    p.n1 = y->ndim > 2 ? (unsigned)y->shape[1] : 1;
    p.n2 = y->ndim > 3 ? (unsigned)y->shape[2] : 1;
    return DN_OK;
}

// Kernel choice by the dtypes of y and the residual: f(Y(), R()).
template <typename F>
void by_row_types(const dn_tensor* y, const dn_tensor* res, F f) {
    if (y->dtype == DN_F32) f(float(), float());
    else if (res && res->dtype == DN_F32) f(__nv_bfloat16(), float());
    else f(__nv_bfloat16(), __nv_bfloat16());
}

int norm_bwd_ctas(int64_t rows) { return (int)std::min<int64_t>(rows, kNormBwdCtas); }

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
    const unsigned grid = (unsigned)(N * ((D + kScanThreads - 1) / kScanThreads));
    by_types(x->dtype, g->dtype, [&](auto xt, auto gt) {
        k_scan_step<decltype(xt), decltype(gt)><<<grid, kScanThreads, 0, stream>>>(p);
    });
    return launched(1);
}

dn_status deltanet_norm_fwd(const dn_tensor* y, const dn_tensor* weight, const dn_tensor* gate, int activation,
                            const dn_tensor* residual, const dn_tensor* scale, const dn_tensor* next_weight,
                            float eps, dn_tensor* out, dn_tensor* residual_out, void* stream_ptr) {
    NormParams p;
    dn_status st = norm_check(y, weight, gate, activation, residual, scale, next_weight, eps, p);
    if (st != DN_OK) return st;
    if ((out != nullptr) != (!residual || next_weight) || (residual_out != nullptr) != (residual != nullptr))
        return DN_ERR_INVALID_ARG;
    if (out && !view_ok(out, y->ndim, y->shape, 1 << y->dtype)) return DN_ERR_INVALID_ARG;
    if (residual && !view_ok(residual_out, y->ndim, y->shape, 1 << residual->dtype)) return DN_ERR_INVALID_ARG;
    if ((st = alias_check({out, residual_out}, {y, weight, gate, residual, scale, next_weight})) != DN_OK) return st;
    int dev = 0, sms = 0;
    if ((st = dn_device_check(dev, sms)) != DN_OK) return st;
    if (p.rows == 0) return DN_OK;
    p.out = row_ref(out);
    p.rout = row_ref(residual_out);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    by_row_types(y, residual, [&](auto yt, auto rt) {
        k_norm_fwd<decltype(yt), decltype(rt)><<<(unsigned)p.rows, kNormThreads, 0, stream>>>(p);
    });
    return launched(1);
}

int64_t deltanet_norm_workspace(int64_t rows, int64_t d) {
    return rows > 0 && d > 0 ? (int64_t)norm_bwd_ctas(rows) * 3 * d : 0;
}

dn_status deltanet_norm_bwd(const dn_tensor* y, const dn_tensor* weight, const dn_tensor* gate, int activation,
                            const dn_tensor* residual, const dn_tensor* scale, const dn_tensor* next_weight,
                            float eps, const dn_tensor* d_out, const dn_tensor* d_residual_out, dn_tensor* d_y,
                            dn_tensor* d_weight, dn_tensor* d_gate, dn_tensor* d_residual, dn_tensor* d_scale,
                            dn_tensor* d_next_weight, dn_tensor* workspace, void* stream_ptr) {
    NormParams p;
    dn_status st = norm_check(y, weight, gate, activation, residual, scale, next_weight, eps, p);
    if (st != DN_OK) return st;
    const int nd = y->ndim, yt = 1 << y->dtype, rt = residual ? 1 << residual->dtype : 0;
    const int64_t d = p.d;
    if ((d_out != nullptr) != (!residual || next_weight)) return DN_ERR_INVALID_ARG;
    if (d_residual_out ? !residual : residual && !next_weight) return DN_ERR_INVALID_ARG;
    if (d_out && !view_ok(d_out, nd, y->shape, yt)) return DN_ERR_INVALID_ARG;
    if (d_residual_out && !view_ok(d_residual_out, nd, y->shape, rt)) return DN_ERR_INVALID_ARG;
    if (!d_y || !view_ok(d_y, nd, y->shape, yt)) return DN_ERR_INVALID_ARG;
    if ((d_gate != nullptr) != (gate != nullptr) || (d_residual != nullptr) != (residual != nullptr))
        return DN_ERR_INVALID_ARG;
    if (d_gate && !view_ok(d_gate, nd, y->shape, yt)) return DN_ERR_INVALID_ARG;
    if (d_residual && !view_ok(d_residual, nd, y->shape, rt)) return DN_ERR_INVALID_ARG;
    const dn_tensor* params[3] = {weight, scale, next_weight};
    const dn_tensor* grads[3] = {d_weight, d_scale, d_next_weight};
    bool sums = false;
    for (int i = 0; i < 3; ++i) {
        if ((params[i] != nullptr) != (grads[i] != nullptr)) return DN_ERR_INVALID_ARG;
        if (grads[i] && !param_ok(grads[i], d, kF32)) return DN_ERR_INVALID_ARG;
        sums |= grads[i] != nullptr;
    }
    const int64_t need = sums ? deltanet_norm_workspace(p.rows, d) : 0;
    if (need > 0 && (!workspace || workspace->ndim != 1 || workspace->dtype != DN_F32 || !workspace->data ||
                     workspace->stride[0] != 1 || !aligned16(workspace->data)))
        return DN_ERR_INVALID_ARG;
    if (need > 0 && workspace->shape[0] < need) return DN_ERR_WORKSPACE;
    if ((st = alias_check({d_y, d_gate, d_residual, d_weight, d_scale, d_next_weight, need > 0 ? workspace : nullptr},
                          {y, weight, gate, residual, scale, next_weight, d_out, d_residual_out})) != DN_OK)
        return st;
    int dev = 0, sms = 0;
    if ((st = dn_device_check(dev, sms)) != DN_OK) return st;
    p.dout = row_ref(d_out);
    p.drout = row_ref(d_residual_out);
    p.dy = row_ref(d_y);
    p.dgate = row_ref(d_gate);
    p.dres = row_ref(d_residual);
    p.part = need > 0 ? static_cast<float*>(workspace->data) : nullptr;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    const int ctas = norm_bwd_ctas(p.rows);
    int launches = 0;
    if (p.rows > 0) {
        const int smem = (int)(3 * d * sizeof(float));
        bool ok = true;
        by_row_types(y, residual, [&](auto yt, auto rt) {
            auto* kern = k_norm_bwd<decltype(yt), decltype(rt)>;
            ok = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * kNormMaxD * 4) ==
                 cudaSuccess;
            if (ok) kern<<<ctas, kNormThreads, smem, stream>>>(p);
        });
        if (!ok) return DN_ERR_CUDA;
        ++launches;
    }
    if (sums) {
        auto f = [](dn_tensor* t) { return t ? static_cast<float*>(t->data) : nullptr; };
        k_norm_bwd_sum<<<dim3((unsigned)((d + 31) / 32), 3), 256, 0, stream>>>(
            p.part, ctas, (int)d, f(d_weight), f(d_scale), f(d_next_weight));
        ++launches;
    }
    return launched(launches);
}

}  // extern "C"
