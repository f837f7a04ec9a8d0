// Host side of deltanet_norm_fwd and deltanet_norm_bwd (include/deltanet.h): argument checks
// and launches only.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "../../include/deltanet.h"
#include "dn_host.h"
#include "dn_norm.cuh"

using namespace dn;

namespace {

bool param_ok(const dn_tensor* t, int64_t d, int dtypes) { return view_ok(t, 1, &d, dtypes); }

ParamVec param(const dn_tensor* t) {
    ParamVec v;
    v.p = t ? t->data : nullptr;
    v.bf16 = t && t->dtype == DN_BF16;
    v.vec = t && aligned16(t->data);
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

// Row dimensions that lie behind one another in every tensor become one.
void norm_collapse(NormParams& p) {
    RowRef* refs[] = {&p.y, &p.gate, &p.res, &p.out, &p.rout, &p.dout, &p.drout, &p.dy, &p.dgate, &p.dres};
    bool in = true, out = true;
    for (const RowRef* r : refs)
        if (r->p) in = in && r->s1 == r->s2 * p.n2;
    if (p.n2 > 1 && in) {                // (i1, i2) -> i1 of n1 * n2
        for (RowRef* r : refs) r->s1 = r->s2;
        p.n1 *= p.n2;
        p.n2 = 1;
    }
    for (const RowRef* r : refs)
        if (r->p) out = out && r->s0 == r->s1 * p.n1;
    if (p.n1 > 1 && p.n2 == 1 && out) {  // (i0, i1) -> i0
        for (RowRef* r : refs) r->s0 = r->s1;
        p.n1 = 1;
    }
}

// Whether every tensor has y's row strides.
bool norm_same(const NormParams& p) {
    const RowRef* refs[] = {&p.gate, &p.res, &p.out, &p.rout, &p.dout, &p.drout, &p.dy, &p.dgate, &p.dres};
    for (const RowRef* r : refs)
        if (r->p && (r->s0 != p.y.s0 || (p.n1 > 1 && r->s1 != p.y.s1) || (p.n2 > 1 && r->s2 != p.y.s2))) return false;
    return true;
}

// Every row of every tensor starts on 16 bytes.
bool norm_wide(const NormParams& p, int ysize, int rsize) {
    const RowRef* ys[] = {&p.y, &p.gate, &p.out, &p.dout, &p.dy, &p.dgate};
    const RowRef* rs[] = {&p.res, &p.rout, &p.drout, &p.dres};
    auto ok = [](const RowRef* r, int es) {
        return !r->p || (aligned16(r->p) && r->s0 * es % 16 == 0 && r->s1 * es % 16 == 0 && r->s2 * es % 16 == 0);
    };
    bool w = p.d % 8 == 0;
    for (const RowRef* r : ys) w = w && ok(r, ysize);
    for (const RowRef* r : rs) w = w && ok(r, rsize);
    return w;
}

// Every tensor itself does.
int norm_line(const NormParams& p) {
    const RowRef* refs[] = {&p.y, &p.gate, &p.res, &p.dout, &p.drout};
    for (const RowRef* r : refs)
        if (r->p && !aligned16(r->p)) return 0;
    return 1;
}

// Threads of a row by its length: f(integral_constant<TPR>, bool_constant<VEC>,
// bool_constant<SAME>); false past the longest row that is held in registers.
template <int TPR, bool VEC, bool SAME, typename F>
bool norm_try(int d, F& f) {
    if (d > (TPR <= 1 ? kNormCta<TPR> : TPR) * 8) return false;
    f(std::integral_constant<int, TPR>(), std::bool_constant<VEC>(), std::bool_constant<SAME>());
    return true;
}
template <bool SAME, typename F>
bool norm_by_length(int d, F& f) {
    return norm_try<8, true, SAME>(d, f) || norm_try<16, true, SAME>(d, f) || norm_try<32, true, SAME>(d, f) ||
           norm_try<128, true, SAME>(d, f) || norm_try<256, true, SAME>(d, f) || norm_try<512, true, SAME>(d, f);
}
template <typename F>
bool norm_by_length(const NormParams& p, bool wide, F f) {
    if (wide) return norm_same(p) ? norm_by_length<true>(p.d, f) : norm_by_length<false>(p.d, f);
    return norm_try<32, false, false>(p.d, f) || norm_try<0, false, false>(p.d, f) || norm_try<1, false, false>(p.d, f);
}

// More than 48 KB of shared memory has to be asked for: the same limit in every call (calls on
// several host threads share the kernel's attribute), above what any of them needs.
constexpr int kNormSmem = 217 * 1024;
template <typename Kern>
bool norm_smem(Kern* kern, int bytes) {
    return bytes <= 32768 ||
           (bytes <= kNormSmem &&
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem) == cudaSuccess);
}

// CTAs of a kernel that the GPU holds at once (they walk the rows, so more would only queue).
template <typename Kern>
int norm_resident(Kern* kern, int threads, int smem, int sms) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem) != cudaSuccess || n < 1) n = 1;
    return n * sms;
}

template <typename Y, typename R, bool RES>
dn_status norm_fwd_run(const NormParams& p, bool wide, int sms, cudaStream_t stream) {
    bool ok = true;
    const bool done = norm_by_length(p, wide, [&](auto tpr, auto vec, auto same) {
        constexpr int TPR = decltype(tpr)::value, CTA = kNormCta<TPR>, ROWS = TPR <= 1 ? 1 : CTA / TPR;
        const int TH = TPR <= 1 ? (p.d + 255) / 256 * 32 : CTA;
        constexpr bool VEC = decltype(vec)::value;
        const int64_t need = (p.rows + ROWS - 1) / ROWS;
        // without 16-byte rows: two places for the lines of a row of each operand
        const int smem = VEC ? 2 * NormPlan<Y, R, RES, false>::all * CTA * 16
                       : p.line ? 2 * ROWS * 16 * (2 * line_pieces<Y>(p.d) + (RES ? line_pieces<R>(p.d) : 0)) : 0;
        auto* kern = k_norm_fwd_rows<Y, R, TPR, VEC, RES, decltype(same)::value>;
        if (!(ok = norm_smem(kern, smem))) return;
        const int64_t grid = need > sms ? std::min<int64_t>(need, norm_resident(kern, TH, smem, sms)) : need;
        kern<<<(unsigned)grid, TH, smem, stream>>>(p);
    });
    if (!done) {
        auto* kern = wide ? k_norm_fwd_long<Y, R, true> : k_norm_fwd_long<Y, R, false>;
        kern<<<(unsigned)std::min<int64_t>(p.rows, 4 * sms), kNormLong, 0, stream>>>(p);
    }
    return ok ? launched(1) : DN_ERR_CUDA;
}

template <typename Y, typename R, bool RES>
dn_status norm_bwd_run(const NormParams& p, bool wide, int sms, int& ctas, cudaStream_t stream) {
    bool ok = true;
    const bool done = norm_by_length(p, wide, [&](auto tpr, auto vec, auto same) {
        constexpr int TPR = decltype(tpr)::value, CTA = kNormCta<TPR>, ROWS = TPR <= 1 ? 1 : CTA / TPR;
        const int TH = TPR <= 1 ? (p.d + 255) / 256 * 32 : CTA;
        constexpr bool VEC = decltype(vec)::value;
        const int smem = (RES ? 6 : 2) * CTA * 16 +
                         (VEC ? 2 * NormPlan<Y, R, RES, true>::all * CTA * 16
                              : p.line ? 2 * ROWS * 16 * (3 * line_pieces<Y>(p.d) + (RES ? 2 * line_pieces<R>(p.d) : 0)) : 0);
        auto* kern = k_norm_bwd_rows<Y, R, TPR, VEC, RES, decltype(same)::value>;
        if (!(ok = norm_smem(kern, smem))) return;
        ctas = (int)std::min<int64_t>(ctas, (p.rows + ROWS - 1) / ROWS);
        if (ctas > sms) ctas = std::min(ctas, norm_resident(kern, TH, smem, sms));
        kern<<<ctas, TH, smem, stream>>>(p);
    });
    if (!done) {
        auto* kern = wide ? k_norm_bwd_long<Y, R, true> : k_norm_bwd_long<Y, R, false>;
        const int smem = 3 * ((p.d + kNormLong * 8 - 1) / (kNormLong * 8)) * kNormLong * 8 * (int)sizeof(float);
        if ((ok = norm_smem(kern, smem))) {
            ctas = std::min(ctas, norm_resident(kern, kNormLong, smem, sms));
            kern<<<ctas, kNormLong, smem, stream>>>(p);
        }
    }
    return ok ? DN_OK : DN_ERR_CUDA;
}

// Kernel choice by types and by whether there is a residual: f(Y(), R(), bool_constant).
template <typename F>
dn_status norm_by_case(const dn_tensor* y, const dn_tensor* res, F f) {
    dn_status st = DN_OK;
    by_row_types(y, res, [&](auto yt, auto rt) {
        if (res) st = f(yt, rt, std::true_type());
        else if constexpr (std::is_same<decltype(yt), decltype(rt)>::value) st = f(yt, rt, std::false_type());
    });
    return st;
}

int norm_bwd_ctas(int64_t rows) { return (int)std::min<int64_t>(rows, kNormBwdCtas); }

}  // namespace

extern "C" {

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
    const bool wide = norm_wide(p, (int)elem_size(y->dtype), residual ? (int)elem_size(residual->dtype) : 4);
    norm_collapse(p);
    p.line = norm_line(p);
    return norm_by_case(y, residual, [&](auto yt, auto rt, auto has) {
        return norm_fwd_run<decltype(yt), decltype(rt), decltype(has)::value>(p, wide, sms, stream);
    });
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
    int ctas = norm_bwd_ctas(p.rows);
    int launches = 0;
    if (p.rows > 0) {
        const bool wide = norm_wide(p, (int)elem_size(y->dtype), residual ? (int)elem_size(residual->dtype) : 4);
        norm_collapse(p);
        p.line = norm_line(p);
        st = norm_by_case(y, residual, [&](auto yt, auto rt, auto has) {
            return norm_bwd_run<decltype(yt), decltype(rt), decltype(has)::value>(p, wide, sms, ctas, stream);
        });
        if (st != DN_OK) return st;
        ++launches;
    }
    if (sums) {
        auto f = [](dn_tensor* t) { return t ? static_cast<float*>(t->data) : nullptr; };
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((d + 31) / 32), 3);
        cfg.blockDim = dim3(32 * kNormSumGroups);
        cfg.stream = stream;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &at;
        cfg.numAttrs = p.rows > 0;
        if (cudaLaunchKernelEx(&cfg, k_norm_bwd_sum, (const float*)p.part, ctas, (int)d, f(d_weight), f(d_scale),
                               f(d_next_weight)) != cudaSuccess)
            return DN_ERR_CUDA;
        ++launches;
    }
    return launched(launches);
}

}  // extern "C"
