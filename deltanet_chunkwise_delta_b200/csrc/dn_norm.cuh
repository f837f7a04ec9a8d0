// deltanet_norm_fwd / _bwd: the norms before and after a block with its gate, residual
// scale and residual sum, and their gradients.
//
// Row by row, d elements each:
//   y1 = y rstd1 weight, y2 = y1 act(gate), r' = residual + scale y2, n = r' rstd2 next_weight
// with rstd = rsqrt(mean(.^2) + eps).  Backward, with mean over the row:
//   dr' = d_residual_out + rstd2 (dn next_weight - r' rstd2^2 mean(dn next_weight r'))
//   d_residual = dr', d_scale = sum dr' y2, dy2 = scale dr'
//   d_gate = dy2 y1 act'(gate), dy1 = dy2 act(gate)
//   d_weight = sum dy1 y rstd1, d_next_weight = sum dn r' rstd2
//   d_y = rstd1 (dy1 weight - y rstd1^2 mean(dy1 weight y))
#pragma once

#include "dn_common.cuh"
#include "dn_vec.cuh"

namespace dn {

constexpr int kNormThreads = 256;
constexpr int kNormMaxD = 16384;
constexpr int kNormBwdCtas = 296;      // most CTAs of the backward kernel (partial sums kept)

// A row tensor: element strides of up to three row dimensions (see NormParams::n1, n2).
struct RowRef {
    const void* p;
    int64_t s0, s1, s2;
};

struct NormParams {
    RowRef y, gate, res, out, rout;    // out / rout are written by the forward kernel
    RowRef dout, drout;                // backward inputs
    RowRef dy, dgate, dres;            // backward outputs
    ParamVec w, sc, nw;
    float* part;                       // backward: [CTAs][3][d] partial sums
    int act;
    float eps;
    int64_t rows;
    unsigned n1, n2;                   // row = (i0 * n1 + i1) * n2 + i2
    int d;
};

template <typename E>
__device__ __forceinline__ E* row_ptr(const RowRef& r, unsigned i0, unsigned i1, unsigned i2) {
    return static_cast<E*>(const_cast<void*>(r.p)) + i0 * r.s0 + i1 * r.s1 + i2 * r.s2;
}

// act(z) and act'(z)
__device__ __forceinline__ float norm_act(float z, int act, float* grad = nullptr) {
    const float s = 1.f / (1.f + expf(-z));
    if (act == 1) {
        if (grad) *grad = s * (1.f - s);
        return s;
    }
    if (grad) *grad = s * (1.f + z * (1.f - s));
    return z * s;
}

// Sum over the CTA (same order on every thread and every call).
__device__ __forceinline__ float cta_sum(float x, float* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += sh[w];
    return s;
}

template <typename Y, typename R>
__global__ void __launch_bounds__(kNormThreads) k_norm_fwd(NormParams p) {
    __shared__ float sh[kNormThreads / 32];
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const unsigned u = (unsigned)row, i2 = u % p.n2, i1 = u / p.n2 % p.n1, i0 = u / p.n2 / p.n1;
        const Y* y = row_ptr<const Y>(p.y, i0, i1, i2);
        const Y* z = p.gate.p ? row_ptr<const Y>(p.gate, i0, i1, i2) : nullptr;
        const R* r = p.res.p ? row_ptr<const R>(p.res, i0, i1, i2) : nullptr;
        float rstd1 = 1.f, rstd2 = 1.f;
        if (p.w.p) {
            float q = 0.f;
            for (int j = threadIdx.x; j < p.d; j += kNormThreads) {
                const float v = ld_elem(y + j);
                q = fmaf(v, v, q);
            }
            rstd1 = rsqrtf(cta_sum(q, sh) / p.d + p.eps);
        }
        auto chain = [&](int j) {      // y2, or r' with a residual
            float v = ld_elem(y + j);
            if (p.w.p) v = v * rstd1 * ld_param(p.w, j);
            if (z) v *= norm_act(ld_elem(z + j), p.act);
            if (r) v = ld_elem(r + j) + (p.sc.p ? ld_param(p.sc, j) * v : v);
            return v;
        };
        if (p.nw.p) {
            float q = 0.f;
            for (int j = threadIdx.x; j < p.d; j += kNormThreads) {
                const float v = chain(j);
                q = fmaf(v, v, q);
            }
            rstd2 = rsqrtf(cta_sum(q, sh) / p.d + p.eps);
        }
        Y* out = p.out.p ? row_ptr<Y>(p.out, i0, i1, i2) : nullptr;
        R* rout = p.rout.p ? row_ptr<R>(p.rout, i0, i1, i2) : nullptr;
        for (int j = threadIdx.x; j < p.d; j += kNormThreads) {
            const float v = chain(j);
            if (rout) st_elem(rout + j, v);
            if (out) st_elem(out + j, p.nw.p ? v * rstd2 * ld_param(p.nw, j) : v);
        }
    }
}

template <typename Y, typename R>
__global__ void __launch_bounds__(kNormThreads) k_norm_bwd(NormParams p) {
    __shared__ float sh[kNormThreads / 32];
    extern __shared__ float acc[];     // [3][d]: sums for weight, scale, next_weight
    const int d = p.d;
    for (int j = threadIdx.x; j < 3 * d; j += kNormThreads) acc[j] = 0.f;
    __syncthreads();
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const unsigned u = (unsigned)row, i2 = u % p.n2, i1 = u / p.n2 % p.n1, i0 = u / p.n2 / p.n1;
        const Y* y = row_ptr<const Y>(p.y, i0, i1, i2);
        const Y* z = p.gate.p ? row_ptr<const Y>(p.gate, i0, i1, i2) : nullptr;
        const R* r = p.res.p ? row_ptr<const R>(p.res, i0, i1, i2) : nullptr;
        const Y* dout = p.dout.p ? row_ptr<const Y>(p.dout, i0, i1, i2) : nullptr;
        const R* drout = p.drout.p ? row_ptr<const R>(p.drout, i0, i1, i2) : nullptr;
        float rstd1 = 1.f, rstd2 = 1.f, m2 = 0.f, m1 = 0.f;
        if (p.w.p) {
            float q = 0.f;
            for (int j = threadIdx.x; j < d; j += kNormThreads) {
                const float v = ld_elem(y + j);
                q = fmaf(v, v, q);
            }
            rstd1 = rsqrtf(cta_sum(q, sh) / d + p.eps);
        }
        struct Elem { float y, y1, y2, a, da, r; };
        auto chain = [&](int j) {
            Elem e;
            e.y = ld_elem(y + j);
            e.y1 = p.w.p ? e.y * rstd1 * ld_param(p.w, j) : e.y;
            e.a = 1.f;
            e.da = 0.f;
            if (z) e.a = norm_act(ld_elem(z + j), p.act, &e.da);
            e.y2 = e.y1 * e.a;
            e.r = r ? ld_elem(r + j) + (p.sc.p ? ld_param(p.sc, j) * e.y2 : e.y2) : 0.f;
            return e;
        };
        if (p.nw.p) {
            float q = 0.f, c = 0.f;
            for (int j = threadIdx.x; j < d; j += kNormThreads) {
                const Elem e = chain(j);
                q = fmaf(e.r, e.r, q);
                c = fmaf(ld_elem(dout + j) * ld_param(p.nw, j), e.r, c);
            }
            rstd2 = rsqrtf(cta_sum(q, sh) / d + p.eps);
            m2 = cta_sum(c, sh) / d * rstd2 * rstd2;
        }
        // gradient of y2 before the residual scale (of r' with a residual)
        auto top = [&](int j, const Elem& e) {
            if (!r) return ld_elem(dout + j);
            float dr = drout ? ld_elem(drout + j) : 0.f;
            if (p.nw.p) dr += rstd2 * (ld_elem(dout + j) * ld_param(p.nw, j) - e.r * m2);
            return dr;
        };
        if (p.w.p) {
            float c = 0.f;
            for (int j = threadIdx.x; j < d; j += kNormThreads) {
                const Elem e = chain(j);
                float dv = top(j, e);
                if (p.sc.p) dv *= ld_param(p.sc, j);
                c = fmaf(dv * e.a * ld_param(p.w, j), e.y, c);
            }
            m1 = cta_sum(c, sh) / d * rstd1 * rstd1;
        }
        for (int j = threadIdx.x; j < d; j += kNormThreads) {
            const Elem e = chain(j);
            float dv = top(j, e);
            if (p.nw.p) acc[2 * d + j] += ld_elem(dout + j) * e.r * rstd2;
            if (r) st_elem(row_ptr<R>(p.dres, i0, i1, i2) + j, dv);
            if (p.sc.p) {
                acc[d + j] += dv * e.y2;
                dv *= ld_param(p.sc, j);
            }
            if (z) st_elem(row_ptr<Y>(p.dgate, i0, i1, i2) + j, dv * e.y1 * e.da);
            dv *= e.a;
            if (p.w.p) {
                acc[j] += dv * e.y * rstd1;
                dv = rstd1 * (dv * ld_param(p.w, j) - e.y * m1);
            }
            st_elem(row_ptr<Y>(p.dy, i0, i1, i2) + j, dv);
        }
    }
    if (!p.part) return;
    __syncthreads();
    float* part = p.part + (int64_t)blockIdx.x * 3 * d;
    for (int j = threadIdx.x; j < 3 * d; j += kNormThreads) part[j] = acc[j];
}

// d_weight, d_scale, d_next_weight from the partial sums of G CTAs: 32 columns per CTA, 8
// groups of partials each added in order, then the groups in order.
__global__ void __launch_bounds__(256) k_norm_bwd_sum(const float* part, int G, int d, float* dw,
                                                      float* ds, float* dn) {
    __shared__ float sh[8][32];
    float* out = blockIdx.y == 0 ? dw : blockIdx.y == 1 ? ds : dn;
    if (!out) return;
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5, j = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (j < d)
        for (int i = grp; i < G; i += 8) s += part[((int64_t)i * 3 + blockIdx.y) * d + j];
    sh[grp][lane] = s;
    __syncthreads();
    if (grp == 0 && j < d) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += sh[i][lane];
        out[j] = t;
    }
}

}  // namespace dn
