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
constexpr int kNormBwdCtas = 444;      // most CTAs of the backward kernels (partial sums kept)

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
    int line;                          // without 16-byte rows: every tensor starts on 16 bytes
};

// On pairs of the 8 elements of a thread: one instruction for two.
__device__ __forceinline__ void mul8(const float* a, const float* b, float* d) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) mul2(a + e, b + e, d + e);
}
__device__ __forceinline__ void mul8(const float* a, float b, float* d) {
    const float bb[2] = {b, b};
#pragma unroll
    for (int e = 0; e < 8; e += 2) mul2(a + e, bb, d + e);
}
__device__ __forceinline__ void fma8(const float* a, const float* b, const float* c, float* d) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) fma2(a + e, b + e, c + e, d + e);
}
__device__ __forceinline__ void fma8(const float* a, float b, const float* c, float* d) {
    const float bb[2] = {b, b};
#pragma unroll
    for (int e = 0; e < 8; e += 2) fma2(a + e, bb, c + e, d + e);
}
// sum of a b
__device__ __forceinline__ float dot8(const float* a, const float* b) {
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 8; e += 2) fma2(a + e, b + e, s, s);
    return s[0] + s[1];
}

template <typename E>
__device__ __forceinline__ E* row_ptr(const RowRef& r, unsigned i0, unsigned i1, unsigned i2) {
    return static_cast<E*>(const_cast<void*>(r.p)) + i0 * r.s0 + i1 * r.s1 + i2 * r.s2;
}

// act(z) and act'(z) from s = 1 / (1 + e^-z): the hardware's 2^x and 1/x, a few ulp each and
// what |z| ulp the exponential adds.  Far out e^-z is inf or 0 and s is 0 or 1.  1 - s is e^-z s:
// the difference has no figures left where s is near 1 (none at z = 17), and the sigmoid's
// derivative s (1 - s) would have none.
__device__ __forceinline__ float norm_act(float z, int act, float* grad = nullptr) {
    const float e = __expf(-z), s = __fdividef(1.f, 1.f + e);
    const float rest = __saturatef(e * s);             // 1 - s; at s = 0 0 as well, not inf times 0
    if (act == 1) {
        if (grad) *grad = s * rest;
        return s;
    }
    if (grad) *grad = s * (1.f + z * rest);
    return z * s;
}

// ---- rows that fit a group of threads, 8 elements each -----------------------------------
//
// TPR threads hold a row in registers (8, 16 or 32 of a warp, or a whole CTA): every element is
// read and written once, the sums over the row go through shuffles and, for a CTA, one barrier
// each.  CTAs stay and walk the rows; with 16-byte rows (VEC) the next row is on its way
// (cp.async, each thread its own pieces, no barrier) while one is worked on.  Without, a
// thread's elements lie TPR apart, TPR 0 and 1 take the CTA's size, the row's length over 8
// (up to 320 and 512 threads), and rows come through shared memory in the 16-byte pieces that
// they lie in (`line`; one barrier more a row) where the tensors themselves start on one:
// 16384 rows of 2049 bf16 elements forward with gate and residual 151 us, 250 read one by one.
//
// B200, 16384 rows of 2048: residual sum and next norm 66 us (93 % of the measured copy rate),
// the whole chain backward 118 us (69 %: 55 % of the issue slots in use, all that the warps of
// two CTAs give); 262144 heads of 128: gated norm 37 us (83 %), backward 60 us (85 %).

template <int TPR>
constexpr int kNormCta = TPR == 0 ? 320 : TPR == 1 ? 512 : TPR <= 32 ? kNormThreads : TPR;
template <int TPR>
__device__ __forceinline__ int norm_tpr() { return TPR <= 1 ? (int)blockDim.x : TPR; }

// The sums of N values over the row's threads, on all of them; `turn` alternates between calls.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float* v, float (*sh)[2][32], int& turn) {
#pragma unroll
    for (int o = (TPR > 1 && TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(~0u, v[n], o);
    if constexpr (TPR <= 1 || TPR > 32) {
        const int W = norm_tpr<TPR>() / 32;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) sh[turn][n][threadIdx.x >> 5] = v[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = 0.f;
            if constexpr (TPR > 1 && TPR <= 256) {
#pragma unroll
                for (int w = 0; w < TPR / 32; ++w) s += sh[turn][n][w];
            } else {
                s = (threadIdx.x & 31) < W ? sh[turn][n][threadIdx.x & 31] : 0.f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
            }
            v[n] = s;
        }
        turn ^= 1;
    }
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}

__device__ __forceinline__ void cp_async8(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}

// A thread's 8 elements of a row.  VEC: 8 neighbours (all bf16: 16 bytes), or, where fp32 takes
// part (SPLIT), two times 4 neighbours 4 TPR apart, so that a warp's accesses stay contiguous
// (8 neighbours of fp32 would move in 16-byte halves of 32-byte pieces: half of each sector
// per access; the residual case went from 87 to 71 us with this).  Without VEC: 8 elements TPR
// apart.
template <typename E, int TPR, bool VEC, bool SPLIT>
struct RowPart {
    static constexpr int kPieces = sizeof(E) / 2;      // of 16 bytes in shared memory
    __device__ static __forceinline__ int col(int l, int e) {
        return !VEC ? e * norm_tpr<TPR>() + l : !SPLIT ? l * 8 + e : (e >> 2) * TPR * 4 + l * 4 + (e & 3);
    }
    __device__ static __forceinline__ void unpack16(const uint4* q, float* f) {
        if constexpr (sizeof(E) == 2) {
            const uint32_t u[4] = {q->x, q->y, q->z, q->w};
#pragma unroll
            for (int i = 0; i < 4; ++i) unpack(u[i], f + 2 * i);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[4 * i] = __uint_as_float(q[i].x);
                f[4 * i + 1] = __uint_as_float(q[i].y);
                f[4 * i + 2] = __uint_as_float(q[i].z);
                f[4 * i + 3] = __uint_as_float(q[i].w);
            }
        }
    }
    __device__ static __forceinline__ void load(const E* row, int l, int d, float* f) {
        if constexpr (VEC) {
            uint4 q[kPieces] = {};
            if constexpr (!SPLIT) {
                if (l * 8 < d)
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) q[i] = __ldg(reinterpret_cast<const uint4*>(row + l * 8) + i);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (col(l, 4 * h) < d) {
                        if constexpr (sizeof(E) == 4) {
                            q[h] = __ldg(reinterpret_cast<const uint4*>(row + col(l, 4 * h)));
                        } else {
                            const uint2 u = __ldg(reinterpret_cast<const uint2*>(row + col(l, 4 * h)));
                            if (h == 0) q[0].x = u.x, q[0].y = u.y;
                            else q[0].z = u.x, q[0].w = u.y;
                        }
                    }
            }
            unpack16(q, f);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = col(l, e) < d ? ld_elem(row + col(l, e)) : 0.f;
        }
    }
    __device__ static __forceinline__ void store(E* row, int l, int d, const float* f) {
        if constexpr (VEC && sizeof(E) == 2) {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) pack(f + 2 * i, u[i]);
            if constexpr (!SPLIT) {
                if (l * 8 < d) *reinterpret_cast<uint4*>(row + l * 8) = make_uint4(u[0], u[1], u[2], u[3]);
            } else {
                if (col(l, 0) < d) *reinterpret_cast<uint2*>(row + col(l, 0)) = make_uint2(u[0], u[1]);
                if (col(l, 4) < d) *reinterpret_cast<uint2*>(row + col(l, 4)) = make_uint2(u[2], u[3]);
            }
        } else if constexpr (VEC) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (col(l, 4 * h) < d)
                    *reinterpret_cast<float4*>(row + col(l, 4 * h)) =
                        make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col(l, e) < d) st_elem(row + col(l, e), f[e]);
        }
    }
    // this thread's pieces into shared memory (16 bytes a thread side by side), and from there
    __device__ static __forceinline__ void fetch(const E* row, int l, int d, uint4* place) {
        if constexpr (!SPLIT) {
            if (l * 8 < d)
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
                    cp_async16(place + i * kNormCta<TPR>, reinterpret_cast<const uint4*>(row + l * 8) + i);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (col(l, 4 * h) < d) {
                    if constexpr (sizeof(E) == 4) cp_async16(place + h * kNormCta<TPR>, row + col(l, 4 * h));
                    else cp_async8(reinterpret_cast<uint2*>(place) + h, row + col(l, 4 * h));
                }
        }
    }
    __device__ static __forceinline__ void take(const uint4* place, float* f) {
        uint4 q[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) q[i] = place[i * kNormCta<TPR>];
        unpack16(q, f);
    }
};

// A row of d elements in the 16-byte pieces that it lies in, copied by its threads; the first
// piece may begin with the end of what is before the row, within the tensor, the last one is
// filled with zeros.
template <typename E>
__host__ __device__ constexpr int line_pieces(int d) { return (d * (int)sizeof(E) + 30) / 16; }
template <typename E>
__device__ __forceinline__ void line_fetch(const E* row, int l, int tpr, int d, uint4* place) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(row) & ~(uintptr_t)15;
    const int bytes = (int)(reinterpret_cast<uintptr_t>(row) - a) + d * (int)sizeof(E);
    for (int i = l; i * 16 < bytes; i += tpr)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(place + i)),
                     "l"(a + (uintptr_t)i * 16), "r"(min(16, bytes - i * 16))
                     : "memory");
}
template <typename E>
__device__ __forceinline__ void line_take(const E* row, int l, int tpr, int d, const uint4* place, float* f) {
    const E* src = reinterpret_cast<const E*>(reinterpret_cast<const char*>(place) + (reinterpret_cast<uintptr_t>(row) & 15));
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = e * tpr + l < d ? ld_elem(src + e * tpr + l) : 0.f;
}
// What a line's readers wait for: the copies of all of the row's threads.
template <int TPR>
__device__ __forceinline__ void line_ready() {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (TPR <= 1 || TPR > 32) __syncthreads();
    else __syncwarp();
}

// 8 of a parameter vector (`none` where it is not given)
template <int TPR, bool VEC, bool SPLIT>
__device__ __forceinline__ void param_part(const ParamVec& v, int l, int d, float none, float* f) {
    if (!v.p) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = none;
    } else if (VEC && v.vec) {
        if (v.bf16) RowPart<__nv_bfloat16, TPR, true, SPLIT>::load(static_cast<const __nv_bfloat16*>(v.p), l, d, f);
        else RowPart<float, TPR, true, SPLIT>::load(static_cast<const float*>(v.p), l, d, f);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = RowPart<float, TPR, VEC, SPLIT>::col(l, e);
            f[e] = c < d ? ld_param(v, c) : 0.f;
        }
    }
}

// Where a row is: every tensor has y's strides (SAME), or each its own.
template <bool SAME>
struct RowAt {
    unsigned i0 = 0, i1 = 0, i2 = 0;
    int64_t off = 0;
    __device__ __forceinline__ RowAt(const NormParams& p, unsigned row) {
        const unsigned q = p.n2 == 1 ? row : row / p.n2;
        i2 = row - q * p.n2;
        i0 = p.n1 == 1 ? q : q / p.n1;
        i1 = q - i0 * p.n1;
        if (SAME) off = i0 * p.y.s0 + i1 * p.y.s1 + i2 * p.y.s2;
    }
    template <typename E>
    __device__ __forceinline__ E* of(const RowRef& r) const {
        return SAME ? static_cast<E*>(const_cast<void*>(r.p)) + off : row_ptr<E>(r, i0, i1, i2);
    }
};

// Rounds of 16 bytes per thread in shared memory: where each operand's begin, and their number.
template <typename Y, typename R, bool RES, bool BWD>
struct NormPlan {
    static constexpr int nY = sizeof(Y) / 2, nR = RES ? (int)sizeof(R) / 2 : 0;
    static constexpr int z = nY, dout = 2 * nY, r = dout + (BWD ? nY : 0), dr = r + nR, all = dr + (BWD ? nR : 0);
};

template <typename Y, typename R, int TPR, bool VEC, bool RES, bool SAME>
__global__ void __launch_bounds__(kNormCta<TPR>, TPR == 0 ? 2 : 1) k_norm_fwd_rows(NormParams p) {
    constexpr bool SPLIT = sizeof(Y) == 4 || (RES && sizeof(R) == 4);
    using PY = RowPart<Y, TPR, VEC, SPLIT>;
    using PR = RowPart<R, TPR, VEC, SPLIT>;
    using Plan = NormPlan<Y, R, RES, false>;
    constexpr int TH = kNormCta<TPR>, ROWS = TPR <= 1 ? 1 : TH / TPR;
    extern __shared__ uint4 ring_mem[];                // [2][Plan::all][TH], with VEC
    __shared__ __align__(16) float sh[2][2][32];
    const int in_row = (int)threadIdx.x / norm_tpr<TPR>();       // of the CTA's rows, this thread's
    const int l = (int)threadIdx.x - in_row * norm_tpr<TPR>(), d = p.d;
    int turn = 0, s = 0;
    const float inv = 1.f / (float)d;
    float w[8], sc[8], nw[8];
    param_part<TPR, VEC, SPLIT>(p.w, l, d, 1.f, w);
    if (RES) {
        param_part<TPR, VEC, SPLIT>(p.sc, l, d, 1.f, sc);
        param_part<TPR, VEC, SPLIT>(p.nw, l, d, 1.f, nw);
    }
    if (VEC) {                                         // what is never fetched reads as zeros
        for (int i = 0; i < 2 * Plan::all; ++i) ring_mem[i * TH + threadIdx.x] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
    const int tpr = norm_tpr<TPR>(), nY = line_pieces<Y>(d), lines = 2 * nY + (RES ? line_pieces<R>(d) : 0);
    auto place = [&](int s, int k) {                   // lines: y, gate, residual one after another
        return VEC ? ring_mem + ((s * Plan::all + k) * TH + threadIdx.x)
                   : ring_mem + ((s * ROWS + in_row) * lines + (k == 0 ? 0 : k == Plan::z ? nY : 2 * nY));
    };
    auto fetch = [&](const RowAt<SAME>& at, bool on, int s) {
        if constexpr (VEC) {
            if (on) {
                PY::fetch(at.template of<const Y>(p.y), l, d, place(s, 0));
                if (p.gate.p) PY::fetch(at.template of<const Y>(p.gate), l, d, place(s, Plan::z));
                if (RES) PR::fetch(at.template of<const R>(p.res), l, d, place(s, Plan::r));
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else if (p.line && on) {
            line_fetch(at.template of<const Y>(p.y), l, tpr, d, place(s, 0));
            if (p.gate.p) line_fetch(at.template of<const Y>(p.gate), l, tpr, d, place(s, Plan::z));
            if (RES) line_fetch(at.template of<const R>(p.res), l, tpr, d, place(s, Plan::r));
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t base = (int64_t)blockIdx.x * ROWS, row = base + in_row;
    RowAt<SAME> at(p, row < p.rows ? (unsigned)row : 0u);
    fetch(at, row < p.rows, 0);
    for (; base < p.rows; base += step, s ^= 1) {
        if (!VEC && p.line) line_ready<TPR>();         // this row is there, the other place is free
        const bool on = row < p.rows;                  // what a row past the last computes is not stored
        row += step;
        const RowAt<SAME> next(p, row < p.rows ? (unsigned)row : 0u);
        fetch(next, row < p.rows, s ^ 1);
        if (VEC) asm volatile("cp.async.wait_group 1;" ::: "memory");
        float v[8], z[8], r[8];
        if constexpr (VEC) {
            PY::take(place(s, 0), v);
            if (p.gate.p) PY::take(place(s, Plan::z), z);
            if (RES) PR::take(place(s, Plan::r), r);
        } else if (p.line) {
            const int dd = on ? d : 0;
            line_take(at.template of<const Y>(p.y), l, tpr, dd, place(s, 0), v);
            if (p.gate.p) line_take(at.template of<const Y>(p.gate), l, tpr, dd, place(s, Plan::z), z);
            if (RES) line_take(at.template of<const R>(p.res), l, tpr, dd, place(s, Plan::r), r);
        } else {
            const int dd = on ? d : 0;
            PY::load(at.template of<const Y>(p.y), l, dd, v);
            if (p.gate.p) PY::load(at.template of<const Y>(p.gate), l, dd, z);
            if (RES) PR::load(at.template of<const R>(p.res), l, dd, r);
        }
        if (p.w.p) {
            float q = dot8(v, v);
            row_sum<TPR, 1>(&q, sh, turn);
            mul8(v, rsqrtf(q * inv + p.eps), v);
            mul8(v, w, v);
        }
        if (p.gate.p)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= norm_act(z[e], p.act);
        if constexpr (!RES) {
            if (on) PY::store(at.template of<Y>(p.out), l, d, v);
        } else {
            fma8(v, sc, r, v);
            if (on) PR::store(at.template of<R>(p.rout), l, d, v);
            if (p.nw.p) {
                float q = dot8(v, v);
                row_sum<TPR, 1>(&q, sh, turn);
                mul8(v, rsqrtf(q * inv + p.eps), v);
                mul8(v, nw, v);
                if (on) PY::store(at.template of<Y>(p.out), l, d, v);
            }
        }
        at = next;
    }
    if (VEC) asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The parameters stay in shared memory in fp32 (a thread's 8 by pairs of float4, as the ring).
template <int TPR, bool VEC>
__device__ __forceinline__ void param_take(const float4* mem, int k, float* f) {
    constexpr int TH = kNormCta<TPR>;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 q = mem[(k * 2 + i) * TH + threadIdx.x];
        f[4 * i] = q.x;
        f[4 * i + 1] = q.y;
        f[4 * i + 2] = q.z;
        f[4 * i + 3] = q.w;
    }
}

template <typename Y, typename R, int TPR, bool VEC, bool RES, bool SAME>
__global__ void __launch_bounds__(kNormCta<TPR>, TPR <= 1 || TPR == 512 ? 1 : TPR == 128 ? 4 : RES ? 2 : 3) k_norm_bwd_rows(NormParams p) {
    constexpr bool SPLIT = sizeof(Y) == 4 || (RES && sizeof(R) == 4);
    using PY = RowPart<Y, TPR, VEC, SPLIT>;
    using PR = RowPart<R, TPR, VEC, SPLIT>;
    using Plan = NormPlan<Y, R, RES, true>;
    constexpr int TH = kNormCta<TPR>, ROWS = TPR <= 1 ? 1 : TH / TPR;
    extern __shared__ uint4 ring_mem[];                // parameters, then [2][Plan::all][TH], with VEC
    __shared__ __align__(16) float sh[2][2][32];
    const int in_row = (int)threadIdx.x / norm_tpr<TPR>();       // of the CTA's rows, this thread's
    const int l = (int)threadIdx.x - in_row * norm_tpr<TPR>(), d = p.d;
    int turn = 0, s = 0;
    const float inv = 1.f / (float)d;
    float aw[8] = {}, as[8] = {}, an[8] = {};          // sums over this thread's rows
    float4* const par = reinterpret_cast<float4*>(ring_mem);
    auto keep = [&](int k, const ParamVec& v) {
        float f[8];
        param_part<TPR, VEC, SPLIT>(v, l, d, 1.f, f);
        par[(k * 2) * TH + threadIdx.x] = make_float4(f[0], f[1], f[2], f[3]);
        par[(k * 2 + 1) * TH + threadIdx.x] = make_float4(f[4], f[5], f[6], f[7]);
    };
    keep(0, p.w);
    if (RES) keep(1, p.sc), keep(2, p.nw);
    uint4* const ring = ring_mem + (RES ? 6 : 2) * TH;
    const int tpr = norm_tpr<TPR>(), nY = line_pieces<Y>(d), nR = RES ? line_pieces<R>(d) : 0, lines = 3 * nY + 2 * nR;
    auto place = [&](int s, int k) {                   // lines: y, gate, d_out, residual, d_residual_out
        return VEC ? ring + ((s * Plan::all + k) * TH + threadIdx.x)
                   : ring + ((s * ROWS + in_row) * lines +
                             (k < Plan::r ? k / Plan::nY * nY : 3 * nY + (k == Plan::r ? 0 : nR)));
    };
    if (VEC) {                                         // what is never fetched reads as zeros
        for (int i = 0; i < 2 * Plan::all; ++i) ring[i * TH + threadIdx.x] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
    auto fetch = [&](const RowAt<SAME>& at, bool on, int s) {
        if constexpr (VEC) {
            if (on) {
                PY::fetch(at.template of<const Y>(p.y), l, d, place(s, 0));
                if (p.gate.p) PY::fetch(at.template of<const Y>(p.gate), l, d, place(s, Plan::z));
                if (p.dout.p) PY::fetch(at.template of<const Y>(p.dout), l, d, place(s, Plan::dout));
                if (RES) PR::fetch(at.template of<const R>(p.res), l, d, place(s, Plan::r));
                if (RES && p.drout.p) PR::fetch(at.template of<const R>(p.drout), l, d, place(s, Plan::dr));
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else if (p.line && on) {
            line_fetch(at.template of<const Y>(p.y), l, tpr, d, place(s, 0));
            if (p.gate.p) line_fetch(at.template of<const Y>(p.gate), l, tpr, d, place(s, Plan::z));
            if (p.dout.p) line_fetch(at.template of<const Y>(p.dout), l, tpr, d, place(s, Plan::dout));
            if (RES) line_fetch(at.template of<const R>(p.res), l, tpr, d, place(s, Plan::r));
            if (RES && p.drout.p) line_fetch(at.template of<const R>(p.drout), l, tpr, d, place(s, Plan::dr));
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t base = (int64_t)blockIdx.x * ROWS, row = base + in_row;
    RowAt<SAME> at(p, row < p.rows ? (unsigned)row : 0u);
    fetch(at, row < p.rows, 0);
    for (; base < p.rows; base += step, s ^= 1) {
        if (!VEC && p.line) line_ready<TPR>();         // this row is there, the other place is free
        const bool on = ROWS == 1 || row < p.rows;     // a row past the last goes into no sum and no output
        row += step;
        const RowAt<SAME> next(p, row < p.rows ? (unsigned)row : 0u);
        fetch(next, row < p.rows, s ^ 1);
        if (VEC) asm volatile("cp.async.wait_group 1;" ::: "memory");
        const int dd = on ? d : 0;
        float y[8], y1[8], a[8], da[8], dv[8], w[8];   // y: y rstd1 from the first sum on
        auto get_y = [&](int k, const RowRef& ref, float* f) {
            if constexpr (VEC) PY::take(place(s, k), f);
            else if (p.line) line_take(at.template of<const Y>(ref), l, tpr, dd, place(s, k), f);
            else PY::load(at.template of<const Y>(ref), l, dd, f);
        };
        auto get_r = [&](int k, const RowRef& ref, float* f) {
            if constexpr (VEC) PR::take(place(s, k), f);
            else if (p.line) line_take(at.template of<const R>(ref), l, tpr, dd, place(s, k), f);
            else PR::load(at.template of<const R>(ref), l, dd, f);
        };
        get_y(0, p.y, y);
        float rstd1 = 1.f;
        if (p.w.p) {
            float q = dot8(y, y);
            row_sum<TPR, 1>(&q, sh, turn);
            rstd1 = rsqrtf(q * inv + p.eps);
            param_take<TPR, VEC>(par, 0, w);
            mul8(y, rstd1, y);
            mul8(y, w, y1);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) y1[e] = y[e];
        }
        if (p.gate.p) {
            get_y(Plan::z, p.gate, a);
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] = norm_act(a[e], p.act, &da[e]);
            mul8(da, y1, da);                          // what dy2 is worth to the gate
            mul8(y1, a, y1);                           // y2
        }
        if constexpr (!RES) {
            get_y(Plan::dout, p.dout, dv);
        } else {
            float sc[8];
            param_take<TPR, VEC>(par, 1, sc);
            if (p.drout.p) {
                get_r(Plan::dr, p.drout, dv);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) dv[e] = 0.f;
            }
            if (p.nw.p) {
                float r[8], dn[8], t[8];
                get_r(Plan::r, p.res, r);
                get_y(Plan::dout, p.dout, dn);
                param_take<TPR, VEC>(par, 2, t);
                fma8(sc, y1, r, r);
                mul8(t, dn, t);
                float v[2] = {dot8(r, r), dot8(t, r)};
                row_sum<TPR, 2>(v, sh, turn);
                const float rstd2 = rsqrtf(v[0] * inv + p.eps);
                const float m2 = -v[1] * inv * rstd2 * rstd2;
                fma8(r, m2, t, t);
                fma8(t, rstd2, dv, dv);
                mul8(r, rstd2, r);
                if (on) fma8(dn, r, an, an);
            }
            if (on) PR::store(at.template of<R>(p.dres), l, d, dv);
            if (p.sc.p) {
                if (on) fma8(dv, y1, as, as);
                mul8(dv, sc, dv);
            }
        }
        if (p.gate.p) {
            mul8(da, dv, da);
            mul8(dv, a, dv);
            if (on) PY::store(at.template of<Y>(p.dgate), l, d, da);
        }
        if (p.w.p) {
            if (on) fma8(dv, y, aw, aw);
            mul8(dv, w, dv);
            float c = dot8(dv, y);
            row_sum<TPR, 1>(&c, sh, turn);
            fma8(y, -c * inv, dv, dv);                 // y holds one rstd1, the factor after it the others
            mul8(dv, rstd1, dv);
        }
        if (on) PY::store(at.template of<Y>(p.dy), l, d, dv);
        at = next;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!p.part) return;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // this CTA's partial sums: its groups of rows in order
    float* sums = p.part + (int64_t)blockIdx.x * 3 * d;
    auto put = [&](int k, const float* acc) {
        if constexpr (ROWS == 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = RowPart<float, TPR, VEC, SPLIT>::col(l, e);
                if (c < d) sums[k * d + c] = acc[e];
            }
        } else {
            __shared__ float group[ROWS][TPR * 8];
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) group[in_row][RowPart<float, TPR, VEC, SPLIT>::col(l, e)] = acc[e];
            __syncthreads();
            for (int c = threadIdx.x; c < d; c += TH) {
                float t = 0.f;
                for (int g = 0; g < ROWS; ++g) t += group[g][c];
                sums[k * d + c] = t;
            }
        }
    };
    if (p.w.p) put(0, aw);
    if (p.sc.p) put(1, as);
    if (p.nw.p) put(2, an);
}

// ---- longer rows: piece by piece, the row read again (from the caches) for each sum ----------

constexpr int kNormLong = 512;

// A piece: 8 elements per thread, kNormLong * 8 of the row from `c0` on.
template <typename Y, typename R, bool VEC>
struct LongRow {
    using PY = RowPart<Y, kNormLong, VEC, VEC>;
    using PR = RowPart<R, kNormLong, VEC, VEC>;
    const NormParams& p;
    const Y *y, *z, *dout;
    const R *r, *drout;
    __device__ __forceinline__ LongRow(const NormParams& p_, const RowAt<false>& at) : p(p_) {
        y = at.of<const Y>(p.y);
        z = p.gate.p ? at.of<const Y>(p.gate) : nullptr;
        r = p.res.p ? at.of<const R>(p.res) : nullptr;
        dout = p.dout.p ? at.of<const Y>(p.dout) : nullptr;
        drout = p.drout.p ? at.of<const R>(p.drout) : nullptr;
    }
    __device__ __forceinline__ void param(const ParamVec& v, int c0, float* f) const {
        ParamVec w = v;
        if (v.p) w.p = static_cast<const char*>(v.p) + (int64_t)c0 * (v.bf16 ? 2 : 4);
        param_part<kNormLong, VEC, VEC>(w, threadIdx.x, p.d - c0, 1.f, f);
    }
    // y rstd1, y2 (before it y1 in da's factor), act, what dy2 is worth to the gate; r' with a residual
    __device__ __forceinline__ void chain(int c0, float rstd1, float* yn, float* y2, float* a, float* da, float* rp) const {
        const int l = threadIdx.x, d = p.d - c0;
        PY::load(y + c0, l, d, yn);
        if (p.w.p) {
            float w[8];
            param(p.w, c0, w);
            mul8(yn, rstd1, yn);
            mul8(yn, w, y2);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) y2[e] = yn[e];
        }
        if (z) {
            PY::load(z + c0, l, d, a);
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] = norm_act(a[e], p.act, &da[e]);
            mul8(da, y2, da);
            mul8(y2, a, y2);
        }
        if (r) {
            float sc[8];
            param(p.sc, c0, sc);
            PR::load(r + c0, l, d, rp);
            fma8(sc, y2, rp, rp);
        }
    }
    __device__ __forceinline__ float rstd_y(float (*sh)[2][32], int& turn) const {
        if (!p.w.p) return 1.f;
        float q = 0.f, v[8];
        for (int c0 = 0; c0 < p.d; c0 += kNormLong * 8) {
            PY::load(y + c0, threadIdx.x, p.d - c0, v);
            q += dot8(v, v);
        }
        row_sum<kNormLong, 1>(&q, sh, turn);
        return rsqrtf(q / (float)p.d + p.eps);
    }
};

template <typename Y, typename R, bool VEC>
__global__ void __launch_bounds__(kNormLong) k_norm_fwd_long(NormParams p) {
    __shared__ __align__(16) float sh[2][2][32];
    int turn = 0;
    const int l = threadIdx.x;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const RowAt<false> at(p, (unsigned)row);
        const LongRow<Y, R, VEC> x(p, at);
        const float rstd1 = x.rstd_y(sh, turn);
        float yn[8], y2[8], a[8], da[8], rp[8], rstd2 = 0.f;
        if (p.nw.p) {
            float q = 0.f;
            for (int c0 = 0; c0 < p.d; c0 += kNormLong * 8) {
                x.chain(c0, rstd1, yn, y2, a, da, rp);
                q += dot8(rp, rp);
            }
            row_sum<kNormLong, 1>(&q, sh, turn);
            rstd2 = rsqrtf(q / (float)p.d + p.eps);
        }
        for (int c0 = 0; c0 < p.d; c0 += kNormLong * 8) {
            x.chain(c0, rstd1, yn, y2, a, da, rp);
            const int d = p.d - c0;
            if (!x.r) {
                LongRow<Y, R, VEC>::PY::store(at.of<Y>(p.out) + c0, l, d, y2);
                continue;
            }
            LongRow<Y, R, VEC>::PR::store(at.of<R>(p.rout) + c0, l, d, rp);
            if (p.nw.p) {
                float nw[8];
                x.param(p.nw, c0, nw);
                mul8(rp, rstd2, rp);
                mul8(rp, nw, rp);
                LongRow<Y, R, VEC>::PY::store(at.of<Y>(p.out) + c0, l, d, rp);
            }
        }
    }
}

template <typename Y, typename R, bool VEC>
__global__ void __launch_bounds__(kNormLong) k_norm_bwd_long(NormParams p) {
    using Row = LongRow<Y, R, VEC>;
    extern __shared__ float4 acc[];        // [3][pieces][2][kNormLong]: sums for weight, scale, next_weight
    __shared__ __align__(16) float sh[2][2][32];
    int turn = 0;
    const int l = threadIdx.x, pieces = (p.d + kNormLong * 8 - 1) / (kNormLong * 8);
    const float inv = 1.f / (float)p.d;
    for (int i = 0; i < 3 * pieces * 2; ++i) acc[i * kNormLong + l] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int k, int c0, const float* f) {    // a thread's own sums
        float4* q = acc + ((k * pieces + c0 / (kNormLong * 8)) * 2) * kNormLong + l;
        float4 u = q[0], v = q[kNormLong];
        u = make_float4(u.x + f[0], u.y + f[1], u.z + f[2], u.w + f[3]);
        v = make_float4(v.x + f[4], v.y + f[5], v.z + f[6], v.w + f[7]);
        q[0] = u;
        q[kNormLong] = v;
    };
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const RowAt<false> at(p, (unsigned)row);
        const Row x(p, at);
        const float rstd1 = x.rstd_y(sh, turn);
        float yn[8], y2[8], a[8], da[8], rp[8], dn[8], t[8], dv[8];
        float rstd2 = 0.f, m2 = 0.f, m1 = 0.f;
        if (p.nw.p) {
            float v[2] = {0.f, 0.f};
            for (int c0 = 0; c0 < p.d; c0 += kNormLong * 8) {
                x.chain(c0, rstd1, yn, y2, a, da, rp);
                Row::PY::load(x.dout + c0, l, p.d - c0, dn);
                x.param(p.nw, c0, t);
                mul8(t, dn, t);
                v[0] += dot8(rp, rp);
                v[1] += dot8(t, rp);
            }
            row_sum<kNormLong, 2>(v, sh, turn);
            rstd2 = rsqrtf(v[0] * inv + p.eps);
            m2 = -v[1] * inv * rstd2 * rstd2;
        }
        // dv: the gradient of r' (of y2 without a residual); leaves r' rstd2 in rp
        auto top = [&](int c0) {
            const int d = p.d - c0;
            if (!x.r) {
                Row::PY::load(x.dout + c0, l, d, dv);
                return;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) dv[e] = 0.f;
            if (x.drout) Row::PR::load(x.drout + c0, l, d, dv);
            if (p.nw.p) {
                Row::PY::load(x.dout + c0, l, d, dn);
                x.param(p.nw, c0, t);
                mul8(t, dn, t);
                fma8(rp, m2, t, t);
                fma8(t, rstd2, dv, dv);
                mul8(rp, rstd2, rp);
            }
        };
        // dv from there to the gradient of y1, times weight
        auto down = [&](int c0, float* w) {
            if (p.sc.p) {
                x.param(p.sc, c0, w);
                mul8(dv, w, dv);
            }
            if (x.z) mul8(dv, a, dv);
            if (p.w.p) x.param(p.w, c0, w);
        };
        float w[8];
        if (p.w.p) {
            float c = 0.f;
            for (int c0 = 0; c0 < p.d; c0 += kNormLong * 8) {
                x.chain(c0, rstd1, yn, y2, a, da, rp);
                top(c0);
                down(c0, w);
                mul8(dv, w, dv);
                c += dot8(dv, yn);
            }
            row_sum<kNormLong, 1>(&c, sh, turn);
            m1 = -c * inv;
        }
        for (int c0 = 0; c0 < p.d; c0 += kNormLong * 8) {
            const int d = p.d - c0;
            x.chain(c0, rstd1, yn, y2, a, da, rp);
            top(c0);
            if (p.nw.p) {
                mul8(dn, rp, dn);
                add(2, c0, dn);
            }
            if (x.r) Row::PR::store(at.of<R>(p.dres) + c0, l, d, dv);
            if (p.sc.p) {
                mul8(y2, dv, y2);
                add(1, c0, y2);
            }
            if (x.z) {
                float dz[8];
                if (p.sc.p) {
                    x.param(p.sc, c0, w);
                    mul8(w, dv, dz);
                    mul8(dz, da, dz);
                } else {
                    mul8(dv, da, dz);
                }
                Row::PY::store(at.of<Y>(p.dgate) + c0, l, d, dz);
            }
            down(c0, w);
            if (p.w.p) {
                mul8(dv, yn, t);
                add(0, c0, t);
                mul8(dv, w, dv);
                fma8(yn, m1, dv, dv);
                mul8(dv, rstd1, dv);
            }
            Row::PY::store(at.of<Y>(p.dy) + c0, l, d, dv);
        }
    }
    if (!p.part) return;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    float* sums = p.part + (int64_t)blockIdx.x * 3 * p.d;
    for (int k = 0; k < 3; ++k)
        for (int i = 0; i < pieces; ++i) {
            const float4 u = acc[((k * pieces + i) * 2) * kNormLong + l], v = acc[((k * pieces + i) * 2 + 1) * kNormLong + l];
            const float f[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = i * kNormLong * 8 + RowPart<float, kNormLong, VEC, VEC>::col(l, e);
                if (c < p.d) sums[k * p.d + c] = f[e];
            }
        }
}

// d_weight, d_scale, d_next_weight from the partial sums of G CTAs: 32 columns per CTA, 32
// groups of partials each added in order, then the groups in order.  A thread's partials are
// all on their way at once, and the CTAs start with the end of the rows' kernel and wait for
// what it wrote (8 groups, one partial after another, after that kernel: the heads' backward
// took 63 us, not 60).
constexpr int kNormSumGroups = 32;
__global__ void __launch_bounds__(32 * kNormSumGroups) k_norm_bwd_sum(const float* part, int G, int d, float* dw,
                                                                       float* ds, float* dn) {
    constexpr int PER = (kNormBwdCtas + kNormSumGroups - 1) / kNormSumGroups;
    __shared__ float sh[kNormSumGroups][33];
    float* out = blockIdx.y == 0 ? dw : blockIdx.y == 1 ? ds : dn;
    if (!out) return;
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5, j = blockIdx.x * 32 + lane;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float v[PER], s = 0.f;
#pragma unroll
    for (int n = 0; n < PER; ++n) {
        const int i = grp + n * kNormSumGroups;
        v[n] = j < d && i < G ? part[((int64_t)i * 3 + blockIdx.y) * d + j] : 0.f;
    }
#pragma unroll
    for (int n = 0; n < PER; ++n) s += v[n];
    sh[grp][lane] = s;
    __syncthreads();
    if (grp == 0 && j < d) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kNormSumGroups; ++i) t += sh[i][lane];
        out[j] = t;
    }
}

}  // namespace dn
