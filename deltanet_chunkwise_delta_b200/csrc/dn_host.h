// Host-side helpers shared by the files behind the C ABI: descriptor checks and the
// per-device / per-stream state that deltanet.cu owns.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include "../../include/deltanet.h"

#define DN_HIDDEN __attribute__((visibility("hidden")))

// Defined in deltanet.cu.
// The current device: its number and SM count; DN_ERR_UNSUPPORTED unless it is sm_100.
DN_HIDDEN dn_status dn_device_check(int& dev, int& sms);
// The error word of (dev, stream) that deltanet_get_error reads, made on first use, inside a
// stream capture too.
DN_HIDDEN dn_status dn_stream_flag(int dev, cudaStream_t stream, int** flag);
// This thread's deltanet_test_set_wait.
DN_HIDDEN void dn_wait_settings(unsigned long long* wait_ns, int* stall_chunk);
// What deltanet_last_launches reports for this thread's last successful call.
DN_HIDDEN void dn_note_launches(int n);

namespace dn {

inline int64_t elem_size(int32_t dt) { return dt == DN_F32 ? 4 : dt == DN_BF16 ? 2 : dt == DN_I32 ? 4 : 0; }

inline bool shape_eq(const dn_tensor* t, int ndim, const int64_t* dims) {
    if (!t || t->ndim != ndim) return false;
    for (int i = 0; i < ndim; ++i)
        if (t->shape[i] != dims[i]) return false;
    return true;
}

inline int64_t numel(const dn_tensor* t) {
    int64_t n = 1;
    for (int i = 0; i < t->ndim; ++i) n *= t->shape[i];
    return n;
}

// Byte span [lo, hi) touched by a strided view (non-negative strides only).
inline bool span(const dn_tensor* t, uintptr_t& lo, uintptr_t& hi) {
    lo = hi = 0;
    if (!t || numel(t) == 0) return true;
    int64_t last = 0;
    for (int i = 0; i < t->ndim; ++i) {
        if (t->stride[i] < 0) return false;
        last += (t->shape[i] - 1) * t->stride[i];
    }
    const int64_t es = elem_size(t->dtype);
    lo = reinterpret_cast<uintptr_t>(t->data);
    hi = lo + static_cast<uintptr_t>((last + 1) * es);
    return true;
}

inline bool overlap(const dn_tensor* a, const dn_tensor* b) {
    uintptr_t a0, a1, b0, b1;
    span(a, a0, a1);
    span(b, b0, b1);
    if (a0 == a1 || b0 == b1) return false;
    return a0 < b1 && b0 < a1;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// q/k/v/out: [B, T, H, d], stride[3] == 1, 16-byte aligned rows and strides.
inline bool token_tensor_ok(const dn_tensor* t) {
    if (t->stride[3] != 1) return false;
    const int64_t es = elem_size(t->dtype);
    if (numel(t) == 0) return true;
    if (!t->data || !aligned16(t->data)) return false;
    for (int i = 0; i < 3; ++i)
        if (t->stride[i] < 0 || (t->stride[i] * es) % 16 != 0) return false;
    return true;
}

inline bool state_tensor_ok(const dn_tensor* t, int64_t dv) {
    if (t->dtype != DN_F32 || t->stride[3] != 1 || t->stride[2] != dv) return false;
    if (numel(t) == 0) return true;
    if (!t->data || !aligned16(t->data)) return false;
    return t->stride[0] >= 0 && t->stride[1] >= 0 && (t->stride[0] * 4) % 16 == 0 &&
           (t->stride[1] * 4) % 16 == 0;
}

constexpr int64_t kMax31 = (int64_t(1) << 31) - 1;

// A tensor of the given shape: a dtype of the mask, last stride 1, non-negative strides,
// data aligned to its element (any address where it has no elements).
constexpr int kF32 = 1 << DN_F32, kBf16 = 1 << DN_BF16;
inline bool view_ok(const dn_tensor* t, int ndim, const int64_t* dims, int dtypes) {
    if (!shape_eq(t, ndim, dims) || t->dtype < 0 || t->dtype > 2 || !(dtypes >> t->dtype & 1)) return false;
    for (int i = 0; i < ndim; ++i)
        if (t->stride[i] < 0) return false;
    if (t->shape[ndim - 1] > 1 && t->stride[ndim - 1] != 1) return false;
    if (numel(t) == 0) return true;
    return t->data && reinterpret_cast<uintptr_t>(t->data) % elem_size(t->dtype) == 0;
}

// No two elements of an output share an address.
inline bool distinct(const dn_tensor* t) {
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
inline bool interleaved(const dn_tensor* a, const dn_tensor* b) {
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

inline bool clash(const dn_tensor* a, const dn_tensor* b) { return overlap(a, b) && !interleaved(a, b); }

// DN_ERR_INVALID_ARG for an output whose own elements overlap, DN_ERR_ALIAS for one that
// overlaps an input or another output (null entries are skipped).
inline dn_status alias_check(std::initializer_list<const dn_tensor*> outs, std::initializer_list<const dn_tensor*> ins) {
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

inline bool index_ok(const dn_tensor* t, int64_t min_len) {
    return t->ndim == 1 && t->dtype == DN_I32 && t->shape[0] >= min_len &&
           (t->shape[0] <= 1 || t->stride[0] == 1) && (t->shape[0] == 0 || t->data) &&
           reinterpret_cast<uintptr_t>(t->data) % 4 == 0;
}

inline dn_status launched(int n) {
    if (cudaGetLastError() != cudaSuccess) return DN_ERR_CUDA;
    dn_note_launches(n);
    return DN_OK;
}

}  // namespace dn
