// Host-side helpers shared by the files behind the C ABI: descriptor checks and the
// per-device / per-stream state that deltanet.cu owns.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/deltanet.h"

#define DN_HIDDEN __attribute__((visibility("hidden")))

// Defined in deltanet.cu.
// The current device: its number and SM count; DN_ERR_UNSUPPORTED unless it is sm_100.
DN_HIDDEN dn_status dn_device_check(int& dev, int& sms);
// The error word of (dev, stream) that deltanet_get_error reads; created on first use, which
// allocates: inside a stream capture that is refused (DN_ERR_WORKSPACE), the capture goes on.
DN_HIDDEN dn_status dn_stream_flag(int dev, cudaStream_t stream, int** flag);
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

}  // namespace dn
