// Host helpers of the C-ABI entry points: alignment, overlap and status words.
#pragma once

#include "launch.h"

namespace sptp {

constexpr size_t kAlign = 256;  // alignment of a workspace and of its parts
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline bool dtype_ok(int dtype) { return dtype == SPTP_BF16 || dtype == SPTP_FP32; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool overlaps(const void* a, size_t an, const void* b, size_t bn) {
    if (a == nullptr || b == nullptr || an == 0 || bn == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + bn && b0 < a0 + an;
}
inline DeviceStatus* ws_status(void* ws) { return reinterpret_cast<DeviceStatus*>(ws); }
inline int reset_status(void* ws, cudaStream_t s) {
    return cudaMemsetAsync(ws, 0, sizeof(DeviceStatus), s) == cudaSuccess ? SPTP_OK : SPTP_ERR_CUDA;
}
// Per-device SM count and compute capability, queried once per device
// (api.cu); SPTP_ERR_DEVICE unless it is 10.3.
int device_info(DevInfo* out);

}  // namespace sptp
