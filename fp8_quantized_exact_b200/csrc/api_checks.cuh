// Argument checks and small host helpers shared by the C entry points.
#pragma once
#include "sage_common.cuh"

namespace sage {

constexpr size_t kAlign = 1024;
constexpr int kMaxGridYZ = 65535;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline int check_dims(int B, int N, int H, int D) {
  if (B < 0 || N < 0 || H < 0 || D < 0) return SAGE_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return SAGE_ERR_UNSUPPORTED;
  // H and B are the y and z extents of the kernels' grids
  if (B > kMaxGridYZ || H > kMaxGridYZ) return SAGE_ERR_UNSUPPORTED;
  // keep every flat index inside int range assumptions of the kernels
  if ((int64_t)B * H > (1 << 30) || N > (1 << 28)) return SAGE_ERR_UNSUPPORTED;
  return SAGE_OK;
}

inline bool empty(int B, int N, int H) { return B == 0 || N == 0 || H == 0; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int check_view(const sage_view_bf16& v) {
  if (!v.data) return SAGE_ERR_INVALID_ARG;
  if (v.stride_b < 0 || v.stride_n < 0 || v.stride_h < 0) return SAGE_ERR_INVALID_ARG;
  if (!aligned16(v.data) || (v.stride_b | v.stride_n | v.stride_h) & 7) return SAGE_ERR_UNSUPPORTED;
  return SAGE_OK;
}

inline int check_out(const void* out, int64_t sb, int64_t sn, int64_t sh) {
  if (!out) return SAGE_ERR_INVALID_ARG;
  if (sb < 0 || sn < 0 || sh < 0) return SAGE_ERR_INVALID_ARG;
  if (!aligned16(out) || (sb | sn | sh) & 7) return SAGE_ERR_UNSUPPORTED;
  return SAGE_OK;
}

inline int check_ws(void* ws, size_t bytes, size_t need) {
  if (!ws) return SAGE_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return SAGE_ERR_WORKSPACE;
  if (bytes < need) return SAGE_ERR_WORKSPACE;
  return SAGE_OK;
}

template <class T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

inline float log2_scale(float sm_scale, int D) {
  if (!(sm_scale > 0.0f)) sm_scale = (float)(1.0 / __builtin_sqrt((double)D));
  return (float)((double)sm_scale * 1.4426950408889634074);
}

}  // namespace sage
