// zr_checks.h — host helpers shared by the C entry points: byte spans and
// overlap, layout tests, device-pointer checks, status mapping, the trace.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <string>

#include "../../include/zr.h"
#include "zr_plan.h"

namespace zr {

// Byte interval [lo, hi) touched by a tensor (empty when numel == 0).
struct Span {
  uintptr_t lo = 0, hi = 0;
};
inline Span span_of(const void* p, int64_t extent, int es = 4) {
  Span s;
  if (p && extent > 0) {
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.hi = s.lo + uintptr_t(extent) * uintptr_t(es);
  }
  return s;
}
inline bool overlaps(const Span& x, const Span& y) {
  return x.hi > x.lo && y.hi > y.lo && x.lo < y.hi && y.lo < x.hi;
}

// Sufficient condition for a strided view to address every element once:
// sorted by stride, each stride exceeds the extent of all smaller dims.
inline bool non_overlapping(const TDesc& t) {
  int idx[kMaxDims];
  int m = 0;
  for (int i = 0; i < t.nd; ++i)
    if (t.size[i] > 1) idx[m++] = i;
  std::sort(idx, idx + m, [&](int x, int y) { return t.stride[x] < t.stride[y]; });
  int64_t reach = 0;  // largest offset reachable with the dims seen so far
  for (int i = 0; i < m; ++i) {
    const int d = idx[i];
    if (t.stride[d] <= reach) return false;
    reach += (t.size[d] - 1) * t.stride[d];
  }
  return true;
}

inline bool same_layout(const TDesc& x, const TDesc& y) {
  if (x.ptr != y.ptr || x.nd != y.nd) return false;
  for (int i = 0; i < x.nd; ++i) {
    if (x.size[i] != y.size[i]) return false;
    if (x.size[i] > 1 && x.stride[i] != y.stride[i]) return false;
  }
  return true;
}

inline int check_device_ptr(const void* p) {
  if (p == nullptr) return ZR_ERR_NULL;
  cudaPointerAttributes at;
  const cudaError_t e = cudaPointerGetAttributes(&at, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return ZR_ERR_DEVICE;
  }
  if (at.type == cudaMemoryTypeUnregistered) return ZR_ERR_DEVICE;
  // Pinned host memory is used through the same address only (unified
  // addressing maps it there); a different device alias is refused.
  if (at.type == cudaMemoryTypeHost && at.devicePointer != p) return ZR_ERR_DEVICE;
  if (at.type == cudaMemoryTypeDevice) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
      cudaGetLastError();
      return ZR_ERR_DEVICE;
    }
    if (at.device != dev) return ZR_ERR_DEVICE;
  }
  return ZR_OK;
}

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? ZR_OK : ZR_ERR_CUDA; }

inline int copy_json(const std::string& s, char* buf, size_t len) {
  if (!buf || len == 0) return ZR_ERR_NULL;
  const size_t m = std::min(len - 1, s.size());
  std::memcpy(buf, s.data(), m);
  buf[m] = '\0';
  return ZR_OK;
}

// ZR_TRACE set (and not "0"): every forward, backward, sum-to-shape, unary and
// training-operator call about to launch writes one line "zr_trace <entry> <plan JSON>" to
// stderr.  Read once per process.
inline bool trace_on() {
  static const bool on = [] {
    const char* e = std::getenv("ZR_TRACE");
    return e != nullptr && e[0] != '\0' && !(e[0] == '0' && e[1] == '\0');
  }();
  return on;
}

// json(): the plan.  It allocates, and the C entry points raise nothing: where
// there is no memory for the line, the call goes on without it.
template <typename F>
inline void trace(const char* entry, F json) noexcept {
  if (!trace_on()) return;
  try {
    std::fprintf(stderr, "zr_trace %s %s\n", entry, json().c_str());
  } catch (...) {
  }
}

}  // namespace zr
