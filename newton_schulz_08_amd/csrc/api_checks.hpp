// Checks that the operators' C entry points share: ranges and types of the
// arguments, buffers and their overlaps, the workspace, the launch itself.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <exception>
#include <string>

#include "../../include/dmuon.h"
#include "api_util.hpp"

namespace dmuon {

// No exception leaves a C entry point.
template <typename F> int guarded(F&& f) noexcept {
  try {
    clear_error();
    return f();
  } catch (const std::exception&) {
    return DMUON_ERR_INVALID_ARG;   // out of host memory for an error text
  }
}

inline int invalid(const std::string& msg) { return fail(DMUON_ERR_INVALID_ARG, msg); }

inline bool is_float(int dt) { return dt == DMUON_F32 || dt == DMUON_BF16; }
inline bool is_index(int dt) { return dt == DMUON_I32 || dt == DMUON_I64; }
inline int64_t size_of(int dt) { return dt == DMUON_BF16 ? 2 : dt == DMUON_I64 ? 8 : 4; }

inline int check_float(int dt, const char* what) {
  return is_float(dt) ? DMUON_OK
                      : fail(DMUON_ERR_UNSUPPORTED_DTYPE, std::string(what) + " must be DMUON_F32 or DMUON_BF16");
}
inline int check_index(int dt, const char* what) {
  return is_index(dt) ? DMUON_OK
                      : fail(DMUON_ERR_UNSUPPORTED_DTYPE, std::string(what) + " must be DMUON_I32 or DMUON_I64");
}
inline int check_range(int64_t v, int64_t lo, int64_t hi, const char* what) {
  if (v >= lo && v <= hi) return DMUON_OK;
  return invalid(std::string(what) + " = " + std::to_string(v) + " outside [" + std::to_string(lo) + ", " +
                 std::to_string(hi) + "]");
}

// A buffer of a call: `rows` rows of `width` bytes, `pitch` bytes apart.
struct Buf {
  const char* name;
  const void* p;
  int64_t rows, width, pitch;
  int64_t align;
  bool written;
  uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t end() const { return begin() + static_cast<uintptr_t>((rows - 1) * pitch + width); }
  bool empty() const { return rows <= 0 || width <= 0; }
};
inline Buf flat(const char* name, const void* p, int64_t bytes, int64_t align, bool written) {
  return Buf{name, p, bytes > 0 ? 1 : 0, bytes, bytes, align, written};
}

inline bool disjoint(const Buf& a, const Buf& b) {
  if (a.end() <= b.begin() || b.end() <= a.begin()) return true;
  // rows of one packed buffer: equally spaced, side by side
  if (a.pitch != b.pitch || a.rows <= 1 || b.rows <= 1) return false;
  const uintptr_t pitch = static_cast<uintptr_t>(a.pitch);
  const uintptr_t d = b.begin() >= a.begin() ? (b.begin() - a.begin()) % pitch
                                             : (pitch - (a.begin() - b.begin()) % pitch) % pitch;
  return d >= static_cast<uintptr_t>(a.width) && d + static_cast<uintptr_t>(b.width) <= pitch;
}
inline bool same(const Buf& a, const Buf& b) {
  return a.p == b.p && a.rows == b.rows && a.width == b.width && (a.rows == 1 || a.pitch == b.pitch);
}

// Pointers set and aligned, written buffers apart from all others.  A written
// buffer may coincide with a read one of the listed in-place pairs.
inline int check_bufs(const Buf* bufs, int n, const int (*in_place)[2] = nullptr, int n_in_place = 0) {
  for (int i = 0; i < n; ++i) {
    if (bufs[i].empty()) continue;
    if (!bufs[i].p) return invalid(std::string(bufs[i].name) + " is NULL");
    if (!aligned(bufs[i].p, static_cast<size_t>(bufs[i].align)))
      return invalid(std::string(bufs[i].name) + " is not aligned to its element size");
  }
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j) {
      if (bufs[i].empty() || bufs[j].empty() || (!bufs[i].written && !bufs[j].written)) continue;
      if (disjoint(bufs[i], bufs[j])) continue;
      bool ok = false;
      for (int k = 0; k < n_in_place && !ok; ++k)
        ok = in_place[k][0] == i && in_place[k][1] == j && same(bufs[i], bufs[j]);
      if (!ok) return invalid(std::string("buffers ") + bufs[i].name + " and " + bufs[j].name + " overlap");
    }
  return DMUON_OK;
}

inline int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return DMUON_OK;
  if (!ws) return fail(DMUON_ERR_WORKSPACE, "workspace is NULL");
  if (have < need)
    return fail(DMUON_ERR_WORKSPACE,
                "workspace has " + std::to_string(have) + " bytes, needs " + std::to_string(need));
  if (!aligned(ws, kAlign)) return fail(DMUON_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  return DMUON_OK;
}

template <typename F>
int launched(const char* what, int cls, double flops, double bytes, void* stream, bool capturing, F&& launch) {
  const hipError_t e = timed(cls, flops, bytes, static_cast<hipStream_t>(stream), launch, capturing);
  if (e != hipSuccess) return fail(DMUON_ERR_HIP, std::string(what) + " launch: " + hipGetErrorString(e));
  return DMUON_OK;
}

#define DMUON_TRY(x) \
  do {               \
    const int st_ = (x); \
    if (st_ != DMUON_OK) return st_; \
  } while (0)

}  // namespace dmuon
