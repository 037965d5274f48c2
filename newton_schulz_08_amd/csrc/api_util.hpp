// What the files behind the C entry points share: the error text, the checks of
// device, stream and buffers, and the kernel timing record.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

namespace dmuon {

// Stores `msg` as the calling thread's last error and returns `code`.
int fail(int code, const std::string& msg);
void clear_error();

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v, size_t a = kAlign) { return (v + a - 1) / a * a; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The device must be a gfx950.  A call that uploads descriptors from host
// memory that lives only for the call cannot be recorded into a graph, so the
// stream must not be capturing either; a call that takes everything by value
// passes `capturing`, is told whether the stream is, and may be recorded.
int check_device(void* hip_stream, bool* capturing = nullptr);

// Kernel families of dmuon_profile_read.
enum KernelClass {
  kKPrologue = 0, kKNorm, kKSyrk, kKGemm, kKApply, kKSquare, kKClip, kKAdamw,
  kKAdamwRows, kKEmbed, kKEmbedPlan, kKEmbedGrad, kKDistill, kKQkNorm, kKQkNormGrad, kKNumClasses
};

struct ProfMark { hipEvent_t start = nullptr, stop = nullptr; };
bool prof_on();
hipError_t prof_begin(hipStream_t stream, ProfMark* mark);
hipError_t prof_end(int cls, double flops, double bytes, hipStream_t stream, const ProfMark& mark);

// Runs `launch` on `stream`, bracketed by events when profiling is on (never
// on a capturing stream, whose events carry no times).
template <typename F>
hipError_t timed(int cls, double flops, double bytes, hipStream_t stream, F&& launch, bool capturing = false) {
  if (capturing || !prof_on()) return launch();
  ProfMark mark;
  hipError_t e = prof_begin(stream, &mark);
  if (e != hipSuccess) return e;
  if ((e = launch()) != hipSuccess) return e;
  return prof_end(cls, flops, bytes, stream, mark);
}

}  // namespace dmuon
