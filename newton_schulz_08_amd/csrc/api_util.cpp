// Error text, device checks and the kernel timing record (api_util.hpp), with
// the C entry points that read them.
#include "api_util.hpp"

#include <algorithm>
#include <cstdio>
#include <cstring>
#include <map>
#include <mutex>
#include <vector>

#include "../../include/dmuon.h"

namespace dmuon {
namespace {

thread_local std::string g_last_error;

std::mutex g_dev_mu;
std::map<int, int> g_dev_status;  // device -> status

const char* kClassNames[kKNumClasses] = {
    "prologue", "norm_finalize", "syrk", "ns_gemm", "apply_x0", "syrk_square", "grad_clip", "adamw",
    "adamw_rows", "embedding", "embedding_plan", "embedding_grad", "distill_loss", "qk_norm_rope", "qk_norm_rope_grad"};

struct ProfRecord {
  int cls;
  hipEvent_t start, stop;
  double flops, bytes;
};

std::mutex g_prof_mu;
bool g_prof_on = false;
std::vector<ProfRecord> g_prof_records;
std::vector<hipEvent_t> g_event_pool;

hipEvent_t take_event() {
  if (!g_event_pool.empty()) {
    hipEvent_t e = g_event_pool.back();
    g_event_pool.pop_back();
    return e;
  }
  hipEvent_t e = nullptr;
  if (hipEventCreate(&e) != hipSuccess) return nullptr;
  return e;
}

}  // namespace

int fail(int code, const std::string& msg) {
  g_last_error = msg;
  return code;
}

void clear_error() { g_last_error.clear(); }

int check_device(void* hip_stream, bool* capturing) {
  int ndev = 0;
  if (hipGetDeviceCount(&ndev) != hipSuccess || ndev <= 0) {
    (void)hipGetLastError();
    return fail(DMUON_ERR_NO_DEVICE, "no HIP device visible");
  }
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return fail(DMUON_ERR_HIP, "hipGetDevice failed");
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    auto it = g_dev_status.find(dev);
    if (it == g_dev_status.end()) {
      hipDeviceProp_t prop;
      if (hipGetDeviceProperties(&prop, dev) != hipSuccess)
        return fail(DMUON_ERR_HIP, "hipGetDeviceProperties failed");
      const int st = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? DMUON_OK : DMUON_ERR_UNSUPPORTED_ARCH;
      g_dev_status[dev] = st;
      if (st != DMUON_OK) return fail(st, std::string("current device is ") + prop.gcnArchName + ", not gfx950");
    } else if (it->second != DMUON_OK) {
      return fail(it->second, "current device is not gfx950");
    }
  }
  hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
  const hipError_t e = hipStreamIsCapturing(static_cast<hipStream_t>(hip_stream), &cs);
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return fail(DMUON_ERR_HIP, std::string("hipStreamIsCapturing: ") + hipGetErrorString(e));
  }
  if (capturing)
    *capturing = cs != hipStreamCaptureStatusNone;
  else if (cs != hipStreamCaptureStatusNone)
    return fail(DMUON_ERR_INVALID_ARG,
                "the stream is capturing a graph; the descriptor upload reads host memory that does not outlive "
                "the call, so these calls cannot be recorded");
  return DMUON_OK;
}

bool prof_on() {
  std::lock_guard<std::mutex> lk(g_prof_mu);
  return g_prof_on;
}

hipError_t prof_begin(hipStream_t stream, ProfMark* mark) {
  {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    mark->start = take_event();
    mark->stop = take_event();
  }
  if (!mark->start || !mark->stop) return hipErrorOutOfMemory;
  return hipEventRecord(mark->start, stream);
}

hipError_t prof_end(int cls, double flops, double bytes, hipStream_t stream, const ProfMark& mark) {
  const hipError_t e = hipEventRecord(mark.stop, stream);
  if (e != hipSuccess) return e;
  std::lock_guard<std::mutex> lk(g_prof_mu);
  g_prof_records.push_back(ProfRecord{cls, mark.start, mark.stop, flops, bytes});
  return hipSuccess;
}

}  // namespace dmuon

using namespace dmuon;

extern "C" {

const char* dmuon_last_error(void) { return g_last_error.c_str(); }

int dmuon_profile_enable(int on) {
  std::lock_guard<std::mutex> lk(g_prof_mu);
  g_prof_on = on != 0;
  return DMUON_OK;
}

int dmuon_profile_read(dmuon_kernel_stat* stats, int max_stats, int* n_stats) {
  clear_error();
  if (!n_stats || (max_stats > 0 && !stats)) return fail(DMUON_ERR_INVALID_ARG, "NULL output");
  std::vector<ProfRecord> recs;
  {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    recs.swap(g_prof_records);
  }
  dmuon_kernel_stat agg[kKNumClasses];
  std::memset(agg, 0, sizeof(agg));
  int status = DMUON_OK;
  for (const auto& r : recs) {
    float ms = 0.0f;
    if (hipEventSynchronize(r.stop) != hipSuccess || hipEventElapsedTime(&ms, r.start, r.stop) != hipSuccess)
      status = fail(DMUON_ERR_HIP, "event timing failed");
    agg[r.cls].launches++;
    agg[r.cls].total_ms += ms;
    agg[r.cls].flops += r.flops;
    agg[r.cls].bytes += r.bytes;
  }
  {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    for (const auto& r : recs) {
      g_event_pool.push_back(r.start);
      g_event_pool.push_back(r.stop);
    }
  }
  int n = 0;
  for (int c = 0; c < kKNumClasses; ++c) {
    if (agg[c].launches == 0) continue;
    if (n < max_stats) {
      stats[n] = agg[c];
      std::snprintf(stats[n].name, sizeof(stats[n].name), "%s", kClassNames[c]);
    }
    ++n;
  }
  *n_stats = std::min(n, std::max(max_stats, 0));
  return status;
}

}  // extern "C"
