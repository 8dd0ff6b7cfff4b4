// Host-side helpers shared by the library's translation units: the thread's last error, the
// early-return macros, stage timing and the bump layout of caller-provided workspaces.
#pragma once

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <string>
#include <vector>

#include "common.cuh"
#include "jolt.h"

namespace jolt {

inline thread_local std::string g_err;

inline jolt_status fail(jolt_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_err = buf;
  return s;
}

#define CUDA_TRY(x)                                                                         \
  do {                                                                                      \
    cudaError_t e_ = (x);                                                                   \
    if (e_ != cudaSuccess) return fail(JOLT_ERR_CUDA, "%s: %s", #x, cudaGetErrorString(e_)); \
  } while (0)
#define JTRY(x)                    \
  do {                             \
    jolt_status j_ = (x);          \
    if (j_ != JOLT_OK) return j_;  \
  } while (0)

// ------------------------------------------------------------------------------------------
// optional stage timing: CUDA events recorded around each stage on the launch stream
// ------------------------------------------------------------------------------------------
struct ProfRec {
  std::string name;
  cudaEvent_t a, b;
  long long units;  // work items the stage processed (for per-launch figures)
};
struct Profiler {
  bool on = false;
  std::vector<ProfRec> recs;
  std::vector<cudaEvent_t> pool;
  cudaEvent_t get() {
    if (!pool.empty()) {
      cudaEvent_t e = pool.back();
      pool.pop_back();
      return e;
    }
    cudaEvent_t e;
    cudaEventCreate(&e);
    return e;
  }
};
inline thread_local Profiler g_prof;

struct ProfScope {
  ProfRec rec;
  cudaStream_t st;
  bool on;
  // (events captured into a graph cannot be read)
  static bool capturing(cudaStream_t s) {
    cudaStreamCaptureStatus c = cudaStreamCaptureStatusNone;
    return cudaStreamIsCapturing(s, &c) != cudaSuccess || c != cudaStreamCaptureStatusNone;
  }
  ProfScope(const char* name, cudaStream_t s, long long units = 1) : st(s), on(g_prof.on && !capturing(s)) {
    if (!on) return;
    rec.name = name;
    rec.units = units;
    rec.a = g_prof.get();
    rec.b = g_prof.get();
    cudaEventRecord(rec.a, st);
  }
  ~ProfScope() {
    if (!on) return;
    cudaEventRecord(rec.b, st);
    g_prof.recs.push_back(rec);
  }
};

// offsets of a workspace's parts, each on a 256-byte boundary
struct Bump {
  size_t off = 0;
  size_t take(size_t bytes) {
    size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  }
};

// Launch with programmatic stream serialization: the blocks may be brought up while the kernel before
// them in the stream ends; every thread waits for that end before it reads or writes.
template <typename... P, typename... Q>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const Q&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace jolt
