// Host-side helpers shared by the tensor-core kernels: the device's SM count,
// the wait budget and tuning knobs from the environment, the driver's
// tensor-map encoder.
#pragma once

#include <cstdlib>

#include <cuda.h>
#include <cuda_runtime.h>

namespace dflash {

inline int num_sms_current() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

// Budget of every mbarrier wait of one launch.  DFLASH_TIMEOUT_NS, read at
// every call (a positive count of nanoseconds; a process may change it
// between calls), takes precedence over DFLASH_TIMEOUT_MS, read once per
// process; without either the budget is 2 s.
inline unsigned long long timeout_ns_from_env() {
  if (const char* e = std::getenv("DFLASH_TIMEOUT_NS")) {
    const long long ns = std::atoll(e);
    if (ns > 0) return static_cast<unsigned long long>(ns);
  }
  static unsigned long long v = [] {
    const char* e = std::getenv("DFLASH_TIMEOUT_MS");
    long long ms = e ? std::atoll(e) : 2000;
    if (ms <= 0) ms = 2000;
    return static_cast<unsigned long long>(ms) * 1000000ull;
  }();
  return v;
}

// Tuning knobs, read at every call (unset: the defaults below).
inline int env_int(const char* name, int dflt, int lo, int hi) {
  const char* e = std::getenv(name);
  if (e == nullptr || e[0] == 0) return dflt;
  int v = std::atoi(e);
  return v < lo ? lo : (v > hi ? hi : v);
}

// Pairs (2-CTA MMA) are used unless DFLASH_PAIR=0 (read at every call).
inline bool pair_allowed() {
  const char* e = std::getenv("DFLASH_PAIR");
  return !(e != nullptr && e[0] == '0');
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiledFn>(nullptr);
    return reinterpret_cast<EncodeTiledFn>(ptr);
  }();
  return fn;
}

}  // namespace dflash
