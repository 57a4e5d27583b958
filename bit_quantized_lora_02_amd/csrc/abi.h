// abi.h -- what the files of the C ABI (abi.hip, head_abi.hip) share: error text, the device check, timed launches,
// size limits (internal to the library).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

#include "launch.h"
#include "qlora.h"

namespace qlora {

// Sets this host thread's error text and returns `code`.
int fail(int code, const char *fmt, ...);
// QLORA_OK where the current device is gfx950 (its index to *dev_out unless NULL).
int check_device(int *dev_out);

// A timed launch gets a pair of events stamped by its own dispatch packet.
struct Timed {
  hipEvent_t a = nullptr, b = nullptr;
  int dev = 0;
  std::string name;
  explicit Timed(const char *kname);
  ~Timed();
};
// The QLORA_E* code of a launch.
int launched(hipError_t e, const char *what, hipStream_t s);

#define LAUNCH(name, call)                             \
  do {                                                 \
    hipError_t e_;                                     \
    {                                                  \
      Timed t_(name);                                  \
      e_ = (call);                                     \
    }                                                  \
    int rc_ = launched(e_, name, s);                   \
    if (rc_ != QLORA_OK) return rc_;                   \
  } while (0)

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
constexpr int64_t kMaxDim = (int64_t)1 << 22;
// Largest weight (n_out n_in) and activation (T n_out, T n_in) element counts: every launch then stays
// below 2^32 work-items per grid dimension (the dequantization runs one work-item per 8 weights, the
// ordered finalize of a split reduction one per output element).
constexpr int64_t kMaxWeights = (int64_t)1 << 34;

constexpr size_t kAlign = 256;  // of workspaces and their parts
inline size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace qlora
