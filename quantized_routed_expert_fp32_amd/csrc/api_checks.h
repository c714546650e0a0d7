// Argument checks and workspace offsets that the C entry points of the operators share.
#pragma once
#include <hip/hip_runtime.h>

#include <string>

#include "moe_host.h"

namespace moe {

constexpr int kMaxDim = 65536;           // hidden, inter, out: int32 sums of 127^2 stay below 2^31
constexpr int kMaxRows = 1 << 20;
constexpr int64_t kMaxLd = 1 << 22;      // 255 rows of 16-bit elements stay below 2^32 bytes

inline int bad(const std::string& m, int st = MOE_EINVAL) {
  set_error(m);
  return st;
}
inline int hip_bad(const char* what, hipError_t e) {
  return bad(std::string(what) + ": " + hipGetErrorName(e) + " (" + hipGetErrorString(e) + ")", MOE_EHIP);
}

inline int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

inline int check_dim(const char* fn, const char* name, int64_t v, int64_t hi) {
  if (v >= 1 && v <= hi) return MOE_OK;
  return bad(std::string(fn) + ": " + name + "=" + std::to_string(v) + " outside 1.." + std::to_string(hi));
}
inline int check_ld(const char* fn, const char* name, int64_t ld, int64_t cols) {
  if (ld >= cols && ld <= kMaxLd) return MOE_OK;
  return bad(std::string(fn) + ": " + name + "=" + std::to_string(ld) + " outside " + std::to_string(cols) + ".." +
             std::to_string(kMaxLd), MOE_ESHAPE);
}
inline int check_dtype(const char* fn, int dt) {
  if (dt == MOE_BF16 || dt == MOE_FP16) return MOE_OK;
  return bad(std::string(fn) + ": dtype " + std::to_string(dt) + " is not MOE_BF16 or MOE_FP16", MOE_EUNSUPPORTED);
}

struct Bump {
  uint64_t at = 0;
  uint64_t take(uint64_t bytes) {
    const uint64_t o = at;
    at = align256(at + bytes);
    return o;
  }
};

inline int check_ws(const char* fn, const void* ws, uint64_t have, uint64_t need) {
  if (!need) return MOE_OK;
  if (!ws) return bad(std::string(fn) + ": NULL ws");
  if (reinterpret_cast<uintptr_t>(ws) % 256) return bad(std::string(fn) + ": ws is not 256-byte aligned");
  if (have < need)
    return bad(std::string(fn) + ": workspace of " + std::to_string(have) + " bytes, needs " + std::to_string(need),
               MOE_ENOSPACE);
  return MOE_OK;
}

}  // namespace moe
