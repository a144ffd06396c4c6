// What the files of the C ABI share: error reporting, the dims a call reads,
// and the checks of pointers and workspaces. Every check runs before the first
// launch of a call.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "swimba.h"

namespace swimba {

// Records the message for swimba_last_error() and returns st.
swimba_status fail(swimba_status st, const char* fmt, ...);
swimba_status hip_status(hipError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Dims {
  int64_t Bt, T, D, H, P, N, G, E, k, L, M, W, HP, GN;
  bool bf16;
  size_t esize;
};

swimba_status read_dims(const swimba_dims* d, Dims& o);
// The same for a size query, which leaves swimba_last_error() as it was.
bool query_dims(const swimba_dims* d, Dims& o);

// The largest record a buffer resource may cover: loads that must read zeros
// take the byte offset 2^31, which has to lie past it.
constexpr int64_t kMaxRecord = 0x7FFFFFF0ll;

swimba_status check_ws(void* ws, size_t have, size_t need);

#define REQUIRE_PTR(p)                                                  \
  do {                                                                  \
    if (!(p)) return fail(SWIMBA_ERR_NULL, "%s is NULL", #p);           \
    if (!aligned16(p)) return fail(SWIMBA_ERR_ALIGN, "%s is not 16-byte aligned", #p); \
  } while (0)
#define OPTIONAL_PTR(p)                                                 \
  do {                                                                  \
    if ((p) && !aligned16(p)) return fail(SWIMBA_ERR_ALIGN, "%s is not 16-byte aligned", #p); \
  } while (0)

}  // namespace swimba
