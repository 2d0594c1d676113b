// Host checks shared by the entry points that take strided tensors and a
// workspace (la_muon_api.cpp, la_norm_api.cpp, la_loss_api.cpp). Not installed.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <exception>
#include <vector>

#include "la_error.h"
#include "layeradam.h"

namespace la {

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Bytes of a la_element_type.
inline int64_t type_bytes(int type) { return type == LA_TYPE_FP32 ? 4 : 2; }

template <typename T>
T* place(void* workspace, int64_t at) {
  return reinterpret_cast<T*>(static_cast<char*>(workspace) + at);
}

// Hands out parts of a workspace from its start.
struct Taker {
  int64_t at = 0;
  int64_t operator()(int64_t bytes) {
    const int64_t here = at;
    at += round_up(bytes, LA_WORKSPACE_ALIGNMENT);
    return here;
  }
};

inline la_status check_workspace(const void* ws, int64_t given, int64_t needed) {
  if (needed == 0) return LA_OK;
  if (ws == nullptr) return fail(LA_ERR_INVALID_ARGUMENT, "workspace is NULL");
  if (!aligned(ws, LA_WORKSPACE_ALIGNMENT))
    return fail(LA_ERR_MISALIGNED, "workspace is not %d-byte aligned", LA_WORKSPACE_ALIGNMENT);
  if (given < needed)
    return fail(LA_ERR_INVALID_ARGUMENT, "workspace_bytes = %lld, need %lld",
                static_cast<long long>(given), static_cast<long long>(needed));
  return LA_OK;
}

// ---- aliasing --------------------------------------------------------------------------

struct Range {
  uintptr_t begin, end;  // [begin, end)
  const char* what;
  int tensor;            // its index, or -1 where the call's tensors have names
};

inline Range range(const void* p, int64_t bytes, const char* what, int tensor = -1) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return {b, b + static_cast<uintptr_t>(bytes), what, tensor};
}

// Written ranges must be pairwise disjoint and disjoint from every range that
// is only read. Ranges are not empty.
inline la_status check_disjoint(std::vector<Range>& written, const std::vector<Range>& read) {
  auto meet = [](const Range& a, const Range& b) { return a.begin < b.end && b.begin < a.end; };
  auto refuse = [](const Range& a, const Range& b) {
    if (a.tensor < 0 && b.tensor < 0)
      return fail(LA_ERR_ALIASING, "%s overlaps %s", a.what, b.what);
    return fail(LA_ERR_ALIASING, "%s of tensor %d overlaps %s of tensor %d", a.what, a.tensor,
                b.what, b.tensor);
  };
  std::sort(written.begin(), written.end(),
            [](const Range& a, const Range& b) { return a.begin < b.begin; });
  for (size_t k = 1; k < written.size(); ++k)
    if (meet(written[k - 1], written[k])) return refuse(written[k - 1], written[k]);
  for (const Range& r : read) {
    // the first written range that ends after r begins: the ranges are
    // disjoint and sorted, so their ends are sorted too
    auto it = std::lower_bound(written.begin(), written.end(), r.begin,
                               [](const Range& w, uintptr_t x) { return w.end <= x; });
    if (it != written.end() && meet(*it, r)) return refuse(r, *it);
  }
  return LA_OK;
}

// No exception leaves the C ABI (a host allocation may fail).
template <typename F>
auto guarded(F f, decltype(f()) on_failure) -> decltype(f()) {
  try {
    return f();
  } catch (const std::exception& e) {
    fail(LA_ERR_INVALID_ARGUMENT, "%s", e.what());
    return on_failure;
  }
}

}  // namespace la
