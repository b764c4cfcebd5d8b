// Which operands of a call share memory (host).
#pragma once

#include <stdint.h>

#include "ttl_internal.h"

namespace ttl {

// n matrices [rows, width bytes] with row stride ld bytes (ld >= width).
struct Operand {
  const char* name;
  const void* const* at;
  int n;
  int64_t rows, ld, width;
};
inline Operand operand(const char* name, const void* const* at, int n, int64_t rows, int64_t ld, int64_t width) {
  return Operand{name, at, n, rows, ld, width};
}
// n contiguous ranges of `bytes` bytes.
inline Operand operand(const char* name, const void* const* at, int n, int64_t bytes) {
  return Operand{name, at, n, 1, bytes, bytes};
}

inline int64_t operand_span(const Operand& a) { return a.rows > 0 ? (a.rows - 1) * a.ld + a.width : 0; }

// Whether the matrix of a at p and the one of b at q share a byte.  Exact for equal row strides (column ranges of one
// matrix do not); for two different ones, whether their spans meet.
inline bool operands_share(const Operand& a, const void* p, const Operand& b, const void* q) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(p), pb = reinterpret_cast<uintptr_t>(q);
  if (pb < pa) return operands_share(b, q, a, p);
  if (pb - pa >= static_cast<uint64_t>(operand_span(a)) || operand_span(b) == 0) return false;
  if (a.rows > 1 && b.rows > 1 && a.ld != b.ld) return true;
  const int64_t ld = a.rows > 1 ? a.ld : (b.rows > 1 ? b.ld : operand_span(a));
  const int64_t d = static_cast<int64_t>((pb - pa) % static_cast<uint64_t>(ld));
  return d < a.width || d + b.width > ld;
}

// Whether any matrix of a shares memory with any of b (of a list with itself: with any other of it).
inline bool operands_meet(const Operand& a, const Operand& b) {
  const bool self = &a == &b;
  auto bounds = [](const Operand& o, uintptr_t& lo, uintptr_t& hi) {
    lo = UINTPTR_MAX;
    hi = 0;
    for (int i = 0; i < o.n; ++i) {
      const uintptr_t p = reinterpret_cast<uintptr_t>(o.at[i]);
      lo = p < lo ? p : lo;
      hi = p > hi ? p : hi;
    }
    hi += static_cast<uintptr_t>(operand_span(o));
  };
  if (!self) {   // lists apart as a whole
    uintptr_t alo, ahi, blo, bhi;
    bounds(a, alo, ahi);
    bounds(b, blo, bhi);
    if (ahi <= blo || bhi <= alo) return false;
  }
  const uintptr_t sa = static_cast<uintptr_t>(operand_span(a)), sb = static_cast<uintptr_t>(operand_span(b));
  for (int i = 0; i < a.n; ++i) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.at[i]);
    for (int j = self ? i + 1 : 0; j < b.n; ++j) {
      const uintptr_t pb = reinterpret_cast<uintptr_t>(b.at[j]);
      if (pa < pb + sb && pb < pa + sa && operands_share(a, a.at[i], b, b.at[j])) return true;
    }
  }
  return false;
}

// TTL_ERR_ARG where an output shares memory with another operand, or two matrices of one output do.
inline int check_alias(const Operand* outs, int n_outs, const Operand* ins, int n_ins, const char* name) {
  for (int o = 0; o < n_outs; ++o) {
    const Operand* met = nullptr;
    for (int p = o; p < n_outs && !met; ++p)
      if (operands_meet(outs[o], outs[p])) met = &outs[p];
    for (int i = 0; i < n_ins && !met; ++i)
      if (operands_meet(outs[o], ins[i])) met = &ins[i];
    if (met) return set_error(TTL_ERR_ARG, "%s: the output %s shares memory with %s", name, outs[o].name, met->name);
  }
  return TTL_OK;
}

}  // namespace ttl
