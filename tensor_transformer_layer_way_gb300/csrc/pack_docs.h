// The documents of a pack, looked up by token.  Compiles for the device and, without CUDA, for the host, where
// the tests run it over bounds that no kernel should meet.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define TTL_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define TTL_HOST_DEVICE inline
#endif

namespace ttl {

struct DocRange {
  int lo, hi;                  // the document's tokens [lo, hi); hi <= lo: the token is in none
};

TTL_HOST_DEVICE int doc_bound(const int32_t* cu, int b) {
#if defined(__CUDA_ARCH__)
  return __ldg(cu + b);
#else
  return cu[b];
#endif
}

// The document of token `tok` of a pack of T tokens, by bisection of bounds that bound(b) reads.  A token outside [0, T) is in none, also where the
// last document ends beyond T: a tile's rows behind the pack are asked for too.  Whatever cu holds, the answer is
// empty or 0 <= lo <= tok < hi <= T: with entries out of order it is some document cut to the pack (the kernels
// report such entries).
template <class Bound>
TTL_HOST_DEVICE DocRange doc_among(const Bound& bound, int batch, int T, int tok) {
  if (batch == 0 || tok < 0 || tok >= T || tok < bound(0) || tok >= bound(batch)) return DocRange{0, 0};
  int l = 0, r = batch;        // bound(l) <= tok < bound(r)
  while (r - l > 1) {
    const int m = (l + r) >> 1;
    if (bound(m) <= tok) l = m; else r = m;
  }
  const int lo = bound(l), hi = bound(r);
  return DocRange{lo < 0 ? 0 : lo, hi > T ? T : hi};
}
struct DocBounds {
  const int32_t* cu;
  TTL_HOST_DEVICE int operator()(int b) const { return doc_bound(cu, b); }
};
TTL_HOST_DEVICE DocRange doc_of(const int32_t* cu, int batch, int T, int tok) {
  return doc_among(DocBounds{cu}, batch, T, tok);
}

// How long a wait may take, in ns.  Some warps wait for the whole of an item, whose steps (key tiles; for dK and dV query
// tiles times heads of the group) are as many as the longest document makes them: 2 s for a wait that nothing ends, and
// 20 us for each step, twelve times what one takes.
inline uint64_t pack_wait_ns(int64_t steps) { return 2000000000ull + 20000ull * static_cast<uint64_t>(steps); }

}  // namespace ttl
