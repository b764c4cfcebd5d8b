// Packed causal attention: what its kernels share.  A pack is one axis of T tokens; document b holds
// tokens [cu[b], cu[b+1]) and a query sees the keys of its own document up to itself.
#pragma once

#include <cmath>

#include "launch_after.cuh"
#include "pack_docs.h"
#include "ttl_device.cuh"
#include "ttl_internal.h"

namespace ttl {

// One shard's operands.  Head c of a row-major [T, heads d] matrix starts at column c d.
struct PackShard {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* o;            // forward: out; backward: in
  float* lse;                  // [n_q/t, T], natural logarithm; forward: out; backward: in
  const __nv_bfloat16* dO;
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
};

struct PackArgs {
  PackShard s[kMaxShards];
  int t, nql, nkvl, grp;       // query and KV heads per shard, query heads per KV head
  int64_t T;
  int64_t ldq, ldk, ldv, ldo, lddo, lddq, lddk, lddv;
  const int32_t* cu;           // [batch + 1]
  int batch;
  float scale;
  float* D;                    // backward: rowsum(dO o), [t][n_q/t][T]
  int* status;
  // Work lists, heaviest first, written by the plan kernel (null: the kernels look their items up)
  const int4* q_list;          // one word a query unit, below
  const int4* kv_list;         // two words a key unit, below
  const int* kv_head;          // [0] entries of kv_list, [1] key tiles in join_list
  int* q_taken;                // items of a list that blocks took beyond their first; 0 at the start
  int* kv_taken;
  const int4* join_list;       // {key tile, first slot, parts, 0} of the key tiles that several items share
  float* part;                 // partial dK and dV: [slot * KV heads + head][2][128][d]
};

// A query unit: {unit, first key tile of its first token tile, of its second, 0}, -1 for a token tile without
// keys; a tile's last key tile is its own.
// A key unit: {key tile, last query tile, first step, end step} {slot of its partial sums or -1, 0, 0, 0}.

// The operands that both kernels of the backward pass load, in boxes of 64 x 128, made once for both.
struct PackMaps {
  CUtensorMap q[kMaxShards], k[kMaxShards], v[kMaxShards], dO[kMaxShards];
};

// What the plan kernel writes for a launch (null: not wanted).
struct PackPlan {
  int4* q_list;
  int q_units, q_per;          // token tiles per query unit
  int* q_taken;
  int4* kv_list;
  int* kv_head;
  int* kv_taken;
  int4* join_list;
  int tiles, lanes;            // key tiles; KV heads over all shards
  int split;                   // key tiles may be cut into several items
};
constexpr int kSplitItems = 456;   // items a cut aims at in all: three for each of 152 SMs
constexpr int kSplitSteps = 8;     // and no shorter than this
// d > 0: the launch also takes A.D.
int pack_attn_plan_launch(const PackArgs& A, const PackPlan& plan, int d, cudaStream_t stream);
int pack_attn_join_launch(const PackArgs& A, int d, cudaStream_t stream);
// Whether key tiles may be cut: few items, and long enough ones.  With eight items or more for each SM the
// list's order alone evens the SMs out.
inline bool pack_split(int64_t tiles, int lanes, int grp) {
  return tiles * lanes < 8 * 152 && tiles * grp > 2 * kSplitSteps;
}

// Raises a kernel's dynamic shared-memory limit, once per kernel and device (thread-safe).
enum PackKernelSlot { kPackFwd128, kPackFwd64, kPackDq128, kPackDq64, kPackDkv128, kPackDkv64, kPackKernelSlots };
int set_core_smem_once(const void* fn, int slot, int bytes, const char* what);

// Launches of the tensor-core kernels (arguments are checked; A.s holds every pointer they need).
// `list`: room for one word of 16 bytes per 128 tokens and one more.
int pack_attn_fwd_launch(const PackArgs& A, int d, void* list, cudaStream_t stream);
int pack_attn_dq_launch(const PackArgs& A, const PackMaps& maps, int d, cudaStream_t stream);    // dQ, after D
int pack_attn_dkv_launch(const PackArgs& A, const PackMaps& maps, int d, cudaStream_t stream);   // dK and dV, after D

constexpr int kTile = 128;       // tokens per query or key tile
constexpr int kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// doc_of for one token of a document (0 <= tok < T, cu[0] <= tok < cu[batch]), by a whole warp: 32 bounds at a time.
__device__ __forceinline__ DocRange doc_of_warp(const int32_t* cu, int batch, int T, int tok) {
  const int lane = threadIdx.x & 31;
  int l = 0, r = batch;
  while (r - l > 1) {
    const int step = (r - l - 1 + 31) / 32;
    const int at = l + step * (lane + 1);
    const unsigned le = __ballot_sync(0xffffffffu, at < r && __ldg(cu + at) <= tok);
    const int n = le == 0xffffffffu ? 32 : __ffs(~le) - 1;
    l += step * n;
    r = r < l + step ? r : l + step;
  }
  const int lo = __ldg(cu + l), hi = __ldg(cu + r);
  return DocRange{lo < 0 ? 0 : lo, hi > T ? T : hi};
}

// Reports cu that does not start at 0 or above, decreases, or ends beyond T.
__device__ __forceinline__ void check_docs(const int32_t* cu, int batch, int64_t T, int* status) {
  bool bad = false;
  for (int b = threadIdx.x; b <= batch; b += blockDim.x) {
    const int c = __ldg(cu + b);
    bad |= c < 0 || c > T || (b > 0 && __ldg(cu + b - 1) > c);
  }
  if (bad) atomicCAS(status, 0, TTL_ERR_DEVICE);
}

// mbar_wait with its polling loop out of line: these kernels wait in some thirty places, and the loop's code
// in each of them would crowd the instruction cache at every change of item.
static __device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, volatile int* abort, int* status,
                                                uint64_t timeout_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i) {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(bar), "r"(parity)
          : "memory");
      if (ok) return true;
    }
    if (*abort) return false;
    if (globaltimer_ns() - t0 > timeout_ns) {
      if (status) atomicCAS(status, 0, TTL_ERR_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort, int* status,
                                        uint64_t timeout_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_longer(smem_u32(bar), parity, abort, status, timeout_ns);
}

// The items of a persistent block after its first, announced by one of its warps and read by the others.  Blocks
// take items from the work list, heaviest first, as they get to them.  One is taken kLead tiles before the loads
// of the one before end: early enough that its documents are looked up by then, late enough that a block which
// ends first finds items left.
constexpr int kLead = 2;
constexpr int kAhead = 4;        // items announced and not yet read
constexpr int kQueueBars = 2 * kAhead;
template <class Item>
struct ItemQueue {
  Item* items;                   // [kAhead], shared memory; shard < 0: no more items
  uint64_t* bars;                // [kQueueBars]
  volatile int* abort;
  int* status;
  uint64_t timeout_ns;

  __device__ __forceinline__ void init(int readers) const {
    for (int a = 0; a < kAhead; ++a) {
      mbar_init(&bars[a], 1);
      mbar_init(&bars[kAhead + a], readers);
    }
  }
  // The n-th item (n >= 1), by one lane; false where the wait for its place ran out.
  __device__ __forceinline__ bool announce(int n, const Item& it) const {
    const int a = (n - 1) % kAhead;
    if (!wait_on(&bars[kAhead + a], (static_cast<uint32_t>((n - 1) / kAhead) & 1u) ^ 1u, abort, status, timeout_ns)) return false;
    items[a] = it;
    mbar_arrive(&bars[a]);
    return true;
  }
  // The n-th item (n >= 1), by a whole warp; false where the wait ran out.
  __device__ __forceinline__ bool next(int n, Item& it) const {
    if (n == 0) return true;     // (the first one each warp finds by itself)
    const int a = (n - 1) % kAhead;
    const bool in_time = wait_on(&bars[a], static_cast<uint32_t>((n - 1) / kAhead) & 1u, abort, status, timeout_ns);
    if (!__all_sync(0xffffffffu, in_time)) return false;
    it = items[a];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bars[kAhead + a]);
    return true;
  }
};

// The warp's index as a value the compiler knows to be the same in all lanes: descriptors computed from it and
// from loop counters stay in uniform registers, which is where the MMA instruction takes them from.
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0); }

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

// 32 lanes x 32 bits, 16 consecutive columns from registers.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Bits [a, b] of a word, for any a and b (none where b < a).
__device__ __forceinline__ uint32_t bits_between(int a, int b) {
  const int lo = a < 0 ? 0 : (a > 32 ? 32 : a), hi = b < -1 ? -1 : (b > 31 ? 31 : b);
  uint32_t m;
  asm("bmsk.clamp.b32 %0, %1, %2;" : "=r"(m) : "r"(lo), "r"(hi < lo ? 0 : hi - lo + 1));
  return m;
}

// 32 fp32 bit patterns of a row as bf16 to 64 bytes of global memory: whole 32-byte sectors where the row allows.
__device__ __forceinline__ void store_bf16x32(__nv_bfloat16* out, const uint32_t (&o)[32]) {
  uint32_t w[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
  if ((reinterpret_cast<uintptr_t>(out) & 31) == 0) {
    st_global_v8(out, w);
    st_global_v8(out + 16, w + 8);
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *reinterpret_cast<uint4*>(out + u * 8) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
  }
}

// ------------------------------------------------------------------ one row by one warp
// Lane l holds columns [l D/32, (l + 1) D/32) of the head.  Every key or query of the range is read, and
// nothing outside it, so what masked places hold (infinities, NaN) never enters.

template <int D>
struct RowVec {
  float x[D / 32];
};

template <int D>
__device__ __forceinline__ RowVec<D> row_load(const __nv_bfloat16* p, int lane) {
  RowVec<D> r;
  if constexpr (D == 128) {
    const uint2 w = *reinterpret_cast<const uint2*>(p + lane * 4);
    r.x[0] = bf16_lo(w.x); r.x[1] = bf16_hi(w.x); r.x[2] = bf16_lo(w.y); r.x[3] = bf16_hi(w.y);
  } else {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p + lane * 2);
    r.x[0] = bf16_lo(w); r.x[1] = bf16_hi(w);
  }
  return r;
}

template <int D>
__device__ __forceinline__ void row_store(__nv_bfloat16* p, const RowVec<D>& r, int lane) {
  if constexpr (D == 128)
    *reinterpret_cast<uint2*>(p + lane * 4) = make_uint2(pack_bf16x2(r.x[0], r.x[1]), pack_bf16x2(r.x[2], r.x[3]));
  else
    *reinterpret_cast<uint32_t*>(p + lane * 2) = pack_bf16x2(r.x[0], r.x[1]);
}

template <int D>
__device__ __forceinline__ float row_dot(const RowVec<D>& a, const RowVec<D>& b) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) s = fmaf(a.x[j], b.x[j], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <int D>
__device__ __forceinline__ RowVec<D> row_zero() {
  RowVec<D> r;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) r.x[j] = 0.0f;
  return r;
}

// o_i and lse_i of query head c at token i: running maximum m and sum l, both in base 2.
template <int D>
__device__ __forceinline__ void fwd_row(const PackArgs& A, const PackShard& S, int c, int i, DocRange doc, int lane) {
  const int g = c / A.grp;
  RowVec<D> acc = row_zero<D>();
  float lse = -INFINITY;
  if (doc.hi > doc.lo) {
    const RowVec<D> q = row_load<D>(S.q + i * A.ldq + c * D, lane);
    const float k2 = A.scale * kLog2e;
    float m = -INFINITY, l = 0.0f;
    for (int j = doc.lo; j <= i; ++j) {
      const float s = row_dot(q, row_load<D>(S.k + j * A.ldk + g * D, lane)) * k2;
      const RowVec<D> v = row_load<D>(S.v + j * A.ldv + g * D, lane);
      const float mn = fmaxf(m, s);
      const float f = m == -INFINITY ? 0.0f : exp2f(m - mn), p = exp2f(s - mn);
      l = l * f + p;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) acc.x[e] = fmaf(acc.x[e], f, p * v.x[e]);
      m = mn;
    }
    const float inv = 1.0f / l;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc.x[e] *= inv;
    lse = (m + log2f(l)) * kLn2;
  }
  row_store<D>(S.o + i * A.ldo + c * D, acc, lane);
  if (lane == 0) S.lse[static_cast<int64_t>(c) * A.T + i] = lse;
}

// dq_i of query head c.
template <int D>
__device__ __forceinline__ void dq_row(const PackArgs& A, const PackShard& S, int shard, int c, int i, DocRange doc,
                                       int lane) {
  const int g = c / A.grp;
  RowVec<D> acc = row_zero<D>();
  if (doc.hi > doc.lo) {
    const RowVec<D> q = row_load<D>(S.q + i * A.ldq + c * D, lane);
    const RowVec<D> go = row_load<D>(S.dO + i * A.lddo + c * D, lane);
    const float Di = A.D[(static_cast<int64_t>(shard) * A.nql + c) * A.T + i];
    const float k2 = A.scale * kLog2e, lse2 = S.lse[static_cast<int64_t>(c) * A.T + i] * kLog2e;
    for (int j = doc.lo; j <= i; ++j) {
      const RowVec<D> k = row_load<D>(S.k + j * A.ldk + g * D, lane);
      const float p = exp2f(row_dot(q, k) * k2 - lse2);
      const float dp = row_dot(go, row_load<D>(S.v + j * A.ldv + g * D, lane));
      const float ds = p * (dp - Di) * A.scale;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) acc.x[e] = fmaf(ds, k.x[e], acc.x[e]);
    }
  }
  row_store<D>(S.dq + i * A.lddq + c * D, acc, lane);
}

// dk_j (want_k) or dv_j of KV head g, summed over the group's query heads.
template <int D>
__device__ __forceinline__ void dkv_row(const PackArgs& A, const PackShard& S, int shard, int g, int j, DocRange doc,
                                        bool want_k, int lane) {
  RowVec<D> acc = row_zero<D>();
  if (doc.hi > doc.lo) {
    const RowVec<D> k = row_load<D>(S.k + j * A.ldk + g * D, lane);
    const RowVec<D> v = row_load<D>(S.v + j * A.ldv + g * D, lane);
    const float k2 = A.scale * kLog2e;
    for (int c = g * A.grp; c < (g + 1) * A.grp; ++c)
      for (int i = j; i < doc.hi; ++i) {
        const RowVec<D> q = row_load<D>(S.q + i * A.ldq + c * D, lane);
        const RowVec<D> go = row_load<D>(S.dO + i * A.lddo + c * D, lane);
        const float p = exp2f(row_dot(q, k) * k2 - S.lse[static_cast<int64_t>(c) * A.T + i] * kLog2e);
        const float ds = p * (row_dot(go, v) - A.D[(static_cast<int64_t>(shard) * A.nql + c) * A.T + i]) * A.scale;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc.x[e] = want_k ? fmaf(ds, q.x[e], acc.x[e]) : fmaf(p, go.x[e], acc.x[e]);
      }
  }
  row_store<D>((want_k ? S.dk + j * A.lddk : S.dv + j * A.lddv) + g * D, acc, lane);
}

}  // namespace ttl
