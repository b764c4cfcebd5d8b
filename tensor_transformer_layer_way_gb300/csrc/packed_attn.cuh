// Packed causal attention: what its kernels share.  A pack is one axis of T tokens; document b holds
// tokens [cu[b], cu[b+1]) and a query sees the keys of its own document up to itself, or with a window the last
// `window` of these and the document's first `sinks`.
#pragma once

#include <cmath>
#include <type_traits>

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
  int window, sinks;           // window 0: none
  float* D;                    // backward: rowsum(dO o), [t][n_q/t][T]
  int* status;
  // Work lists, heaviest first, written by the plan kernel (null: the kernels look their items up)
  const int4* q_list;          // one word a query unit, below
  const int4* kv_list;         // two words a key unit, below
  const int* kv_head;          // [0] entries of kv_list, [1] key tiles in join_list
  int* q_taken;                // items of a list that blocks took beyond their first; 0 at the start
  int* kv_taken;
  const int4* join_list;       // {key tile, first slot, parts, 0} of the key tiles that several items share
  const struct KvShares* kv_shares;   // with a window, beside kv_list: the work as one line, cut evenly
  float* part;                 // partial dK and dV: [slot * KV heads + head][2][128][d]
  struct RedoEntry* redo;      // room for the rows that are computed again
};

// The key tiles of all KV heads, one head's after the other's, as a line of steps: tile t of a head lies at
// [before[t], before[t + 1]), its own cost tile_cost(d) first and then its steps.  Block b of the launch works on an even share
// [b total / blocks, (b + 1) total / blocks) of the line.  A tile that a border cuts is summed in parts: block b's
// part of a tile that it continues has slot 2 b, of one that it begins and does not end slot 2 b + 1.
struct KvShares {
  long long head, total;       // a KV head's length, and all of them
  int blocks, joins;           // 0 blocks: whole tiles from kv_list; cut tiles, in join_list: {key tile, slot of the first
                               // part, parts, KV head}
  int4 first[152];             // {KV head, key tile} where a block's share begins
};
constexpr int kShareBlocks = 152;
// Of a tile beside its steps, in steps (measured: 8400 to 10400 of 2700 cycles, heads of 64 4800 of 3000).
__host__ __device__ constexpr int tile_cost(int d) { return d == 128 ? 4 : 2; }
constexpr int kLeastShare = 6; // and what a share is not cut below

// A query unit: {unit, first key tile of its first token tile, of its second, 0}, -1 for a token tile without
// keys; a tile's last key tile is its own.  With a window, in place of a first key tile: the first token of the
// document that the token tile begins in.
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
  KvShares* kv_shares;
  long long* kv_before;        // [tiles + 1], behind kv_shares
  int share_blocks;            // blocks of the dK, dV launch
  int cost;                    // tile_cost
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
// Pairs of a query and a key that it sees, in one document of T tokens (the lengths are on the device).
inline double pack_pairs(const PackArgs& A) {
  const double T = static_cast<double>(A.T), W = A.window ? A.window : T;
  if (W >= T) return T * (T + 1) / 2;
  return W * (W + 1) / 2 + (T - W) * (W + (A.sinks < T - W ? A.sinks : T - W));
}

// Launches of the tensor-core kernels (arguments are checked; A.s holds every pointer they need).
// `list`: room for one word of 16 bytes per 128 tokens and one more; A.redo: for 4 words of 8 bytes per 128 tokens and
// query head (backward: and twice as many per KV head, if that is more).
int pack_attn_fwd_launch(const PackArgs& A, int d, void* list, cudaStream_t stream);
int pack_attn_dq_launch(const PackArgs& A, const PackMaps& maps, int d, cudaStream_t stream);    // dQ, after D
int pack_attn_dkv_launch(const PackArgs& A, const PackMaps& maps, int d, cudaStream_t stream);   // dK and dV, after D

template <int D>
using Width = std::integral_constant<int, D>;   // a head's width, as an argument

constexpr int kTile = 128;       // tokens per query or key tile
constexpr int kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// With a window: whether the key tiles' work is dealt out in even shares.  Not where every tile has a block of its own and the
// longest (of one document) is no longer than about a share, or short: a cut costs the write and the sum of its parts.
inline bool pack_shares(int64_t tiles, int lanes, int grp, int window, int sinks) {
  const int64_t seen = (window + kTile - 2) / kTile + 1;            // query tiles that see a key tile
  const int64_t usual = (seen < tiles ? seen : tiles) * grp, longest = sinks > 0 ? tiles * grp : usual;
  return tiles * lanes > kShareBlocks ||
         (longest > 2 * kSplitSteps && 3 * longest * kShareBlocks > 4 * tiles * lanes * usual);
}

// ---- windows
// With a window (W) the query at token i of a document that begins at lo sees the keys [near, i] and, before these, the
// sinks [lo, sink), sink <= near.  (window and sinks are at most T, below 2^28: no sum of theirs leaves 32 bits.)
__device__ __forceinline__ int near_key(const PackArgs& A, int lo, int i) { return max(lo, i - A.window + 1); }
__device__ __forceinline__ int sink_end(const PackArgs& A, int lo, int near) { return min(lo + A.sinks, near); }

// The key tiles of the query tile at q0 whose first row's document begins at token lo: [beg, gap) with its sinks and
// [wbeg, q0 / kTile]; other documents begin in the tile itself.  Neighbours are one range: gap = wbeg then.
struct TileRange {
  int beg, gap, wbeg;
};
__device__ __forceinline__ TileRange key_tiles(const PackArgs& A, int q0, int lo) {
  TileRange r;
  r.wbeg = near_key(A, lo, q0) / kTile;
  r.beg = A.sinks > 0 ? lo / kTile : r.wbeg;
  r.gap = A.sinks > 0 ? min((lo + A.sinks - 1) / kTile + 1, r.wbeg) : r.wbeg;
  return r;
}
// The part of a work item that only windows have: key tiles [.., gap) and [wbeg, ..).
template <bool W>
struct Gap {};
template <>
struct Gap<true> {
  int gap, wbeg;
};
// The item's key tile behind tile j.
template <bool W>
__device__ __forceinline__ int tile_after(const Gap<W>& it, int j) {
  if constexpr (W) {
    if (j + 1 == it.gap) return it.wbeg;
  }
  return j + 1;
}

// One past the last query that sees the key at token j of the document `doc`.
template <bool W>
__device__ __forceinline__ int query_end(const PackArgs& A, const DocRange& doc, int j) {
  if constexpr (W) {
    if (j - doc.lo >= A.sinks) return min(doc.hi, j + A.window);
  }
  return doc.hi;
}
// The last query tile that sees a key of tile k0 whose last token, v1 - 1, is of the document `doc`: documents that
// end in the tile are seen from there.
template <bool W>
__device__ __forceinline__ int last_query_tile(const PackArgs& A, const DocRange& doc, int k0, int v1) {
  // with a window: from the tile's last token, unless the document's sinks reach into the tile
  const int hi = query_end<W>(A, doc, W && max(k0, doc.lo) - doc.lo < A.sinks ? doc.lo : v1 - 1);
  return (hi > v1 ? hi - 1 : v1 - 1) / kTile;
}

// doc_of for one token of a document (0 <= tok < T, cu[0] <= tok < cu[batch]), by a whole warp: 32 bounds at a time.
// Beside the range, the document's number.
struct DocAt {
  DocRange range;
  int doc;
};
__device__ __forceinline__ DocAt doc_at_warp(const int32_t* cu, int batch, int T, int tok) {
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
  return DocAt{DocRange{lo < 0 ? 0 : lo, hi > T ? T : hi}, l};
}
__device__ __forceinline__ DocRange doc_of_warp(const int32_t* cu, int batch, int T, int tok) {
  return doc_at_warp(cu, batch, T, tok).range;
}

// Lane l has read the bound c of number b + l, all of them below `end`.  The number, b at least, that 32 stand before the next to
// read: where all are the same, of documents without tokens, the rest of the run is passed by bisection.  (Out of line: rare, and
// its code in the kernels cost them 2%.)
static __device__ __noinline__ int pass_empty(const int32_t* cu, int batch, int b, int c, int end) {
  const int least = __shfl_sync(0xffffffffu, c, 0);
  if (least != __shfl_sync(0xffffffffu, c, 31)) return b;
  return max(b, doc_at_warp(cu, batch, end, least).doc - 31);
}

// Bit r of begins: a document begins at row r of the tile at q0, v0 < q0 + r < v1, where token v0 is of document `doc`.  By
// a whole warp: 32 bounds at a time.  (A row's own bisection each took 2000 to 4000 cycles for the tile.)
__device__ __forceinline__ void begins_in_tile(const int32_t* cu, int batch, int doc, int q0, int v0, int v1,
                                               uint32_t (&begins)[4]) {
  const int lane = threadIdx.x & 31;
  bool go = true;
  for (int b = doc + 1; go; b += 32) {
    const int c = b + lane <= batch ? __ldg(cu + b + lane) : v1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = c - q0 - u * 32;
      begins[u] |= __reduce_or_sync(0xffffffffu, c > v0 && c < v1 && r >= 0 && r < 32 ? 1u << r : 0u);
    }
    go = __all_sync(0xffffffffu, c < v1);
    if (go) b = pass_empty(cu, batch, b, c, v1);
  }
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

// Bit e of a word as a mask of element e: bit 8 j + k stands in the sign of byte j of the word shifted left by 7 - k, which
// one byte permutation spreads.
struct SeenBits {
  uint32_t y[8];
  __device__ __forceinline__ explicit SeenBits(uint32_t see) {
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = see << (7 - k);
  }
  __device__ __forceinline__ static uint32_t spread(uint32_t a, uint32_t b, uint32_t select) {
    uint32_t m;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(m) : "r"(a), "r"(b), "r"(select));
    return m;
  }
  // Elements e (even) and e + 1 as halves of a word.
  __device__ __forceinline__ uint32_t pair(int e) const {
    return spread(y[e & 7], y[(e & 7) + 1], 0xcc88u + 0x1111u * static_cast<uint32_t>(e >> 3));
  }
};
// Makes the hidden ones of 32 bf16 values 0.
__device__ __forceinline__ void hide_pairs(uint32_t (&pk)[16], uint32_t see) {
  const SeenBits seen(see);
#pragma unroll
  for (int e = 0; e < 32; e += 2) pk[e >> 1] &= seen.pair(e);
}

// A row's 32 values times f, or 0 where the row is none (`all`: every row of the warp is one); bad becomes NaN in both
// halves' sum with the first that is not finite.
__device__ __forceinline__ void scale_row(uint32_t (&o)[32], float f, bool in, bool all, uint64_t& bad) {
  if (!all && !in) {
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = 0;
  }
  const uint64_t f2 = f2_pack(f, f);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const uint64_t v = fmul2(f2_pack(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), f2);
    bad = ffma2(v, 0, bad);
    const float2 w = f2_unpack(v);
    o[e] = __float_as_uint(w.x);
    o[e + 1] = __float_as_uint(w.y);
  }
}
__device__ __forceinline__ bool is_bad(uint64_t bad) {
  const float2 b = f2_unpack(bad);
  return b.x + b.y != 0.0f;
}

// 32 rows of 32 fp32 values, a row a thread, as bf16 to rows of stride ld (16-byte aligned), of which the first `rows`
// exist.  Groups of four lanes exchange their rows' 16-byte words, so that a store instruction covers 64 bytes of
// eight rows.  (32 bytes of 32 rows at a time: 84 cycles an instruction, 2700 for a query tile's dQ of 128 columns.)
__device__ __forceinline__ void store_rows_bf16x32(__nv_bfloat16* at, int64_t ld, int rows, const uint32_t (&o)[32]) {
  const int lane = threadIdx.x & 31;
  uint32_t w[4][4];                    // word q of the lane's row; then of row 4 (lane / 4) + q the lane's word
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e >> 2][e & 3] = pack_bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
#pragma unroll
  for (int far = 1; far <= 2; far <<= 1) {
    const bool up = lane & far;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q & far) continue;           // places q and q + far
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[q][e] : w[q + far][e], far);
        if (up) w[q][e] = got;
        else w[q + far][e] = got;
      }
    }
  }
  at += (lane & 3) * 8;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int row = (lane & ~3) + q;
    if (row < rows) *reinterpret_cast<uint4*>(at + row * ld) = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
  }
}

// ------------------------------------------------------------------ rows that are computed again
// A masked place enters a product as 0, and 0 times an infinite or NaN value is NaN, so a row whose result is not
// finite may owe that to places that it does not see.  A block lists such rows while it runs and computes them again
// when its items are done, from what they see alone: nothing waits for that, however long it takes.  It is only
// done where a masked place of the row's first or last tile (no other tile has places that it does not see) holds such
// a value: a row that is not finite by what it sees keeps the product's result.
// Measured, 8192 tokens in 12 documents, 32 and 8 heads of 128 over 8 shards (129 us forward, 329 us backward, calls one at a
// time): one NaN inside the longest document 0.8 and 1.9 to 3.5 ms, NaN in all rows behind the documents 0.4 and 14 ms; row
// by row at the end of the item they took 23, 72 to 100, 4.2 and 80 ms.

// Rows [32 slot', 32 slot' + 32) of one head: which of them, and the block's next listed slot.
struct RedoEntry {
  uint32_t rows, next;
};
constexpr uint32_t kRedoNone = 0xffffffffu;
__host__ __device__ __forceinline__ uint32_t redo_slots(int heads, int64_t T) {
  return static_cast<uint32_t>(heads) * static_cast<uint32_t>((T + kTile - 1) / kTile) * 4u;
}
// Slot of rows [q0 + 32 quad, + 32) of head `head` (over all shards; dK and dV: of two heads per KV head).
__device__ __forceinline__ uint32_t redo_slot(int head, int64_t T, int q0, int quad) {
  return redo_slots(head, T) + static_cast<uint32_t>(q0 / kTile) * 4u + static_cast<uint32_t>(quad);
}
struct RedoPlace {
  int head, row0;
};
__device__ __forceinline__ RedoPlace redo_place(uint32_t slot, int64_t T) {
  const uint32_t groups = redo_slots(1, T);
  return RedoPlace{static_cast<int>(slot / groups), static_cast<int>(slot % groups) * 32};
}
// A block's list: the slot listed last and how many were, in shared memory.  The walk ends by the count and at a
// slot that there is not, whatever the entries hold (a workspace that two calls write at once).
struct RedoList {
  uint32_t head, count;
};
// By one lane.
__device__ __forceinline__ void redo_later(RedoEntry* entries, RedoList* list, uint32_t slot, uint32_t rows) {
  entries[slot] = RedoEntry{rows, atomicExch(&list->head, slot)};
  atomicAdd(&list->count, 1u);
}
// Up to R of the rows in `mask`, taken out of it, as numbers from row0; the last one again where there are fewer.
template <int R>
__device__ __forceinline__ int redo_take(uint32_t& mask, int row0, int (&i)[R]) {
  int n = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (mask) {
      i[r] = row0 + __ffs(mask) - 1;
      mask &= mask - 1;
      ++n;
    } else {
      i[r] = i[r > 0 ? r - 1 : 0];
    }
  }
  return n;
}

// Up to R query rows in `mask`, taken out of it.  With a window those of one document: between the sinks (or windows) of two lies
// the length of a document that none of the rows sees.
template <bool W, int R>
__device__ __forceinline__ void redo_take_queries(const PackArgs& A, uint32_t& mask, int row0, int (&i)[R]) {
  if constexpr (W) {
    const int at = __ffs(mask) - 1;
    const DocRange doc = doc_of(A.cu, A.batch, static_cast<int>(A.T), row0 + at);
    uint32_t same = mask & (bits_between(doc.lo - row0, doc.hi - 1 - row0) | 1u << at);
    mask &= ~same;
    redo_take(same, row0, i);
    mask |= same;
  } else {
    redo_take(mask, row0, i);
  }
}

// The work of one warp: kRedoRows rows together, 32 keys (or queries) at a time.  A lane takes the scores of one of
// them, and lane l sums columns [l D/32, (l + 1) D/32) of the results.  The rows' ranges differ by a few places (or,
// without a window, a document); what a row does not see is left out of its sums, not multiplied by 0.
constexpr int kRedoRows = 4;

template <int D>
struct RowVec {
  float x[D / 32];
};

template <int D>
__device__ __forceinline__ void row_store(__nv_bfloat16* p, const RowVec<D>& r, int lane) {
  if constexpr (D == 128)
    *reinterpret_cast<uint2*>(p + lane * 4) = make_uint2(pack_bf16x2(r.x[0], r.x[1]), pack_bf16x2(r.x[2], r.x[3]));
  else
    *reinterpret_cast<uint32_t*>(p + lane * 2) = pack_bf16x2(r.x[0], r.x[1]);
}

template <int D>
__device__ __forceinline__ RowVec<D> row_zero() {
  RowVec<D> r;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) r.x[j] = 0.0f;
  return r;
}

// s[r] = a[r] . b by one lane, rows of D values (a is the same in all lanes).  (Eight lanes to a row, whose loads take whole
// lines, were no faster: the instructions of the products bound it.)
template <int D, int R>
__device__ __forceinline__ void lane_dots(float (&s)[R], const __nv_bfloat16* const (&a)[R], const __nv_bfloat16* b) {
#pragma unroll
  for (int r = 0; r < R; ++r) s[r] = 0.0f;
#pragma unroll 2
  for (int u = 0; u < D; u += 8) {
    const uint4 y = __ldg(reinterpret_cast<const uint4*>(b + u));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(a[r] + u));
      s[r] = fmaf(bf16_lo(x.x), bf16_lo(y.x), s[r]);
      s[r] = fmaf(bf16_hi(x.x), bf16_hi(y.x), s[r]);
      s[r] = fmaf(bf16_lo(x.y), bf16_lo(y.y), s[r]);
      s[r] = fmaf(bf16_hi(x.y), bf16_hi(y.y), s[r]);
      s[r] = fmaf(bf16_lo(x.z), bf16_lo(y.z), s[r]);
      s[r] = fmaf(bf16_hi(x.z), bf16_hi(y.z), s[r]);
      s[r] = fmaf(bf16_lo(x.w), bf16_lo(y.w), s[r]);
      s[r] = fmaf(bf16_hi(x.w), bf16_hi(y.w), s[r]);
    }
  }
}

// acc[r] += w[r] of place e times row e of m (row stride ld) for e in [from[r], to[r]); e < n <= 32, lane e holds place
// e's weights.
template <int D, int R>
__device__ __forceinline__ void add_rows(RowVec<D> (&acc)[R], const float (&w)[R], const int (&from)[R], const int (&to)[R],
                                         const __nv_bfloat16* m, int64_t ld, int n, int lane) {
  constexpr int kBatch = 4;     // rows loaded ahead of their products
  using Words = typename std::conditional<D == 128, uint2, uint32_t>::type;
  const __nv_bfloat16* at = m + lane * (D / 32);
#pragma unroll 1
  for (int e0 = 0; e0 < n; e0 += kBatch) {
    Words v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) v[u] = __ldg(reinterpret_cast<const Words*>(at + (e0 + u < n ? e0 + u : n - 1) * ld));
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int e = e0 + u;
      float f[D / 32];
      if constexpr (D == 128) {
        f[0] = bf16_lo(v[u].x); f[1] = bf16_hi(v[u].x); f[2] = bf16_lo(v[u].y); f[3] = bf16_hi(v[u].y);
      } else {
        f[0] = bf16_lo(v[u]); f[1] = bf16_hi(v[u]);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float we = __shfl_sync(0xffffffffu, w[r], e & 31);
        if (e >= from[r] && e < to[r]) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) acc[r].x[c] = fmaf(we, f[c], acc[r].x[c]);
        }
      }
    }
  }
}

// What rows see in turn: part 0 the keys lo..i, or with a window part 0 the sinks and part 1 the window.  Row r sees
// [from[r], to[r]); [begin, end) holds them all.
template <bool W, int R>
__device__ __forceinline__ void row_keys(const PackArgs& A, int part, const int (&i)[R], const int (&lo)[R], int (&from)[R],
                                         int (&to)[R], int& begin, int& end) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    from[r] = lo[r];
    to[r] = i[r] + 1;
    if constexpr (W) {
      const int near = near_key(A, lo[r], i[r]);
      if (part == 0) to[r] = sink_end(A, lo[r], near);
      else from[r] = near;
    }
    begin = r ? min(begin, from[r]) : from[r];
    end = r ? max(end, to[r]) : to[r];
  }
}

// o and lse of query head c at tokens i[0..n), whose documents begin at lo: running maximum m and sum l, in base 2.
template <int D, bool W, int R>
__device__ __forceinline__ void fwd_rows(const PackArgs& A, const PackShard& S, int c, const int (&i)[R], const int (&lo)[R],
                                         int n, int lane) {
  const int g = c / A.grp;
  const float k2 = A.scale * kLog2e;
  RowVec<D> acc[R];
  float m[R], l[R];                                // (l: this lane's part)
  const __nv_bfloat16* q[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    acc[r] = row_zero<D>();
    m[r] = -INFINITY;
    l[r] = 0.0f;
    q[r] = S.q + i[r] * A.ldq + c * D;
  }
#pragma unroll 1
  for (int part = 0; part < (W ? 2 : 1); ++part) {
    int first[R], past[R], begin, end;
    row_keys<W>(A, part, i, lo, first, past, begin, end);
#pragma unroll 1
    for (int j0 = begin; j0 < end; j0 += 32) {
      const int j = j0 + lane;
      float s[R];
      int from[R], to[R];
      lane_dots<D, R>(s, q, S.k + min(j, end - 1) * A.ldk + g * D);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s[r] = j >= first[r] && j < past[r] ? s[r] * k2 : -INFINITY;
        float mn = fmaxf(m[r], s[r]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        const float base = mn == -INFINITY ? 0.0f : mn;
        const float f = exp2f(m[r] - base);
        s[r] = exp2f(s[r] - base);
        l[r] = l[r] * f + s[r];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[r].x[e] *= f;
        m[r] = mn;
        from[r] = first[r] - j0;
        to[r] = past[r] - j0;
      }
      add_rows<D, R>(acc, s, from, to, S.v + j0 * A.ldv + g * D, A.ldv, min(32, end - j0), lane);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
    const float inv = 1.0f / l[r];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[r].x[e] *= inv;
    if (r < n) {
      row_store<D>(S.o + i[r] * A.ldo + c * D, acc[r], lane);
      if (lane == 0) S.lse[static_cast<int64_t>(c) * A.T + i[r]] = (m[r] + log2f(l[r])) * kLn2;
    }
  }
}

// dq of query head c at tokens i[0..n).
template <int D, bool W, int R>
__device__ __forceinline__ void dq_rows(const PackArgs& A, const PackShard& S, int shard, int c, const int (&i)[R],
                                        const int (&lo)[R], int n, int lane) {
  const int g = c / A.grp;
  const float k2 = A.scale * kLog2e;
  RowVec<D> acc[R];
  float lse2[R], Di[R];
  const __nv_bfloat16* q[R];
  const __nv_bfloat16* go[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    acc[r] = row_zero<D>();
    q[r] = S.q + i[r] * A.ldq + c * D;
    go[r] = S.dO + i[r] * A.lddo + c * D;
    lse2[r] = S.lse[static_cast<int64_t>(c) * A.T + i[r]] * kLog2e;
    Di[r] = A.D[(static_cast<int64_t>(shard) * A.nql + c) * A.T + i[r]];
  }
#pragma unroll 1
  for (int part = 0; part < (W ? 2 : 1); ++part) {
    int first[R], past[R], begin, end;
    row_keys<W>(A, part, i, lo, first, past, begin, end);
#pragma unroll 1
    for (int j0 = begin; j0 < end; j0 += 32) {
      const int at = min(j0 + lane, end - 1);
      float s[R], dp[R];
      int from[R], to[R];
      lane_dots<D, R>(s, q, S.k + at * A.ldk + g * D);
      lane_dots<D, R>(dp, go, S.v + at * A.ldv + g * D);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s[r] = exp2f(s[r] * k2 - lse2[r]) * (dp[r] - Di[r]) * A.scale;
        from[r] = first[r] - j0;
        to[r] = past[r] - j0;
      }
      add_rows<D, R>(acc, s, from, to, S.k + j0 * A.ldk + g * D, A.ldk, min(32, end - j0), lane);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (r < n) row_store<D>(S.dq + i[r] * A.lddq + c * D, acc[r], lane);
}

// dk (want_k) or dv of KV head g at tokens j[0..n), seen by the queries j to hi - 1, summed over the group's query heads.
template <int D, int R>
__device__ __forceinline__ void dkv_rows(const PackArgs& A, const PackShard& S, int shard, int g, const int (&j)[R],
                                         const int (&hi)[R], int n, bool want_k, int lane) {
  const float k2 = A.scale * kLog2e;
  RowVec<D> acc[R];
  const __nv_bfloat16* k[R];
  const __nv_bfloat16* v[R];
  int begin = j[0], end = hi[0];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    acc[r] = row_zero<D>();
    k[r] = S.k + j[r] * A.ldk + g * D;
    v[r] = S.v + j[r] * A.ldv + g * D;
    begin = min(begin, j[r]);
    end = max(end, hi[r]);
  }
  for (int c = g * A.grp; c < (g + 1) * A.grp; ++c) {
    const float* lse = S.lse + static_cast<int64_t>(c) * A.T;
    const float* Dr = A.D + (static_cast<int64_t>(shard) * A.nql + c) * A.T;
#pragma unroll 1
    for (int i0 = begin; i0 < end; i0 += 32) {
      const int at = min(i0 + lane, end - 1);
      float w[R];
      int from[R], to[R];
      lane_dots<D, R>(w, k, S.q + at * A.ldq + c * D);
      const float lse2 = lse[at] * kLog2e;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        w[r] = exp2f(w[r] * k2 - lse2);
        from[r] = j[r] - i0;
        to[r] = hi[r] - i0;
      }
      if (want_k) {
        float dp[R];
        lane_dots<D, R>(dp, v, S.dO + at * A.lddo + c * D);
#pragma unroll
        for (int r = 0; r < R; ++r) w[r] *= (dp[r] - Dr[at]) * A.scale;
      }
      const __nv_bfloat16* m = want_k ? S.q + i0 * A.ldq + c * D : S.dO + i0 * A.lddo + c * D;
      add_rows<D, R>(acc, w, from, to, m, want_k ? A.ldq : A.lddo, min(32, end - i0), lane);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (r < n) row_store<D>((want_k ? S.dk + j[r] * A.lddk : S.dv + j[r] * A.lddv) + g * D, acc[r], lane);
}

// ---- what the products of a tile's rows met beside what the rows see

// Bit r: row k0 + r (below T) of some heads' columns holds a value that is not finite.
struct BadRows {
  uint32_t w[4];
  // any row of [a, b), numbered from the tile's first
  __device__ __forceinline__ bool any(int a, int b) const {
    uint32_t hit = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) hit |= w[u] & bits_between(a - u * 32, b - 1 - u * 32);
    return hit != 0;
  }
};
template <int D>
__device__ __forceinline__ void add_bad_rows(BadRows& b, const __nv_bfloat16* m, int64_t ld, int col, int k0, int64_t T, int lane) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = k0 + u * 32 + lane;
    bool bad = false;
    if (i < T) {
      const uint4* p = reinterpret_cast<const uint4*>(m + i * ld + col);
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = __ldg(p + c);
        const uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)     // an exponent of ones
          bad |= (q[e] & 0x7f800000u) == 0x7f800000u || (q[e] & 0x7f80u) == 0x7f80u;
      }
    }
    b.w[u] |= __ballot_sync(0xffffffffu, bad);
  }
}
constexpr int kRedoShort = 2 * kTile;   // rows of fewer places are computed again without that look

// For query rows: m is what the product sums over the keys (V or K).  Keys before row i's document in the first tile,
// keys behind it in its own.  (A row of kRedoShort keys or more belongs to the document of its tile's first row.)
struct QueryEdges {
  BadRows first, own;
  int first0, own0;
  template <int D>
  __device__ __forceinline__ void look(const __nv_bfloat16* m, int64_t ld, int col, int lo, int row0, int64_t T, int lane) {
    first = own = BadRows{{0, 0, 0, 0}};
    first0 = lo / kTile * kTile;
    own0 = row0 / kTile * kTile;
    add_bad_rows<D>(first, m, ld, col, first0, T, lane);
    add_bad_rows<D>(own, m, ld, col, own0, T, lane);
  }
  __device__ __forceinline__ bool met(int lo, int i) const {
    return first.any(0, lo - first0) || own.any(i + 1 - own0, kTile);
  }
};
// For key rows: m is what the product sums over the queries (Q or dO), of the group's heads.  Queries before row j in its
// own tile, queries behind its document in the last one.  (Of kRedoShort queries or more: the tile's last document.)
struct KeyEdges {
  BadRows own, last;
  int own0, last0;
  template <int D>
  __device__ __forceinline__ void look(const PackArgs& A, const PackShard& S, int g, int row0, int hi, bool want_k, int lane) {
    const __nv_bfloat16* m = want_k ? S.q : S.dO;
    const int64_t ld = want_k ? A.ldq : A.lddo;
    own = last = BadRows{{0, 0, 0, 0}};
    own0 = row0 / kTile * kTile;
    last0 = (hi - 1) / kTile * kTile;
    for (int c = g * A.grp; c < (g + 1) * A.grp; ++c) {
      add_bad_rows<D>(own, m, ld, c * D, own0, A.T, lane);
      add_bad_rows<D>(last, m, ld, c * D, last0, A.T, lane);
    }
  }
  __device__ __forceinline__ bool met(int j, int hi) const {
    return own.any(0, j - own0) || last.any(hi - last0, kTile);
  }
};

// The same with a window.  For query rows, masked places are in the tile of the document's first token, the last one with
// sinks, the two that the window of the tile's rows begins in, and the own one.
struct WindowQueryEdges {
  BadRows at[5];
  int k0[5];
  template <int D>
  __device__ __forceinline__ void look(const PackArgs& A, const __nv_bfloat16* m, int64_t ld, int col, int lo, int row0, int lane) {
    const int own = row0 / kTile;
    const TileRange r = key_tiles(A, own * kTile, lo);
    k0[0] = r.beg;
    k0[1] = max(r.beg, r.gap - 1);
    k0[2] = r.wbeg;
    k0[3] = min(r.wbeg + 1, own);
    k0[4] = own;
#pragma unroll 1
    for (int k = 0; k < 5; ++k) {
      k0[k] *= kTile;
      at[k] = BadRows{{0, 0, 0, 0}};
      add_bad_rows<D>(at[k], m, ld, col, k0[k], A.T, lane);
    }
  }
  __device__ __forceinline__ bool met(const PackArgs& A, int lo, int i) const {
    const int near = near_key(A, lo, i), sink = sink_end(A, lo, near);
    uint32_t hit = 0;
#pragma unroll 1
    for (int k = 0; k < 5; ++k)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c0 = k0[k] + u * 32;
        hit |= at[k].w[u] & ~(bits_between(near - c0, i - c0) | bits_between(lo - c0, sink - 1 - c0));
      }
    return hit != 0;
  }
};
// For key rows: queries before row j in its own tile, queries from its end on in the last two that the tile meets (of a key
// that ends before these, beside sinks, without a look).
struct WindowKeyEdges {
  BadRows own, last[2];
  int own0, last0[2];
  template <int D>
  __device__ __forceinline__ void look(const PackArgs& A, const PackShard& S, int g, int row0, bool want_k, int lane) {
    const __nv_bfloat16* m = want_k ? S.q : S.dO;
    const int64_t ld = want_k ? A.ldq : A.lddo;
    own0 = row0 / kTile * kTile;
    const int T = static_cast<int>(A.T), end = min(min(own0 + kTile, __ldg(A.cu + A.batch)), T);
    const int tile = last_query_tile<true>(A, doc_of(A.cu, A.batch, T, end - 1), own0, end);
    last0[0] = max(own0, (tile - 1) * kTile);
    last0[1] = max(own0, tile * kTile);
    own = last[0] = last[1] = BadRows{{0, 0, 0, 0}};
    for (int c = g * A.grp; c < (g + 1) * A.grp; ++c) {
      add_bad_rows<D>(own, m, ld, c * D, own0, A.T, lane);
      add_bad_rows<D>(last[0], m, ld, c * D, last0[0], A.T, lane);
      add_bad_rows<D>(last[1], m, ld, c * D, last0[1], A.T, lane);
    }
  }
  __device__ __forceinline__ bool met(int j, int end) const {
    return end < last0[0] || own.any(0, j - own0) || last[0].any(end - last0[0], kTile) || last[1].any(end - last0[1], kTile);
  }
};
template <bool W>
using QueryLook = typename std::conditional<W, WindowQueryEdges, QueryEdges>::type;
template <bool W>
using KeyLook = typename std::conditional<W, WindowKeyEdges, KeyEdges>::type;

}  // namespace ttl
