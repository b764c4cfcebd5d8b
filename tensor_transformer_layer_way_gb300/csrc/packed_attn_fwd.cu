// Forward kernel of packed causal attention on the tensor cores.
//
// The token axis is cut into 128-token tiles wherever documents begin: row i of a query tile
// sees the keys [lo_i, i] of its own document, so a tile's key tiles run from the one that holds the
// first row's lo to its own, and short documents share tiles.  One work item is two query tiles
// that read the same K and V tiles (two heads of a group over the same tokens, or, where the group
// has an odd number of heads, two neighbouring token tiles of one head): every K or V byte loaded
// serves 256 rows, 32 bytes per MMA cycle and SM where one tile alone would need 64.
//
// Per item and key tile, for x in {0, 1}: S_x = Q_x K^T (fp32, tensor memory); one thread per
// row takes the row's maximum, P = 2^(s k - m) as bf16 over S_x's own columns, O_x += P V with P
// read from tensor memory.  The running maximum m only moves when a row's new maximum is more than
// 8 above it (in base 2): P then stays below 2^8, which bf16 and the fp32 sums hold as exactly,
// and the accumulator is rescaled rarely.  The row sum l is taken from the unrounded P.  P is rounded to bf16 once, as
// the product's operands have one type and V is bf16 (error against 64 bits 1.8 to 2.0e-3, with P in fp32 1.5e-3;
// P as two bf16 parts would cost the product twice).
//
// Roles (384 threads, persistent): warp 0 issues the TMA loads (Q_0, Q_1, then K_j, V_j through a ring), warp 1
// the MMAs, warps 2 and 3 look up the coming item and the documents of its rows, warps 4..7 and 8..11 are the
// softmax of tile 0 and 1 and store its result.  A softmax thread holds a whole row of 128 scores: its warpgroups
// take 208 registers a thread and the first leaves with 88 (together the 384 x 168 of the launch).  Per tile x
// the order of MMAs is S_x(j), P_x V(j), S_x(j + 1), and the two tiles alternate, so one tile's softmax runs under
// the other's products; the next item's first S is issued before this item's results are stored.  (A
// warpgroup of its own for the results was slower: it leaves the softmax 176 registers, and a key tile of one
// long document then takes 3200 cycles, with 208 it takes 2700.)
//
// What bounds it: the turn of a tile, 2700 cycles (clock stamps: softmax 1300, product and next scores 1100, the rest
// hand-overs), which the other tile's turn fills up to the products' 2050; tensor memory has no columns left in
// which the next scores could wait.  Measured: one document of 32768 tokens, 4 query heads and 1 KV head of 128: 665 to 705 us,
// 1560 to 1650 TFLOP/s; 8192 tokens in 12 documents, 32 query and 8 KV heads over 8 shards: 94 us (with items
// dealt out beforehand 5 more); 16384 tokens, 8 and 2 heads of 64: 292 us.  With many short documents an
// item costs about 10000 cycles beside its key tiles (masks, the wait for the last product, the result).
//
// A masked place enters the product as P = 0, and 0 times an infinite or NaN value is NaN: a row whose
// result is not finite for that reason is computed again over its own keys alone when the block's items are done.

#include <cstring>
#include <type_traits>

#include "packed_attn.cuh"

namespace ttl {
namespace {

constexpr int kRing = 4;       // (five places were no faster; the fifth's room stages the results)
constexpr int kFwdThreads = 384;
constexpr float kLazy = 8.0f;

struct FwdParams {
  CUtensorMap q[kMaxShards];   // box 64 x 128
  CUtensorMap k[kMaxShards];
  CUtensorMap v[kMaxShards];
  CUtensorMap o[kMaxShards];   // box 64 x 32
  PackArgs a;
  int pair_heads;              // 1: an item is two heads of a group; 0: two token tiles of one head
  int units;                   // token tiles (or pairs of them)
  int lanes;                   // items per unit
  uint64_t timeout_ns;
};

// One query tile of an item: tokens [q0, q0 + 128) of head c, key tiles [jbeg, jend).
struct QTile {
  int c, q0, jbeg, jend;
};
struct Item {
  int shard, g;                // shard < 0: no more items
  QTile x[2];
  int jlo, jhi;                // union of the key tiles
};

template <int D>
struct FwdCfg {
  static constexpr int KB = D / 64;
  static constexpr int TILE = KB * kTile * 128;   // bytes of a Q, K or V tile
  static constexpr int OFF_RING = 2 * TILE;
  static constexpr int OFF_OUT = OFF_RING + kRing * TILE;    // 32 rows x 64 columns of results per softmax warp
  static constexpr int OFF_ROWS = OFF_OUT + 8 * 4096;        // RowDocs [2]
  static constexpr int OFF_BAR = OFF_ROWS + 96;
  static constexpr int SMEM = OFF_BAR + 256 + kAhead * static_cast<int>(sizeof(Item)) + 1024;
  static_assert(SMEM <= 232448, "shared memory beyond the per-CTA limit");
};

// First key tile of the query tile at token q0, or -1; found by the whole warp.
__device__ __forceinline__ int first_key(const PackArgs& A, int q0) {
  const int T = static_cast<int>(A.T);
  if (A.batch == 0) return -1;
  const int first = __ldg(A.cu), last = __ldg(A.cu + A.batch);
  const int v0 = q0 > first ? q0 : first;
  int v1 = q0 + kTile < last ? q0 + kTile : last;
  v1 = v1 < T ? v1 : T;
  return v0 < v1 ? doc_of_warp(A.cu, A.batch, T, v0).lo / kTile : -1;
}

// The item of index `at` whose unit and first keys are e.
__device__ __forceinline__ Item item_from(const FwdParams& P, int at, int4 e) {
  const PackArgs& A = P.a;
  const int lane = at % P.lanes;
  Item it;
  const int per = P.pair_heads ? A.nql / 2 : A.nql;
  it.shard = lane / per;
  const int c = (lane % per) * (P.pair_heads ? 2 : 1);
  it.g = c / A.grp;
  const int t0 = P.pair_heads ? e.x : 2 * e.x;
  auto tile = [&](int head, int t, int first) {
    return QTile{head, t * kTile, first < 0 ? 0 : first, first < 0 ? 0 : t + 1};
  };
  it.x[0] = tile(c, t0, e.y);
  it.x[1] = P.pair_heads ? tile(c + 1, t0, e.y) : tile(c, t0 + 1, e.z);
  const bool a = it.x[0].jend > 0, b = it.x[1].jend > 0;
  it.jlo = a && (!b || it.x[0].jbeg < it.x[1].jbeg) ? it.x[0].jbeg : it.x[1].jbeg;
  it.jhi = b ? it.x[1].jend : it.x[0].jend;
  return it;
}

// A block's first item, found by a whole warp: from the list, or without one the last token tiles first.
__device__ __forceinline__ Item first_item(const FwdParams& P) {
  const PackArgs& A = P.a;
  const int at = static_cast<int>(blockIdx.x);
  if (A.q_list) return item_from(P, at, __ldg(A.q_list + at / P.lanes));
  const int unit = P.units - 1 - at / P.lanes;
  int4 e = make_int4(unit, -1, -1, 0);
  e.y = first_key(A, unit * (P.pair_heads ? 1 : 2) * kTile);
  if (!P.pair_heads) e.z = first_key(A, (unit * 2 + 1) * kTile);
  return item_from(P, at, e);
}

__device__ __forceinline__ bool active(const QTile& q, int j) { return j >= q.jbeg && j < q.jend; }

// A query tile and the documents of its rows: rows [v0, v1) belong to some; the first of them to one that begins at
// token lo, and bit r of `begins` is set where another begins at row r.
struct RowDocs {
  uint32_t begins[4];
  int lo, v0, v1;
  int shard;                   // the tile itself, for the warps that work on it (< 0: no more)
  QTile tile;
};
static_assert(sizeof(RowDocs) == 48, "two of them in 96 bytes");

// First token of row r's document.
__device__ __forceinline__ int first_token(const RowDocs& d, int q0, int r) {
  int w = r >> 5;
  uint32_t m = d.begins[w] & (0xffffffffu >> (31 - (r & 31)));
  while (m == 0 && w > 0) m = d.begins[--w];
  return m ? q0 + w * 32 + 31 - __clz(m) : d.lo;
}

// The listed rows again, by `warps` warps, of which this is number w: the rows of an entry in groups, the groups in turn.
template <int D>
__device__ __noinline__ void redo_rows(const PackArgs& A, RedoList list, int w, int warps, int lane) {
  const uint32_t slots = redo_slots(A.t * A.nql, A.T);
  int turn = 0;
  for (uint32_t slot = list.head; slot < slots && list.count > 0; --list.count) {
    const RedoEntry e = A.redo[slot];
    const RedoPlace at = redo_place(slot, A.T);
    const PackShard& S = A.s[at.head / A.nql];
    const int c = at.head % A.nql;
    QueryEdges edges;
    bool looked = false;
    for (uint32_t rows = e.rows; rows;) {
      int i[kRedoRows], lo[kRedoRows];
      redo_take(rows, at.row0, i);
      if (turn++ % warps != w) continue;
      uint32_t again = 0;
#pragma unroll
      for (int r = 0; r < kRedoRows; ++r) {
        const int first = doc_of(A.cu, A.batch, static_cast<int>(A.T), i[r]).lo;
        bool met = i[r] - first < kRedoShort;
        if (!met) {
          if (!looked) edges.look<D>(S.v, A.ldv, c / A.grp * D, first, at.row0, A.T, lane);
          looked = true;
          met = edges.met(first, i[r]);
        }
        if (met) again |= 1u << (i[r] - at.row0);
      }
      if (again == 0) continue;
      const int n = redo_take(again, at.row0, i);
#pragma unroll
      for (int r = 0; r < kRedoRows; ++r) lo[r] = doc_of(A.cu, A.batch, static_cast<int>(A.T), i[r]).lo;
      fwd_rows<D>(A, S, c, i, lo, n, lane);
    }
    slot = e.next;
  }
}

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 1) pack_fwd_kernel(const __grid_constant__ FwdParams P) {
  using C = FwdCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + C::OFF_RING;
  RowDocs* docs = reinterpret_cast<RowDocs*>(smem + C::OFF_ROWS);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_empty = q_full + 1;
  uint64_t* ring_full = q_empty + 1;
  uint64_t* ring_empty = ring_full + kRing;
  uint64_t* s_full = ring_empty + kRing;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* rows_full = o_full + 2;
  uint64_t* rows_empty = rows_full + 1;
  uint64_t* done_bar = rows_empty + 1;
  uint64_t* item_bars = done_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(item_bars + kQueueBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  RedoList* redo_list = reinterpret_cast<RedoList*>(tmem_slot + 2);
  static_assert((2 + 2 * kRing + 8 + 1 + kQueueBars) * 8 + 16 <= 256, "barrier area");

  const PackArgs& A = P.a;
  const int warp = uniform_warp();
  const int lane = threadIdx.x & 31;
  const int total = P.units * P.lanes;
  int* status = A.status;
  const uint64_t tmo = P.timeout_ns;
  const ItemQueue<Item> queue{reinterpret_cast<Item*>(smem + C::OFF_BAR + 256), item_bars, abort_flag, status, tmo};

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&ring_full[s], 1);
      mbar_init(&ring_empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);   // the tile's four softmax warps
      mbar_init(&o_full[x], 1);
    }
    mbar_init(rows_full, 2);
    mbar_init(rows_empty, 8);
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    *redo_list = RedoList{kRedoNone, 0};
    fence_mbarrier_init();
  }
  if (threadIdx.x == 64) {
    queue.init(3);
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  await_previous();   // the list, and with it whatever ran before it
  if (blockIdx.x == 0) check_docs(A.cu, A.batch, A.T, status);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp == 0) {
    // ------------------------------------------------------------------ TMA loads
    bool ok = true;
    int pos = 0, nq = 0;
    Item it = first_item(P);
    for (int n = 0; lane == 0 && ok && it.shard >= 0; ++n) {
      Item coming = {};
      coming.shard = -1;
      auto announce = [&]() {
        if (A.q_list) {
          const int at = static_cast<int>(gridDim.x) + atomicAdd(A.q_taken, 1);
          if (at < total) coming = item_from(P, at, __ldg(A.q_list + at / P.lanes));
        }
        ok = queue.announce(n + 1, coming);
      };
      const int when = max(it.jlo, it.jhi - kLead);
      if (it.jhi <= it.jlo) {
        announce();
      } else {
        auto load = [&](const CUtensorMap* map, int j) {
          const int slot = pos % kRing;
          if (!wait_on(&ring_empty[slot], (static_cast<uint32_t>(pos / kRing) & 1u) ^ 1u, abort_flag, status, tmo))
            return false;
          mbar_arrive_expect_tx(&ring_full[slot], C::TILE);
          for (int kb = 0; kb < C::KB; ++kb)
            tma_load_2d(sRing + slot * C::TILE + kb * 16384, map, &ring_full[slot], it.g * D + kb * 64, j * kTile);
          ++pos;
          return true;
        };
        // the first K does not wait for the item before to be done with Q
        ok = load(&P.k[it.shard], it.jlo) &&
             wait_on(q_empty, (static_cast<uint32_t>(nq) & 1u) ^ 1u, abort_flag, status, tmo);
        if (ok) {
          const bool two = it.x[1].jend > it.x[1].jbeg, one = it.x[0].jend > it.x[0].jbeg;
          mbar_arrive_expect_tx(q_full, (two ? C::TILE : 0) + (one ? C::TILE : 0));
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (x ? two : one)
              for (int kb = 0; kb < C::KB; ++kb)
                tma_load_2d(sQ + x * C::TILE + kb * 16384, &P.q[it.shard], q_full, it.x[x].c * D + kb * 64, it.x[x].q0);
          ++nq;
        }
        ok = ok && load(&P.v[it.shard], it.jlo);
        if (ok && it.jlo == when) announce();
        for (int j = it.jlo + 1; ok && j < it.jhi; ++j) {
          ok = load(&P.k[it.shard], j) && load(&P.v[it.shard], j);
          if (ok && j == when) announce();
        }
      }
      it = coming;
    }
    if (lane == 0) {
      // No copy may still be landing when the CTA leaves: wait (bounded) for the last loads.
      int dummy = 0;
      volatile int* da = reinterpret_cast<volatile int*>(&dummy);
      if (nq > 0) wait_on(q_full, static_cast<uint32_t>(nq - 1) & 1u, da, status, tmo);
      const int pending = pos < kRing ? pos : kRing;
      for (int i = pos - pending; i < pos; ++i)
        wait_on(&ring_full[i % kRing], static_cast<uint32_t>(i / kRing) & 1u, da, status, tmo);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMAs
    // The whole warp runs this loop, one elected lane issues (4260 -> 2820 cycles per key tile against one lane
    // running it alone, whose every MMA first moved its descriptors to uniform registers).  A wait that runs
    // out is in the status word and raises the abort flag, after which every wait returns at once: the loop
    // then ends over what is in memory.
    int nq = 0, np0 = 0, np1 = 0;
    int slot = 0, lap = 0;                 // ring place of the key tile about to be scored, and its round
    const uint32_t ring0 = smem_u32(sRing);
    const uint64_t qd = smem_desc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t kd0 = smem_desc_sw128(ring0, 16, 1024);
    const uint64_t vd0 = smem_desc_sw128(ring0, 16384, 1024);
    const uint32_t idesc_s = idesc_bf16_f32(kTile, kTile, false, false);
    const uint32_t idesc_o = idesc_bf16_f32(kTile, D, false, true);
    const bool leader = elect_one();
    auto wait = [&](uint64_t* bar, int phase) {
      wait_on(bar, static_cast<uint32_t>(phase) & 1u, abort_flag, status, tmo);
    };
    Item it = first_item(P);
    for (int n = 0; queue.next(n, it) && it.shard >= 0; ++n) {
      if (it.jhi <= it.jlo) continue;
      wait(q_full, nq);
      tc_fence_after_sync();
      ++nq;
      // Step j issues P V of key tile j and then S of key tile j + 1, tile by tile.
      for (int j = it.jlo - 1; j < it.jhi; ++j) {
        // V_j stands one place before K_(j + 1)
        const int ks = slot, vs = slot == 0 ? kRing - 1 : slot - 1;
        if (j >= it.jlo) wait(&ring_full[vs], slot == 0 ? lap - 1 : lap);
        if (j + 1 < it.jhi) wait(&ring_full[ks], lap);
        const uint64_t kd = desc_advance(kd0, ks * C::TILE), vd = desc_advance(vd0, vs * C::TILE);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (active(it.x[x], j)) {
            wait(&p_full[x], x ? np1 : np0);
            if (x) ++np1; else ++np0;
            tc_fence_after_sync();
            const uint32_t more = j > it.x[x].jbeg ? 1u : 0u;
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)
                umma_bf16_ts(tmem + 256 + x * 128, tmem + x * 128 + kk * 8, desc_advance(vd, kk * 2048), idesc_o,
                             kk ? 1u : more);
              if (j + 1 == it.x[x].jend) umma_commit(&o_full[x]);
            }
          }
          if (active(it.x[x], j + 1)) {
            tc_fence_after_sync();
            if (leader) {
#pragma unroll
              for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  umma_bf16(tmem + x * 128, desc_advance(qd, x * C::TILE + kb * 16384 + kk * 32),
                            desc_advance(kd, kb * 16384 + kk * 32), idesc_s, (kb | kk) ? 1u : 0u);
              umma_commit(&s_full[x]);
            }
          }
        }
        if (leader) {
          if (j >= it.jlo) umma_commit(&ring_empty[vs]);
          if (j + 1 < it.jhi) umma_commit(&ring_empty[ks]);
          if (j + 2 == it.jhi) umma_commit(q_empty);   // the last S of the item is issued
        }
        __syncwarp();
        if (j + 1 < it.jhi) {              // on to K_(j + 2), past V_(j + 1)
          slot += 2;
          if (slot >= kRing) {
            slot -= kRing;
            ++lap;
          }
        }
      }
    }
    if (leader) umma_commit(done_bar);   // every MMA issued here must finish before TMEM is released
    __syncwarp();
    int dummy = 0;
    wait_on(done_bar, 0, reinterpret_cast<volatile int*>(&dummy), status, tmo);
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------------------ documents of the rows of tile x
    const int x = warp - 2;
    bool ok = true;
    Item it = first_item(P);
    for (int n = 0; ok && it.shard >= 0 && queue.next(n, it); ++n) {   // (the end is passed on too)
      const QTile qt = x ? it.x[1] : it.x[0];
      RowDocs d = {{0, 0, 0, 0}, 0, 0, 0, it.shard, qt};
      if (qt.jend > qt.jbeg) {
        const int T = static_cast<int>(A.T);
        const int first = __ldg(A.cu), last = min(__ldg(A.cu + A.batch), T);
        d.v0 = max(qt.q0, first);
        d.v1 = min(qt.q0 + kTile, last);
        d.lo = doc_of(A.cu, A.batch, T, d.v0).lo;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = qt.q0 + u * 32 + lane;
          const bool begins = i > d.v0 && i < d.v1 && doc_of(A.cu, A.batch, T, i).lo == i;
          d.begins[u] = __ballot_sync(0xffffffffu, begins);
        }
      }
      ok = wait_on(rows_empty, (static_cast<uint32_t>(n) & 1u) ^ 1u, abort_flag, status, tmo);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) docs[x] = d;
      __syncwarp();
      if (lane == 0) mbar_arrive(rows_full);
    }
  } else {
    // ------------------------------------------------------------------ softmax of tile x
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int quad = warp & 3;
    const int x = (warp - 4) >> 2;
    const int r = quad * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t s_col = lane_base + x * 128, o_col = lane_base + 256 + x * 128;
    uint8_t* stage = smem + C::OFF_OUT + (warp - 4) * 4096;
    const float k2 = A.scale * kLog2e;
    const int T = static_cast<int>(A.T);
    bool ok = true;
    uint32_t ns = 0, no = 0;
    for (int n = 0; ok; ++n) {
      ok = mbar_wait(rows_full, static_cast<uint32_t>(n) & 1u, abort_flag, status, tmo);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      const QTile qt = docs[x].tile;
      const int shard = docs[x].shard;
      if (shard < 0) break;
      const PackShard& S = A.s[shard];
      const int i = qt.q0 + r;
      const bool in = i >= docs[x].v0 && i < docs[x].v1;        // a row of a document (so i < T)
      const int lo = in ? first_token(docs[x], qt.q0, r) : 0x7fffffff, hi = in ? i : -1;   // it sees the keys lo..hi
      __syncwarp();
      if (lane == 0) mbar_arrive(rows_empty);
      const int lo_max = __reduce_max_sync(0xffffffffu, lo), hi_min = __reduce_min_sync(0xffffffffu, hi);
      const int lo_min = __reduce_min_sync(0xffffffffu, lo), hi_max = __reduce_max_sync(0xffffffffu, hi);
      float m = -INFINITY, l = 0.0f;
      for (int j = qt.jbeg; ok && j < qt.jend; ++j) {
        ok = mbar_wait(&s_full[x], ns & 1u, abort_flag, status, tmo);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        ++ns;
        tc_fence_after_sync();
        // A tile that every row of the warp sees whole takes straight-line code; else 32 keys at a time, seen by
        // every row, by some (the others' scores become -inf), or by none (their P is 0 without a look).
        const int k0 = j * kTile;
        auto tile = [&](auto whole) {
          constexpr bool WHOLE = decltype(whole)::value;
          auto live = [&](int u) { return WHOLE || (k0 + u * 32 <= hi_max && k0 + u * 32 + 31 >= lo_min); };
          uint32_t s[4][32];
          auto read_scores = [&]() {
#pragma unroll
            for (int u = 0; u < 4; ++u) tmem_ld_32x32b_x32(s_col + u * 32, s[u]);
            tmem_ld_wait();
            if constexpr (!WHOLE) {
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const int c0 = k0 + u * 32;
                if (live(u) && (c0 < lo_max || c0 + 31 > hi_min)) {
                  const uint32_t see = bits_between(lo - c0, hi - c0);
#pragma unroll
                  for (int e = 0; e < 32; ++e) s[u][e] = (see >> e) & 1u ? s[u][e] : 0xff800000u;
                }
              }
            }
          };
          read_scores();
          float mxs[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            mxs[u] = -INFINITY;
            if (live(u)) {
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                mxs[u] = fmax3(mxs[u], __uint_as_float(s[u][e]), __uint_as_float(s[u][e + 1]));
            }
          }
          const float mx = fmaxf(fmaxf(mxs[0], mxs[1]), fmaxf(mxs[2], mxs[3])) * k2;
          const bool move = mx > m + kLazy || (m == -INFINITY && mx > m);
          if (__any_sync(0xffffffffu, move)) {
            const float mn = move ? mx : m;
            const float f = move ? ex2_approx(m - mn) : 1.0f;
            l *= f;
            m = mn;
            if (j > qt.jbeg) {
              // O_x holds the products up to key tile j - 1: they were issued before S_x(j), which is complete.
#pragma unroll 1
              for (int u = 0; u < D / 32; ++u) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(o_col + u * 32, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st_32x32b_x32(o_col + u * 32, o);
              }
              read_scores();   // again: their registers are O's meanwhile
            }
          }
          const float nm = m == -INFINITY ? 0.0f : -m;
          const uint64_t kk2 = f2_pack(k2, k2), nm2 = f2_pack(nm, nm);
          uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t p[32];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              if (live(2 * h + q)) {
                const uint32_t(&c)[32] = s[2 * h + q];
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                  const float2 a = f2_unpack(ffma2(f2_pack(__uint_as_float(c[e]), __uint_as_float(c[e + 1])), kk2, nm2));
                  const float2 b =
                      f2_unpack(ffma2(f2_pack(__uint_as_float(c[e + 2]), __uint_as_float(c[e + 3])), kk2, nm2));
                  const float a0 = ex2_approx(a.x), a1 = ex2_approx(a.y), b0 = ex2_approx(b.x), b1 = ex2_approx(b.y);
                  sum0 = fadd2(sum0, f2_pack(a0, a1));
                  sum1 = fadd2(sum1, f2_pack(b0, b1));
                  p[q * 16 + (e >> 1)] = pack_bf16x2(a0, a1);
                  p[q * 16 + (e >> 1) + 1] = pack_bf16x2(b0, b1);
                }
              } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) p[q * 16 + e] = 0;
              }
            }
            tmem_st_32x32b_x32(s_col + h * 32, p);
          }
          const float2 t0 = f2_unpack(sum0), t1 = f2_unpack(sum1);
          l += (t0.x + t0.y) + (t1.x + t1.y);
        };
        if (k0 < lo_max || k0 + kTile - 1 > hi_min) tile(std::false_type{});
        else tile(std::true_type{});
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      if (!ok) break;
      // ---- the row's result
      if (i < T) S.lse[static_cast<int64_t>(qt.c) * A.T + i] = in ? (m + __log2f(l)) * kLn2 : -INFINITY;
      const float inv = in ? 1.0f / l : 0.0f;
      const bool computed = qt.jend > qt.jbeg;
      if (computed) {
        ok = mbar_wait(&o_full[x], no & 1u, abort_flag, status, tmo);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        ++no;
        tc_fence_after_sync();
      }
      float bad = 0.0f;   // becomes NaN with the first value that is not finite
      // 64 columns at a time: a row per thread into the warp's swizzled tile, which a TMA store takes to memory (rows
      // past T are clipped).  Stored by the threads, 64 bytes of 32 different rows at a time, it took 3100
      // cycles an item.
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint32_t o[2][32];
#pragma unroll
        for (int e = 0; e < 64; ++e) o[e >> 5][e & 31] = 0;
        if (computed) {
          tmem_ld_32x32b_x32(o_col + h * 64, o[0]);
          tmem_ld_32x32b_x32(o_col + h * 64 + 32, o[1]);
          tmem_ld_wait();
        }
        if (lane == 0) bulk_wait_group_read<0>();   // the tile's last store has read it
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = u * 8 + 2 * e;
            const float lo_v = in ? __uint_as_float(o[c >> 5][c & 31]) * inv : 0.0f;
            const float hi_v = in ? __uint_as_float(o[c >> 5][(c & 31) + 1]) * inv : 0.0f;
            bad = fmaf(lo_v, 0.0f, fmaf(hi_v, 0.0f, bad));
            w[e] = pack_bf16x2(lo_v, hi_v);
          }
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&P.o[shard], stage, qt.c * D + h * 64, qt.q0 + quad * 32);
          bulk_commit_group();
        }
      }
      tc_fence_before_sync();
      const unsigned again = __ballot_sync(0xffffffffu, in && bad != 0.0f);
      if (again && lane == 0) redo_later(A.redo, redo_list, redo_slot(shard * A.nql + qt.c, A.T, qt.q0, quad), again);
    }
    if (lane == 0) bulk_wait_group_all();   // every store complete before the CTA's shared memory goes away
    __syncwarp();
    // The eight softmax warps, all of which come here, meet: the list is whole and every store of its rows complete.
    // (Within this branch, whose registers the code is given; behind the block's last barrier heads of 64 took 4% longer.)
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (redo_list->count > 0 && !*abort_flag) redo_rows<D>(A, *redo_list, warp - 4, 8, lane);
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

int pack_attn_fwd_launch(const PackArgs& A, int d, void* list, cudaStream_t stream) {
  FwdParams P;
  std::memset(static_cast<void*>(&P), 0, sizeof(P));
  P.a = A;
  const int64_t qc = static_cast<int64_t>(A.nql) * d, kc = static_cast<int64_t>(A.nkvl) * d;
  int rc = TTL_OK;
  for (int i = 0; i < A.t; ++i) {
    if ((rc = encode_map_bf16(&P.q[i], A.s[i].q, A.T, qc, A.ldq, 64, kTile)) ||
        (rc = encode_map_bf16(&P.k[i], A.s[i].k, A.T, kc, A.ldk, 64, kTile)) ||
        (rc = encode_map_bf16(&P.v[i], A.s[i].v, A.T, kc, A.ldv, 64, kTile)) ||
        (rc = encode_map_bf16(&P.o[i], A.s[i].o, A.T, qc, A.ldo, 64, 32)))
      return rc;
  }
  const int tiles = static_cast<int>((A.T + kTile - 1) / kTile);
  P.pair_heads = A.grp % 2 == 0;
  P.units = P.pair_heads ? tiles : (tiles + 1) / 2;
  P.lanes = P.pair_heads ? A.t * A.nql / 2 : A.t * A.nql;
  P.timeout_ns = pack_wait_ns(tiles);
  const int64_t items = static_cast<int64_t>(P.units) * P.lanes;
  if (items >= (int64_t(1) << 30)) return set_error(TTL_ERR_SHAPE, "packed attention: too many query tiles");
  const int sms = num_sms();
  const unsigned grid = static_cast<unsigned>(items < sms ? items : sms);
  if (items > sms) {   // more than one round: the order counts
    PackPlan plan = {};
    plan.q_list = static_cast<int4*>(list);
    plan.q_units = P.units;
    plan.q_per = P.pair_heads ? 1 : 2;
    plan.q_taken = reinterpret_cast<int*>(plan.q_list + tiles);
    if ((rc = pack_attn_plan_launch(A, plan, 0, stream))) return rc;
    P.a.q_list = plan.q_list;
    P.a.q_taken = plan.q_taken;
  }
  const double tri = static_cast<double>(A.T) * (A.T + 1) / 2.0;   // one document: the lengths are on the device
  TraceScope trace(stream, TTL_K_ATTN_CORE, 4.0 * tri * d * A.nql * A.t,
                   2.0 * A.T * (2.0 * qc + 2.0 * kc) * A.t);
  // Behind the plan its blocks may be brought up early.  Without one the kernel before is the caller's: a block that
  // held all of tensor memory while one of that kernel's still had to allocate some would keep it from ending.
  auto launch = [&](auto kernel, size_t smem) {
    return cuda_check(P.a.q_list ? launch_after(kernel, dim3(grid), kFwdThreads, smem, stream, P)
                                 : launch_first(kernel, dim3(grid), kFwdThreads, smem, stream, P),
                      "pack_fwd_kernel launch");
  };
  if (d == 128) {
    if ((rc = allow_smem<pack_fwd_kernel<128>>(FwdCfg<128>::SMEM, "cudaFuncSetAttribute(packed attention forward)")))
      return rc;
    rc = launch(pack_fwd_kernel<128>, FwdCfg<128>::SMEM);
  } else {
    if ((rc = allow_smem<pack_fwd_kernel<64>>(FwdCfg<64>::SMEM, "cudaFuncSetAttribute(packed attention forward)")))
      return rc;
    rc = launch(pack_fwd_kernel<64>, FwdCfg<64>::SMEM);
  }
  return rc;
}

}  // namespace ttl
