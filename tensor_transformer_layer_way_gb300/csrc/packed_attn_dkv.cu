// dK and dV of packed causal attention on the tensor cores.
//
// One work item is a 128-token key tile of one KV head; it meets the query tiles from its own to the one
// that holds the last token of its last key's document, each with every query head of the group
// (step n: query tile, head), the last query tile first.  With the keys as rows:
//   S^T = K Q^T, dP^T = V dO^T (fp32, tensor memory), P^T = 2^(s k - lse), dS^T = P^T (dP^T - D),
//   dV += P^T dO, dK += dS^T Q, dK scaled once at the end.
// P^T and dS^T go back to tensor memory as bf16 over the columns of S^T and dP^T, where they are the A
// operands; the Q and dO tiles are read K-major for the scores and MN-major for the sums.  Nothing but
// the four operand tiles passes through shared memory.
//
// S^T, dP^T, dK and dV fill tensor memory (4 x 128 columns), so the order of the products is what keeps the
// tensor pipe busy: S(n+1), dK(n), dP(n+1), dV(n+1), S(n+2), ...  While the elementwise warps turn S(n+1)
// into P, dK(n) and dP(n+1) run; while they form dS(n+1), dV(n+1) and S(n+2) do.
//
// What bounds it: the turns of tensor pipe and elementwise warps, 3000 cycles a step where the products need 2050.
// Measured: one document of 16384 tokens, 4 query heads and 1 KV head of 128: 370 us, 1490 TFLOP/s.  P^T and dS^T are
// rounded to bf16 once, the type of dO and Q in their products.
//
// Blocks take items from the list, heaviest first, as they get to them; warp 0 takes one while its last tiles wait for
// a place, and announces it to the others.  (Dealt out beforehand, in turn and back: 188 us for 12 documents of
// 8192 tokens together, 32 and 8 heads over 8 shards; taken: 145 to 149.)
//
// Roles (640 threads, persistent): warp 0 the TMA loads, warp 1 the MMAs, warp 2 brings each step's lse and D to
// shared memory, warp 3 the documents of the coming item's keys, warps 4..19 the elementwise work: a key row per
// thread, each of the four warpgroups on 32 of the queries (on 64 each, two warpgroups took 1450 cycles from
// S to P, longer than dK and dP run).

#include "packed_attn.cuh"

namespace ttl {
namespace {

constexpr int kKvThreads = 640;
constexpr int kKvWarps = 16;   // elementwise warps
constexpr int kRing = 5;       // places of the Q and dO tiles: Q_0, dO_0, Q_1, dO_1, ...
constexpr int kStat = 2;       // lse and D stages

struct KvParams {
  PackMaps m;
  PackArgs a;
  int tiles, lanes;
  uint64_t timeout_ns;
};

// Steps [t0, t0 + steps) of a key tile: step n is query tile qt_last - n / group, head n % group of the group.
struct KvItem {
  int shard, g, k0, qt_last, t0, steps;   // (shard < 0: no more items)
  int slot;                    // >= 0: a part of the key tile's sums, for that place of the partial buffers
};

template <int D>
struct KvCfg {
  static constexpr int KB = D / 64;
  static constexpr int TILE = KB * kTile * 128;
  static constexpr int OFF_V = TILE;
  static constexpr int OFF_RING = 2 * TILE;
  static constexpr int OFF_STAT = OFF_RING + kRing * TILE;   // float [kStat][2][128]: -lse log2(e), -D
  static constexpr int OFF_ROWS = OFF_STAT + kStat * 1024;  // int [128]: the last query that sees a key
  static constexpr int OFF_BAR = OFF_ROWS + 512;
  static constexpr int SMEM = OFF_BAR + 336 + kAhead * static_cast<int>(sizeof(KvItem));   // (the block begins on 1024 bytes; the kernel checks it)
  static_assert(SMEM <= 232448, "shared memory beyond the per-CTA limit");
};

// The listed item of index `at`.
__device__ __forceinline__ KvItem listed_item(const KvParams& P, int at) {
  const PackArgs& A = P.a;
  const int ln = at % P.lanes;
  const int4 e = __ldg(A.kv_list + 2 * (at / P.lanes));
  const int slot = __ldg(A.kv_list + 2 * (at / P.lanes) + 1).x;
  return KvItem{ln / A.nkvl, ln % A.nkvl, e.x * kTile, e.y, e.z, e.w - e.z, slot < 0 ? -1 : slot * P.lanes + ln};
}

// A block's first item (of `total`), found by a whole warp.
__device__ __forceinline__ KvItem first_item(const KvParams& P, int total) {
  const PackArgs& A = P.a;
  const int at = static_cast<int>(blockIdx.x), ln = at % P.lanes, tile = at / P.lanes;
  if (at >= total) return KvItem{-1, 0, 0, 0, 0, 0, -1};
  if (A.kv_list) return listed_item(P, at);
  KvItem it = {ln / A.nkvl, ln % A.nkvl, tile * kTile, tile - 1, 0, 0, -1};
  if (A.batch > 0) {
    const int T = static_cast<int>(A.T);
    const int first = __ldg(A.cu), last = __ldg(A.cu + A.batch);
    const int v0 = it.k0 > first ? it.k0 : first;
    int v1 = it.k0 + kTile < last ? it.k0 + kTile : last;
    v1 = v1 < T ? v1 : T;
    if (v0 < v1) {
      const int hi = doc_of_warp(A.cu, A.batch, T, v1 - 1).hi;   // > v1 - 1
      it.qt_last = (hi > v1 ? hi - 1 : v1 - 1) / kTile;
      it.steps = (it.qt_last - tile + 1) * A.grp;
    }
  }
  return it;
}

// Those of the rows j of dK (want_k) or dV, whose sums are not finite, that masked places may have made so, again.
// `edges` are looked at once for the rows of a tile.
template <int D, int R>
__device__ __noinline__ void redo_keys(const PackArgs& A, int shard, int g, int (&j)[R], bool want_k, KeyEdges& edges,
                                          bool& looked, int lane) {
  const PackShard& S = A.s[shard];
  const int T = static_cast<int>(A.T), row0 = j[0] & ~31;
  uint32_t again = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int hi = doc_of(A.cu, A.batch, T, j[r]).hi;
    bool met = hi - j[r] < kRedoShort;
    if (!met) {
      if (!looked) edges.look<D>(A, S, g, row0, hi, want_k, lane);
      looked = true;
      met = edges.met(j[r], hi);
    }
    if (met) again |= 1u << (j[r] - row0);
  }
  if (again == 0) return;
  const int m = redo_take(again, row0, j);
  int hi[R];
#pragma unroll
  for (int r = 0; r < R; ++r) hi[r] = doc_of(A.cu, A.batch, T, j[r]).hi;
  dkv_rows<D>(A, S, shard, g, j, hi, m, want_k, lane);
}

// The listed rows again, by `warps` warps, of which this is number w: the rows of an entry in groups, the groups in turn.
template <int D>
__device__ __noinline__ void redo_rows(const PackArgs& A, RedoList list, int w, int warps, int lane) {
  const uint32_t slots = redo_slots(A.t * A.nkvl * 2, A.T);
  int turn = 0;
  for (uint32_t slot = list.head; slot < slots && list.count > 0; --list.count) {
    const RedoEntry e = A.redo[slot];
    const RedoPlace at = redo_place(slot, A.T);
    const int kv = at.head >> 1;
    KeyEdges edges;
    bool looked = false;
    for (uint32_t rows = e.rows; rows;) {
      int j[kRedoRows];
      redo_take(rows, at.row0, j);
      if (turn++ % warps == w) redo_keys<D>(A, kv / A.nkvl, kv % A.nkvl, j, (at.head & 1) == 0, edges, looked, lane);
    }
    slot = e.next;
  }
}

template <int D>
__global__ void __launch_bounds__(kKvThreads, 1) pack_dkv_kernel(const __grid_constant__ KvParams P) {
  using C = KvCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  uint8_t* sK = smem;
  uint8_t* sV = smem + C::OFF_V;
  uint8_t* sRing = smem + C::OFF_RING;
  float* stat = reinterpret_cast<float*>(smem + C::OFF_STAT);
  int* row_hi = reinterpret_cast<int*>(smem + C::OFF_ROWS);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_empty = k_full + 1;
  uint64_t* v_full = k_empty + 1;
  uint64_t* v_empty = v_full + 1;
  uint64_t* ring_full = v_empty + 1;
  uint64_t* ring_empty = ring_full + kRing;
  uint64_t* st_full = ring_empty + kRing;
  uint64_t* st_empty = st_full + kStat;
  uint64_t* s_full = st_empty + kStat;
  uint64_t* p_full = s_full + 1;
  uint64_t* dp_full = p_full + 1;
  uint64_t* ds_full = dp_full + 1;
  uint64_t* acc_full = ds_full + 1;
  uint64_t* rows_full = acc_full + 1;
  uint64_t* rows_empty = rows_full + 1;
  uint64_t* x_bar = rows_empty + 1;    // the elementwise warps meet
  uint64_t* done_bar = x_bar + 1;
  uint64_t* item_bars = done_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(item_bars + kQueueBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* flags = tmem_slot + 2;     // [2][4]: rows of a quadrant to be done again, of dK and of dV
  RedoList* redo_list = reinterpret_cast<RedoList*>(flags + 8);
  static_assert((4 + 2 * kRing + 2 * kStat + 9 + kQueueBars) * 8 + 48 <= 336, "barrier area");
  constexpr uint32_t T_DP = 128, T_DK = 256, T_DV = 384;

  const PackArgs& A = P.a;
  const int warp = uniform_warp();
  const int lane = threadIdx.x & 31;
  if (smem_u32(smem_raw) & 1023u) {   // the tiles' swizzle needs it; every block of the launch ends here alike
    if (threadIdx.x == 0) atomicCAS(A.status, 0, TTL_ERR_ALIGN);
    return;
  }
  await_previous();   // (the dQ kernel; through it D and the list)
  const int total = (A.kv_list ? __ldg(A.kv_head) : P.tiles) * P.lanes;
  int* status = A.status;
  const uint64_t tmo = P.timeout_ns;
  const ItemQueue<KvItem> queue{reinterpret_cast<KvItem*>(smem + C::OFF_BAR + 336), item_bars, abort_flag, status, tmo};
  // The item's n-th step: the last query tile first, the group's heads in turn.
  auto step_q0 = [&](const KvItem& it, int n) { return (it.qt_last - (it.t0 + n) / A.grp) * kTile; };
  auto step_head = [&](const KvItem& it, int n) { return it.g * A.grp + (it.t0 + n) % A.grp; };

  if (threadIdx.x == 0) {
    mbar_init(k_full, 1);
    mbar_init(k_empty, 1);
    mbar_init(v_full, 1);
    mbar_init(v_empty, 1);
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&ring_full[s], 1);
      mbar_init(&ring_empty[s], 1);
    }
    for (int s = 0; s < kStat; ++s) {
      mbar_init(&st_full[s], 1);
      mbar_init(&st_empty[s], kKvWarps);
    }
    mbar_init(s_full, 1);
    mbar_init(p_full, kKvWarps);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, kKvWarps);
    mbar_init(acc_full, 1);
    mbar_init(rows_full, 1);
    mbar_init(rows_empty, kKvWarps);
    mbar_init(x_bar, kKvWarps);
    mbar_init(done_bar, 1);
    for (int q = 0; q < 8; ++q) flags[q] = 0;
    *redo_list = RedoList{kRedoNone, 0};
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (threadIdx.x == 64) {
    queue.init(kKvWarps + 3);
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA loads
    bool ok = true;
    int nk = 0, nv = 0, pos = 0;   // loads started: K, V, ring places
    KvItem it = first_item(P, total);
    for (int n = 0; lane == 0 && ok && it.shard >= 0; ++n) {
      KvItem coming = {};
      coming.shard = -1;
      auto announce = [&]() {
        if (A.kv_list) {
          const int at = static_cast<int>(gridDim.x) + atomicAdd(A.kv_taken, 1);
          if (at < total) coming = listed_item(P, at);
        }
        ok = queue.announce(n + 1, coming);
      };
      const int when = max(0, it.steps - kLead);
      if (it.steps == 0) {
        announce();
      } else {
        auto load = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* full, uint64_t* empty, uint32_t phase, int x, int y) {
          if (!wait_on(empty, (phase & 1u) ^ 1u, abort_flag, status, tmo)) return false;
          mbar_arrive_expect_tx(full, C::TILE);
          for (int kb = 0; kb < C::KB; ++kb) tma_load_2d(dst + kb * 16384, map, full, x + kb * 64, y);
          return true;
        };
        auto load_ring = [&](const CUtensorMap* map, int x, int y) {
          const int slot = pos % kRing;
          if (!load(sRing + slot * C::TILE, map, &ring_full[slot], &ring_empty[slot], pos / kRing, x, y)) return false;
          ++pos;
          return true;
        };
        for (int t = 0; ok && t < it.steps; ++t) {
          if (t == 0) {
            ok = load(sK, &P.m.k[it.shard], k_full, k_empty, nk, it.g * D, it.k0);
            nk += ok;
          }
          ok = ok && load_ring(&P.m.q[it.shard], step_head(it, t) * D, step_q0(it, t));
          if (ok && t == 0) {
            ok = load(sV, &P.m.v[it.shard], v_full, v_empty, nv, it.g * D, it.k0);
            nv += ok;
          }
          ok = ok && load_ring(&P.m.dO[it.shard], step_head(it, t) * D, step_q0(it, t));
          if (ok && t == when) announce();
        }
      }
      it = coming;
    }
    if (lane == 0) {
      // No copy may still be landing when the CTA leaves: wait (bounded) for the last loads.
      int dummy = 0;
      volatile int* da = reinterpret_cast<volatile int*>(&dummy);
      if (nk > 0) wait_on(k_full, static_cast<uint32_t>(nk - 1) & 1u, da, status, tmo);
      if (nv > 0) wait_on(v_full, static_cast<uint32_t>(nv - 1) & 1u, da, status, tmo);
      for (int i = pos > kRing ? pos - kRing : 0; i < pos; ++i)
        wait_on(&ring_full[i % kRing], static_cast<uint32_t>(i / kRing) & 1u, da, status, tmo);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMAs
    // The whole warp runs this loop, one elected lane issues.  A wait that runs out is in the status word and raises
    // the abort flag, after which every wait returns at once: the loop then ends over what is in memory.
    int ni = 0, p = 0;                     // items; steps scored
    int qs = 0, lap = 0, old = 0;          // ring place of Q_(t + 1), its round; place of Q_t
    const uint64_t kd = smem_desc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t vd = smem_desc_sw128(smem_u32(sV), 16, 1024);
    const uint64_t rk0 = smem_desc_sw128(smem_u32(sRing), 16, 1024);      // K-major
    const uint64_t rn0 = smem_desc_sw128(smem_u32(sRing), 16384, 1024);   // MN-major
    const uint32_t idesc_s = idesc_bf16_f32(kTile, kTile, false, false);
    const uint32_t idesc_acc = idesc_bf16_f32(kTile, D, false, true);
    const bool leader = elect_one();
    auto wait = [&](uint64_t* bar, int phase) {
      wait_on(bar, static_cast<uint32_t>(phase) & 1u, abort_flag, status, tmo);
    };
    // [keys x queries] = A B^T, both K-major tiles of D columns
    auto scores = [&](uint32_t dst, uint64_t ad, uint64_t bd) {
#pragma unroll
      for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16(dst, desc_advance(ad, kb * 16384 + kk * 32), desc_advance(bd, kb * 16384 + kk * 32), idesc_s,
                    (kb | kk) ? 1u : 0u);
    };
    // [keys x D] += A B: A from tensor memory (queries [32 w, 32 w + 32) at columns 32 w ..), B read MN-major
    auto sum = [&](uint32_t dst, uint32_t acol, uint64_t bd, uint32_t more) {
#pragma unroll
      for (int kk = 0; kk < kTile / 16; ++kk)
        umma_bf16_ts(dst, acol + (kk >> 1) * 32 + (kk & 1) * 8, desc_advance(bd, kk * 2048), idesc_acc, kk ? 1u : more);
    };
    KvItem it = first_item(P, total);
    for (int n = 0; queue.next(n, it) && it.shard >= 0; ++n) {
      if (it.steps == 0) continue;
      wait(k_full, ni);
      // S^T of step t overwrites P^T of the step before, whose dV product was issued before it (the tensor
      // pipe runs one thread's products in order); likewise dP^T and dK.
      for (int t = -1; t < it.steps; ++t) {
        const int ds = qs + 1 == kRing ? 0 : qs + 1;   // place of dO_(t + 1): the one behind Q_(t + 1)
        if (t + 1 < it.steps) {
          wait(&ring_full[qs], lap);
          tc_fence_after_sync();
          if (leader) {
            scores(tmem, kd, desc_advance(rk0, qs * C::TILE));
            umma_commit(s_full);
            if (t + 2 == it.steps) umma_commit(k_empty);
          }
        }
        if (t >= 0) {
          wait(ds_full, p - 1);
          tc_fence_after_sync();
          if (leader) {
            sum(tmem + T_DK, tmem + T_DP, desc_advance(rn0, old * C::TILE), t > 0 ? 1u : 0u);
            umma_commit(&ring_empty[old]);
          }
        }
        if (t + 1 < it.steps) {
          if (t < 0) wait(v_full, ni);
          wait(&ring_full[ds], ds == 0 ? lap + 1 : lap);
          tc_fence_after_sync();
          if (leader) {
            scores(tmem + T_DP, vd, desc_advance(rk0, ds * C::TILE));
            umma_commit(dp_full);
            if (t + 2 == it.steps) umma_commit(v_empty);
          }
          wait(p_full, p);
          tc_fence_after_sync();
          if (leader) {
            sum(tmem + T_DV, tmem, desc_advance(rn0, ds * C::TILE), t >= 0 ? 1u : 0u);
            umma_commit(&ring_empty[ds]);
          }
          ++p;
          old = qs;
          qs += 2;
          if (qs >= kRing) {
            qs -= kRing;
            ++lap;
          }
        }
        __syncwarp();
      }
      if (leader) umma_commit(acc_full);
      __syncwarp();
      ++ni;
    }
    if (leader) umma_commit(done_bar);   // every MMA issued here must finish before TMEM is released
    __syncwarp();
    int dummy = 0;
    wait_on(done_bar, 0, reinterpret_cast<volatile int*>(&dummy), status, tmo);
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------------ lse and D of each step's queries
    bool ok = true;
    int pos = 0;
    KvItem it = first_item(P, total);
    for (int n = 0; ok && queue.next(n, it) && it.shard >= 0; ++n) {
      const float* lse = A.s[it.shard].lse;
      const float* Dr = A.D + static_cast<int64_t>(it.shard) * A.nql * A.T;
      for (int t = 0; t < it.steps; ++t, ++pos) {
        const int st = pos % kStat;
        const int64_t row = static_cast<int64_t>(step_head(it, t)) * A.T;
        const int q0 = step_q0(it, t);
        float a[4], b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int q = q0 + u * 32 + lane;
          a[u] = q < A.T ? -__ldg(lse + row + q) * kLog2e : 0.0f;
          b[u] = q < A.T ? -__ldg(Dr + row + q) : 0.0f;
        }
        ok = wait_on(&st_empty[st], (static_cast<uint32_t>(pos / kStat) & 1u) ^ 1u, abort_flag, status, tmo);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          stat[st * 256 + u * 32 + lane] = a[u];
          stat[st * 256 + 128 + u * 32 + lane] = b[u];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&st_full[st]);
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------------ last queries of the coming item's keys
    bool ok = true;
    KvItem it = first_item(P, total);
    for (int n = 0; ok && queue.next(n, it) && it.shard >= 0; ++n) {
      int hi[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        DocRange doc{0, 0};
        if (it.steps > 0) doc = doc_of(A.cu, A.batch, static_cast<int>(A.T), it.k0 + u * 32 + lane);
        hi[u] = doc.hi > doc.lo ? doc.hi - 1 : -1;   // a token of no document is seen by none
      }
      ok = wait_on(rows_empty, (static_cast<uint32_t>(n) & 1u) ^ 1u, abort_flag, status, tmo);
      if (!__all_sync(0xffffffffu, ok)) break;
#pragma unroll
      for (int u = 0; u < 4; ++u) row_hi[u * 32 + lane] = hi[u];
      __syncwarp();
      if (lane == 0) mbar_arrive(rows_full);
    }
  } else {
    // ------------------------------------------------------------------ P^T and dS^T
    const int quad = warp & 3;
    const int w = (warp - 4) >> 2;             // queries [32 w, 32 w + 32) of each tile
    const int r = quad * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const float k2 = A.scale * kLog2e;
    const uint64_t kk2 = f2_pack(k2, k2);
    const int T = static_cast<int>(A.T);
    bool ok = true;
    int pos = 0, ni = 0;
    uint32_t met = 0;
    KvItem it = first_item(P, total);
    for (int n = 0; ok && queue.next(n, it) && it.shard >= 0; ++n) {
      const PackShard& S = A.s[it.shard];
      const int key = it.k0 + r;
      ok = mbar_wait(rows_full, static_cast<uint32_t>(n) & 1u, abort_flag, status, tmo);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      const int hi = row_hi[r];                      // the queries lo..hi see the key
      __syncwarp();
      if (lane == 0) mbar_arrive(rows_empty);
      const bool in = hi >= 0;                       // a key of a document
      const int lo = in ? key : 0x7fffffff;
      const int lo_max = __reduce_max_sync(0xffffffffu, lo), hi_min = __reduce_min_sync(0xffffffffu, hi);
      for (int t = 0; ok && t < it.steps; ++t, ++pos) {
        const int st = pos % kStat;
        const int q0 = step_q0(it, t) + w * 32;
        const bool masked = q0 < lo_max || q0 + 31 > hi_min;
        const float4* nl = reinterpret_cast<const float4*>(stat + st * 256 + w * 32);
        const float4* nD = reinterpret_cast<const float4*>(stat + st * 256 + 128 + w * 32);
        ok = mbar_wait(&st_full[st], static_cast<uint32_t>(pos / kStat) & 1u, abort_flag, status, tmo) &&
             mbar_wait(s_full, static_cast<uint32_t>(pos) & 1u, abort_flag, status, tmo);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        uint32_t s[32];
        tmem_ld_32x32b_x32(lane_base + w * 32, s);
        tmem_ld_wait();
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 n4 = nl[e >> 2];
          const float2 u =
              f2_unpack(ffma2(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), kk2, f2_pack(n4.x, n4.y)));
          const float2 v =
              f2_unpack(ffma2(f2_pack(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), kk2, f2_pack(n4.z, n4.w)));
          s[e] = __float_as_uint(ex2_approx(u.x));
          s[e + 1] = __float_as_uint(ex2_approx(u.y));
          s[e + 2] = __float_as_uint(ex2_approx(v.x));
          s[e + 3] = __float_as_uint(ex2_approx(v.y));
          pk[e >> 1] = pack_bf16x2(__uint_as_float(s[e]), __uint_as_float(s[e + 1]));
          pk[(e >> 1) + 1] = pack_bf16x2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
        }
        // hidden queries: P and, whatever dP and D hold, dS are 0
        const uint32_t see = masked ? bits_between(lo - q0, hi - q0) : 0xffffffffu;
        auto hide = [&]() {
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            pk[e >> 1] &= ((see >> e) & 1u ? 0x0000ffffu : 0u) | ((see >> (e + 1)) & 1u ? 0xffff0000u : 0u);
        };
        if (masked) hide();
        tmem_st_32x32b_x16(lane_base + w * 32, pk);   // over this thread's own columns of S^T
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
        ok = mbar_wait(dp_full, static_cast<uint32_t>(pos) & 1u, abort_flag, status, tmo);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        uint32_t dp[32];
        tmem_ld_32x32b_x32(lane_base + T_DP + w * 32, dp);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 n4 = nD[e >> 2];
          const float2 u = f2_unpack(
              fmul2(fadd2(f2_pack(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])), f2_pack(n4.x, n4.y)),
                    f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1]))));
          const float2 v = f2_unpack(
              fmul2(fadd2(f2_pack(__uint_as_float(dp[e + 2]), __uint_as_float(dp[e + 3])), f2_pack(n4.z, n4.w)),
                    f2_pack(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]))));
          pk[e >> 1] = pack_bf16x2(u.x, u.y);
          pk[(e >> 1) + 1] = pack_bf16x2(v.x, v.y);
        }
        if (masked) hide();
        tmem_st_32x32b_x16(lane_base + T_DP + w * 32, pk);
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(ds_full);
          mbar_arrive(&st_empty[st]);
        }
      }
      if (!ok) break;
      // ---- two warpgroups store dK, two dV; the last products are running
      const int kind = w >> 1, col = (w & 1) * (D / 2);
      const bool computed = it.steps > 0;
      if (computed) {
        ok = mbar_wait(acc_full, static_cast<uint32_t>(ni) & 1u, abort_flag, status, tmo);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        ++ni;
        tc_fence_after_sync();
      }
      float bad = 0.0f;   // becomes NaN with the first value that is not finite
      const float f = kind || it.slot >= 0 ? 1.0f : A.scale;
      const int64_t off = (kind ? A.lddv : A.lddk) * static_cast<int64_t>(key < T ? key : 0) + it.g * D + col;
      __nv_bfloat16* out = (kind ? S.dv : S.dk) + off;
      float* part = A.part + ((static_cast<int64_t>(it.slot < 0 ? 0 : it.slot) * 2 + kind) * kTile + r) * D + col;
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {
        uint32_t o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0;
        if (computed) {
          tmem_ld_32x32b_x32(lane_base + (kind ? T_DV : T_DK) + col + u * 32, o);
          tmem_ld_wait();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float v = in ? __uint_as_float(o[e]) * f : 0.0f;
          bad = fmaf(v, 0.0f, bad);
          o[e] = __float_as_uint(v);
        }
        if (it.slot >= 0) {
#pragma unroll
          for (int q = 0; q < 4; ++q) st_global_v8(part + u * 32 + q * 8, o + q * 8);
        } else if (key < T) {
          store_bf16x32(out + u * 32, o);
        }
      }
      tc_fence_before_sync();
      // A row is listed, by one of its two warpgroups, if either found its columns not finite.  (All sixteen warps
      // meet, with a bounded wait, unlike a hardware barrier.)
      const unsigned mine = __ballot_sync(0xffffffffu, in && bad != 0.0f && it.slot < 0);
      if (mine && lane == 0) atomicOr(&flags[kind * 4 + quad], mine);
      __syncwarp();
      if (lane == 0) mbar_arrive(x_bar);
      ok = mbar_wait(x_bar, met & 1u, abort_flag, status, tmo);
      ++met;
      if (!__all_sync(0xffffffffu, ok)) break;
      if ((w & 1) == 0) {
        const unsigned again = flags[kind * 4 + quad];
        __syncwarp();
        if (again && lane == 0) {
          flags[kind * 4 + quad] = 0;
          redo_later(A.redo, redo_list, redo_slot((it.shard * A.nkvl + it.g) * 2 + kind, A.T, it.k0, quad), again);
        }
      }
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (warp >= 4 && redo_list->count > 0 && !*abort_flag) redo_rows<D>(A, *redo_list, warp - 4, kKvWarps, lane);
}

// Adds up the parts of the key tiles that several items shared, in the order of their steps: one warp per row
// of dK or dV, eight rows of a tile per block.
template <int D>
__global__ void __launch_bounds__(256, 4) pack_join_kernel(const __grid_constant__ PackArgs A) {
  __shared__ uint32_t redo[2];       // rows of the eight whose sums are not finite; of the eight before, spent
  await_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = A.t * A.nkvl;
  const int64_t rows = static_cast<int64_t>(__ldg(A.kv_head + 1)) * lanes * 2 * kTile;
  if (threadIdx.x < 2) redo[threadIdx.x] = 0;
  __syncthreads();
  int now = 0;
  for (int64_t w0 = static_cast<int64_t>(blockIdx.x) * 8; w0 < rows; w0 += gridDim.x * 8, now ^= 1) {
    const int r0 = static_cast<int>(w0 % kTile), half = static_cast<int>(w0 / kTile) & 1, r = r0 + warp;
    const int64_t at = w0 / (2 * kTile);
    const int ln = static_cast<int>(at % lanes);
    const int4 e = __ldg(A.join_list + at / lanes);
    const int key0 = e.x * kTile + r0, key = key0 + warp;
    const int shard = ln / A.nkvl, g = ln % A.nkvl;
    const PackShard& S = A.s[shard];
    if (key < A.T) {
      RowVec<D> acc = row_zero<D>();
      for (int p = 0; p < e.z; ++p) {
        const float* src = A.part + ((static_cast<int64_t>(e.y + p) * lanes + ln) * 2 + half) * kTile * D +
                           static_cast<int64_t>(r) * D + lane * (D / 32);
#pragma unroll
        for (int u = 0; u < D / 32; ++u) acc.x[u] += src[u];
      }
      bool fine = true;
#pragma unroll
      for (int u = 0; u < D / 32; ++u) {
        if (half == 0) acc.x[u] *= A.scale;
        fine &= fabsf(acc.x[u]) < INFINITY;
      }
      row_store<D>((half ? S.dv + key * A.lddv : S.dk + key * A.lddk) + g * D, acc, lane);
      if (!__all_sync(0xffffffffu, fine) && lane == 0) atomicOr(&redo[now], 1u << warp);
    }
    __syncthreads();                 // (and all eight rows are stored)
    uint32_t again = redo[now];
    if (threadIdx.x == 0) redo[now ^ 1] = 0;
    if (again && warp < 8 / kRedoRows) {
      again &= ((1u << kRedoRows) - 1) << (warp * kRedoRows);
      int j[kRedoRows];
      KeyEdges edges;
      bool looked = false;
      if (redo_take(again, key0, j) > 0) redo_keys<D>(A, shard, g, j, half == 0, edges, looked, lane);
    }
    __syncthreads();
  }
}

}  // namespace

int pack_attn_join_launch(const PackArgs& A, int d, cudaStream_t stream) {
  TraceScope trace(stream, TTL_K_OTHER, 0.0, 0.0);
  const unsigned grid = static_cast<unsigned>(num_sms()) * 4;
  if (d == 128)
    return cuda_check(launch_after(pack_join_kernel<128>, dim3(grid), 256, 0, stream, A), "pack_join_kernel launch");
  return cuda_check(launch_after(pack_join_kernel<64>, dim3(grid), 256, 0, stream, A), "pack_join_kernel launch");
}

int pack_attn_dkv_launch(const PackArgs& A, const PackMaps& maps, int d, cudaStream_t stream) {
  KvParams P;
  P.a = A;
  P.m = maps;
  const int64_t qc = static_cast<int64_t>(A.nql) * d, kc = static_cast<int64_t>(A.nkvl) * d;
  int rc = TTL_OK;
  P.tiles = static_cast<int>((A.T + kTile - 1) / kTile);
  P.lanes = A.t * A.nkvl;
  P.timeout_ns = pack_wait_ns(static_cast<int64_t>(P.tiles) * A.grp);
  const int64_t items = static_cast<int64_t>(P.tiles) * P.lanes;
  if (items >= (int64_t(1) << 30)) return set_error(TTL_ERR_SHAPE, "packed attention: too many key tiles");
  const int sms = num_sms();
  const unsigned grid = static_cast<unsigned>(items < sms && !A.kv_list ? items : sms);
  const double tri = static_cast<double>(A.T) * (A.T + 1) / 2.0;   // one document: the lengths are on the device
  TraceScope trace(stream, TTL_K_ATTN_CORE, 4.0 * tri * d * A.nql * A.t, 2.0 * A.T * (2.0 * qc + 4.0 * kc) * A.t);
  if (d == 128) {
    if ((rc = allow_smem<pack_dkv_kernel<128>>(KvCfg<128>::SMEM, "cudaFuncSetAttribute(packed attention dK dV)")))
      return rc;
    rc = cuda_check(launch_after(pack_dkv_kernel<128>, dim3(grid), kKvThreads, KvCfg<128>::SMEM, stream, P), "pack_dkv_kernel launch");
  } else {
    if ((rc = allow_smem<pack_dkv_kernel<64>>(KvCfg<64>::SMEM, "cudaFuncSetAttribute(packed attention dK dV)")))
      return rc;
    rc = cuda_check(launch_after(pack_dkv_kernel<64>, dim3(grid), kKvThreads, KvCfg<64>::SMEM, stream, P), "pack_dkv_kernel launch");
  }
  return rc;
}

}  // namespace ttl
