// dQ of packed causal attention on the tensor cores.
//
// One work item is a 128-token query tile of one head; its key tiles are those of the forward kernel.
// Per key tile:  S = Q K^T and dP = dO V^T (fp32, tensor memory), P = 2^(s k - lse), dS = P (dP - D) as
// bf16 in tensor memory, dQ += dS K with dS as the A operand; dQ is scaled once at the end.  dQ and
// (dK, dV) are two kernels, so every sum has one owner and a fixed order: the price is S and dP twice
// (7 products where one kernel with atomic additions into dQ would need 5).
//
// Roles (640 threads, persistent): warp 0 the TMA loads (K three slots deep, read by S_j and again by dQ_j; V two),
// warp 1 the MMAs in the order S_(j+1), dP_(j+1), dQ_j, so that two products run while the elementwise warps
// form dS_j; warps 2 and 3 bring lse, D and the first key of the coming item's rows to shared memory; warps 4..19
// form dS: a row per thread, each of the four warpgroups on 32 of the keys (on 64 each, two warpgroups took
// longer over a tile than the products they run under).
// S, dP and dQ take 384 columns of tensor memory and two dS buffers the rest.
//
// What bounds it: the products' reads of shared memory, 1750 of the 2340 cycles a key tile takes.  Measured: one
// document of 16384 tokens, 4 query heads and 1 KV head of 128: 273 us, 1510 TFLOP/s; 8192 tokens in 12
// documents, 32 and 8 heads over 8 shards: 129 us.  dS is rounded to bf16 once, the type of K in their product (error of
// the gradients against 64 bits 2.5e-3, with P and dS in fp32 1.8e-3).

#include "packed_attn.cuh"

namespace ttl {
namespace {

constexpr int kDqThreads = 640;
constexpr int kDqWarps = 16;   // elementwise warps
constexpr int kKSlots = 3;
constexpr int kVSlots = 2;

struct DqParams {
  PackMaps m;
  PackArgs a;
  int tiles, lanes;
  uint64_t timeout_ns;
};

struct DqItem {
  int shard, c, g, q0, jbeg, jend;
};

template <int D>
struct DqCfg {
  static constexpr int KB = D / 64;
  static constexpr int TILE = KB * kTile * 128;
  static constexpr int OFF_DO = TILE;
  static constexpr int OFF_K = 2 * TILE;
  static constexpr int OFF_V = OFF_K + kKSlots * TILE;
  static constexpr int OFF_X = OFF_V + kVSlots * TILE;   // of each row: -lse log2(e), D, first key
  static constexpr int OFF_BAR = OFF_X + 1536;
  static constexpr int SMEM = OFF_BAR + 320 + kAhead * static_cast<int>(sizeof(DqItem)) + 1024;
  static_assert(SMEM <= 232448, "shared memory beyond the per-CTA limit");
};

// The item of index `at` whose query tile is `tile` and first key tile `first` (-1: none).
__device__ __forceinline__ DqItem item_from(const DqParams& P, int at, int tile, int first) {
  const int ln = at % P.lanes;
  DqItem it;
  it.shard = ln / P.a.nql;
  it.c = ln % P.a.nql;
  it.g = it.c / P.a.grp;
  it.q0 = tile * kTile;
  it.jbeg = first < 0 ? 0 : first;
  it.jend = first < 0 ? 0 : tile + 1;
  return it;
}

// The listed item of index `at`.
__device__ __forceinline__ DqItem listed_item(const DqParams& P, int at) {
  const int4 e = __ldg(P.a.q_list + at / P.lanes);
  return item_from(P, at, e.x, e.y);
}

// A block's first item, found by a whole warp.
__device__ __forceinline__ DqItem first_item(const DqParams& P) {
  const PackArgs& A = P.a;
  const int at = static_cast<int>(blockIdx.x);
  if (A.q_list) return listed_item(P, at);
  const int tile = P.tiles - 1 - at / P.lanes, q0 = tile * kTile;
  int first_tile = -1;
  if (A.batch > 0) {
    const int T = static_cast<int>(A.T);
    const int first = __ldg(A.cu), last = __ldg(A.cu + A.batch);
    const int v0 = q0 > first ? q0 : first;
    int v1 = q0 + kTile < last ? q0 + kTile : last;
    v1 = v1 < T ? v1 : T;
    if (v0 < v1) first_tile = doc_of_warp(A.cu, A.batch, T, v0).lo / kTile;
  }
  return item_from(P, at, tile, first_tile);
}

// The listed rows again, by `warps` warps, of which this is number w: the rows of an entry in groups, the groups in turn.
template <int D>
__device__ __noinline__ void redo_rows(const PackArgs& A, RedoList list, int w, int warps, int lane) {
  const uint32_t slots = redo_slots(A.t * A.nql, A.T);
  int turn = 0;
  for (uint32_t slot = list.head; slot < slots && list.count > 0; --list.count) {
    const RedoEntry e = A.redo[slot];
    const RedoPlace at = redo_place(slot, A.T);
    const int shard = at.head / A.nql, c = at.head % A.nql;
    const PackShard& S = A.s[shard];
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
          if (!looked) edges.look<D>(S.k, A.ldk, c / A.grp * D, first, at.row0, A.T, lane);
          looked = true;
          met = edges.met(first, i[r]);
        }
        if (met) again |= 1u << (i[r] - at.row0);
      }
      if (again == 0) continue;
      const int n = redo_take(again, at.row0, i);
#pragma unroll
      for (int r = 0; r < kRedoRows; ++r) lo[r] = doc_of(A.cu, A.batch, static_cast<int>(A.T), i[r]).lo;
      dq_rows<D>(A, S, shard, c, i, lo, n, lane);
    }
    slot = e.next;
  }
}

template <int D>
__global__ void __launch_bounds__(kDqThreads, 1) pack_dq_kernel(const __grid_constant__ DqParams P) {
  using C = DqCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sDO = smem + C::OFF_DO;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  float* row_nl = reinterpret_cast<float*>(smem + C::OFF_X);
  float* row_D = row_nl + kTile;
  int* row_lo = reinterpret_cast<int*>(row_D + kTile);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_empty = q_full + 1;
  uint64_t* k_full = q_empty + 1;
  uint64_t* k_empty = k_full + kKSlots;
  uint64_t* v_full = k_empty + kKSlots;
  uint64_t* v_empty = v_full + kVSlots;
  uint64_t* s_full = v_empty + kVSlots;
  uint64_t* s_empty = s_full + 1;
  uint64_t* dp_full = s_empty + 1;
  uint64_t* dp_empty = dp_full + 1;
  uint64_t* ds_full = dp_empty + 1;    // [2]
  uint64_t* ds_empty = ds_full + 2;    // [2]
  uint64_t* dq_full = ds_empty + 2;
  uint64_t* dq_empty = dq_full + 1;
  uint64_t* x_bar = dq_empty + 1;      // the elementwise warps meet
  uint64_t* rows_full = x_bar + 1;
  uint64_t* rows_empty = rows_full + 1;
  uint64_t* done_bar = rows_empty + 1;
  uint64_t* item_bars = done_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(item_bars + kQueueBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* flags = tmem_slot + 2;     // [4]: rows of a quadrant to be done again
  RedoList* redo_list = reinterpret_cast<RedoList*>(flags + 4);
  static_assert((2 + 2 * kKSlots + 2 * kVSlots + 14 + kQueueBars) * 8 + 32 <= 320, "barrier area");
  constexpr uint32_t T_DP = 128, T_DQ = 256, T_DS = 384;

  const PackArgs& A = P.a;
  const int warp = uniform_warp();
  const int lane = threadIdx.x & 31;
  const int total = P.tiles * P.lanes;
  int* status = A.status;
  const uint64_t tmo = P.timeout_ns;
  const ItemQueue<DqItem> queue{reinterpret_cast<DqItem*>(smem + C::OFF_BAR + 320), item_bars, abort_flag, status, tmo};

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < kKSlots; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < kVSlots; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_empty, kDqWarps);
    mbar_init(dp_full, 1);
    mbar_init(dp_empty, kDqWarps);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ds_full[b], kDqWarps);
      mbar_init(&ds_empty[b], 1);
    }
    mbar_init(dq_full, 1);
    mbar_init(dq_empty, kDqWarps);
    mbar_init(x_bar, kDqWarps);
    mbar_init(rows_full, 2);
    mbar_init(rows_empty, kDqWarps);
    mbar_init(done_bar, 1);
    for (int q = 0; q < 4; ++q) flags[q] = 0;
    *redo_list = RedoList{kRedoNone, 0};
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (threadIdx.x == 64) {
    queue.init(kDqWarps + 3);
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  await_previous();   // D and the list
  if (blockIdx.x == 0) check_docs(A.cu, A.batch, A.T, status);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA loads
    bool ok = true;
    int pos = 0, nq = 0;    // key tiles and items started
    DqItem it = first_item(P);
    for (int n = 0; lane == 0 && ok && it.shard >= 0; ++n) {
      DqItem coming = {};
      coming.shard = -1;
      auto announce = [&]() {
        if (A.q_list) {
          const int at = static_cast<int>(gridDim.x) + atomicAdd(A.q_taken, 1);
          if (at < total) coming = listed_item(P, at);
        }
        ok = queue.announce(n + 1, coming);
      };
      const int when = max(it.jbeg, it.jend - kLead);
      if (it.jend <= it.jbeg) {
        announce();
      } else {
        ok = wait_on(q_empty, (static_cast<uint32_t>(nq) & 1u) ^ 1u, abort_flag, status, tmo);
        if (ok) {
          mbar_arrive_expect_tx(q_full, 2 * C::TILE);
          for (int kb = 0; kb < C::KB; ++kb) {
            tma_load_2d(sQ + kb * 16384, &P.m.q[it.shard], q_full, it.c * D + kb * 64, it.q0);
            tma_load_2d(sDO + kb * 16384, &P.m.dO[it.shard], q_full, it.c * D + kb * 64, it.q0);
          }
          ++nq;
        }
        for (int j = it.jbeg; ok && j < it.jend; ++j, ++pos) {
          const int ks = pos % kKSlots, vs = pos % kVSlots;
          ok = wait_on(&k_empty[ks], (static_cast<uint32_t>(pos / kKSlots) & 1u) ^ 1u, abort_flag, status, tmo);
          if (!ok) break;
          mbar_arrive_expect_tx(&k_full[ks], C::TILE);
          for (int kb = 0; kb < C::KB; ++kb)
            tma_load_2d(sK + ks * C::TILE + kb * 16384, &P.m.k[it.shard], &k_full[ks], it.g * D + kb * 64, j * kTile);
          // (K was started: from here the position counts as started even if the wait for V fails)
          ok = wait_on(&v_empty[vs], (static_cast<uint32_t>(pos / kVSlots) & 1u) ^ 1u, abort_flag, status, tmo);
          if (!ok) {
            int dummy = 0;
            wait_on(&k_full[ks], static_cast<uint32_t>(pos / kKSlots) & 1u, reinterpret_cast<volatile int*>(&dummy),
                      status, tmo);
            break;
          }
          mbar_arrive_expect_tx(&v_full[vs], C::TILE);
          for (int kb = 0; kb < C::KB; ++kb)
            tma_load_2d(sV + vs * C::TILE + kb * 16384, &P.m.v[it.shard], &v_full[vs], it.g * D + kb * 64, j * kTile);
          if (j == when) announce();
        }
      }
      it = coming;
    }
    if (lane == 0) {
      // No copy may still be landing when the CTA leaves: wait (bounded) for the last loads.
      int dummy = 0;
      volatile int* da = reinterpret_cast<volatile int*>(&dummy);
      if (nq > 0) wait_on(q_full, static_cast<uint32_t>(nq - 1) & 1u, da, status, tmo);
      for (int i = pos > kKSlots ? pos - kKSlots : 0; i < pos; ++i)
        wait_on(&k_full[i % kKSlots], static_cast<uint32_t>(i / kKSlots) & 1u, da, status, tmo);
      for (int i = pos > kVSlots ? pos - kVSlots : 0; i < pos; ++i)
        wait_on(&v_full[i % kVSlots], static_cast<uint32_t>(i / kVSlots) & 1u, da, status, tmo);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMAs
    // The whole warp runs this loop, one elected lane issues.  A wait that runs out is in the status word and raises
    // the abort flag, after which every wait returns at once: the loop then ends over what is in memory.
    int p = 0, nq = 0;                     // key tiles scored, items
    int ks = 0, klap = 0, old = 0;         // K place of the tile about to be scored; of the one before
    const uint64_t qd = smem_desc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t dod = smem_desc_sw128(smem_u32(sDO), 16, 1024);
    const uint64_t kd0 = smem_desc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t kn0 = smem_desc_sw128(smem_u32(sK), 16384, 1024);
    const uint64_t vd0 = smem_desc_sw128(smem_u32(sV), 16, 1024);
    const uint32_t idesc_s = idesc_bf16_f32(kTile, kTile, false, false);
    const uint32_t idesc_dq = idesc_bf16_f32(kTile, D, false, true);
    static_assert(kVSlots == 2, "the V place is the parity of the key tile");
    const bool leader = elect_one();
    auto wait = [&](uint64_t* bar, int phase) {
      wait_on(bar, static_cast<uint32_t>(phase) & 1u, abort_flag, status, tmo);
    };
    DqItem it = first_item(P);
    for (int n = 0; queue.next(n, it) && it.shard >= 0; ++n) {
      const int nt = it.jend - it.jbeg;
      if (nt <= 0) continue;
      wait(q_full, nq);
      tc_fence_after_sync();
      ++nq;
      for (int j = -1; j < nt; ++j) {
        const int ds = p - 1;              // the key tile of dS_j: the last one scored before this step
        if (j + 1 < nt) {
          const int vs = p & 1;
          wait(&k_full[ks], klap);
          wait(s_empty, p + 1);
          tc_fence_after_sync();
          const uint64_t kd = desc_advance(kd0, ks * C::TILE);
          if (leader) {
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_bf16(tmem, desc_advance(qd, kb * 16384 + kk * 32), desc_advance(kd, kb * 16384 + kk * 32), idesc_s,
                          (kb | kk) ? 1u : 0u);
            umma_commit(s_full);
          }
          wait(&v_full[vs], p >> 1);
          wait(dp_empty, p + 1);
          tc_fence_after_sync();
          const uint64_t vd = desc_advance(vd0, vs * C::TILE);
          if (leader) {
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_bf16(tmem + T_DP, desc_advance(dod, kb * 16384 + kk * 32), desc_advance(vd, kb * 16384 + kk * 32),
                          idesc_s, (kb | kk) ? 1u : 0u);
            umma_commit(dp_full);
            umma_commit(&v_empty[vs]);
            if (j + 2 == nt) umma_commit(q_empty);   // the item's last read of Q and dO
          }
        }
        if (j >= 0) {
          const int b = ds & 1;
          wait(&ds_full[b], ds >> 1);
          // the previous item's dQ has been read before this one's first product overwrites it
          if (j == 0) wait(dq_empty, nq);
          tc_fence_after_sync();
          const uint64_t kd = desc_advance(kn0, old * C::TILE);
          const uint32_t more = j > 0 ? 1u : 0u;
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              umma_bf16_ts(tmem + T_DQ, tmem + T_DS + b * 64 + kk * 8, desc_advance(kd, kk * 2048), idesc_dq,
                           kk ? 1u : more);
            umma_commit(&ds_empty[b]);
            umma_commit(&k_empty[old]);
            if (j + 1 == nt) umma_commit(dq_full);
          }
        }
        __syncwarp();
        if (j + 1 < nt) {
          ++p;
          old = ks;
          if (++ks == kKSlots) {
            ks = 0;
            ++klap;
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
    // ------------------------------------------------------------------ lse, D and first keys of 64 rows
    const int r0 = (warp - 2) * 64;
    const int T = static_cast<int>(A.T);
    bool ok = true;
    DqItem it = first_item(P);
    for (int n = 0; ok && queue.next(n, it) && it.shard >= 0; ++n) {
      const PackShard& S = A.s[it.shard];
      int lo[2];
      float nl[2], Dr[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = it.q0 + r0 + u * 32 + lane;
        DocRange doc{0, 0};
        if (it.jend > it.jbeg) doc = doc_of(A.cu, A.batch, T, i);
        const bool in = doc.hi > doc.lo;
        lo[u] = in ? doc.lo : 0x7fffffff;        // a token of no document has no keys
        const int64_t row = static_cast<int64_t>(it.c) * A.T + i;
        nl[u] = in ? -__ldg(S.lse + row) * kLog2e : 0.0f;
        Dr[u] = in ? __ldg(A.D + static_cast<int64_t>(it.shard) * A.nql * A.T + row) : 0.0f;
      }
      ok = wait_on(rows_empty, (static_cast<uint32_t>(n) & 1u) ^ 1u, abort_flag, status, tmo);
      if (!__all_sync(0xffffffffu, ok)) break;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        row_lo[r0 + u * 32 + lane] = lo[u];
        row_nl[r0 + u * 32 + lane] = nl[u];
        row_D[r0 + u * 32 + lane] = Dr[u];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(rows_full);
    }
  } else {
    // ------------------------------------------------------------------ dS
    const int quad = warp & 3;
    const int g = (warp - 4) >> 2;             // keys [32 g, 32 g + 32) of each tile
    const int r = quad * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const float k2 = A.scale * kLog2e;
    const int T = static_cast<int>(A.T);
    bool ok = true;
    int pos = 0, no = 0;
    uint32_t met = 0;
    // All elementwise warps meet (a bounded wait, unlike a hardware barrier).
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(x_bar);
      const bool in_time = mbar_wait(x_bar, met & 1u, abort_flag, status, tmo);
      ++met;
      return static_cast<bool>(__all_sync(0xffffffffu, in_time));
    };
    DqItem it = first_item(P);
    for (int n = 0; ok && queue.next(n, it) && it.shard >= 0; ++n) {
      const PackShard& S = A.s[it.shard];
      const int i = it.q0 + r;
      ok = mbar_wait(rows_full, static_cast<uint32_t>(n) & 1u, abort_flag, status, tmo);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      const int lo = row_lo[r];                      // the row sees the keys lo..hi
      const float nl = row_nl[r], Di = row_D[r];
      __syncwarp();
      if (lane == 0) mbar_arrive(rows_empty);
      const bool in = lo != 0x7fffffff;              // a row of a document (so i < T)
      const int hi = in ? i : -1;
      const int lo_max = __reduce_max_sync(0xffffffffu, lo), hi_min = __reduce_min_sync(0xffffffffu, hi);
      const uint64_t kk2 = f2_pack(k2, k2), nl2 = f2_pack(nl, nl), nD2 = f2_pack(-Di, -Di);
      for (int j = it.jbeg; ok && j < it.jend; ++j, ++pos) {
        ok = mbar_wait(s_full, static_cast<uint32_t>(pos) & 1u, abort_flag, status, tmo);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        uint32_t s[32];
        tmem_ld_32x32b_x32(lane_base + g * 32, s);
        tmem_ld_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(s_empty);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 a = f2_unpack(ffma2(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), kk2, nl2));
          s[e] = __float_as_uint(ex2_approx(a.x));
          s[e + 1] = __float_as_uint(ex2_approx(a.y));
        }
        ok = mbar_wait(dp_full, static_cast<uint32_t>(pos) & 1u, abort_flag, status, tmo);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        uint32_t dp[32];
        tmem_ld_32x32b_x32(lane_base + T_DP + g * 32, dp);
        tmem_ld_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(dp_empty);
        uint32_t ds[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const uint64_t d2 = fadd2(f2_pack(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])), nD2);
          const float2 v = f2_unpack(fmul2(d2, f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1]))));
          ds[e >> 1] = pack_bf16x2(v.x, v.y);
        }
        const int k0 = j * kTile + g * 32;
        if (k0 < lo_max || k0 + 31 > hi_min) {   // some row of the warp does not see every key: its dS is 0
          const uint32_t see = bits_between(lo - k0, hi - k0);
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            ds[e >> 1] &= ((see >> e) & 1u ? 0x0000ffffu : 0u) | ((see >> (e + 1)) & 1u ? 0xffff0000u : 0u);
        }
        const int b = pos & 1;
        ok = mbar_wait(&ds_empty[b], (static_cast<uint32_t>(pos >> 1) & 1u) ^ 1u, abort_flag, status, tmo);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        tmem_st_32x32b_x16(lane_base + T_DS + b * 64 + g * 16, ds);
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ds_full[b]);
      }
      if (!ok) break;
      const bool computed = it.jend > it.jbeg;
      if (computed) {
        ok = mbar_wait(dq_full, static_cast<uint32_t>(no) & 1u, abort_flag, status, tmo);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        ++no;
        tc_fence_after_sync();
      }
      float bad = 0.0f;   // becomes NaN with the first value that is not finite
      if (g < D / 32) {   // 32 of the head's columns
        uint32_t o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0;
        if (computed) {
          tmem_ld_32x32b_x32(lane_base + T_DQ + g * 32, o);
          tmem_ld_wait();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float v = in ? __uint_as_float(o[e]) * A.scale : 0.0f;
          bad = fmaf(v, 0.0f, bad);
          o[e] = __float_as_uint(v);
        }
        if (i < T) store_bf16x32(S.dq + i * A.lddq + it.c * D + g * 32, o);
      }
      if (computed) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(dq_empty);
      }
      // A row is listed, by the first warpgroup, if any found its columns not finite.
      const unsigned mine = __ballot_sync(0xffffffffu, in && bad != 0.0f);
      if (mine && lane == 0) atomicOr(&flags[quad], mine);
      if (!(ok = meet())) break;
      if (g == 0) {
        const unsigned again = flags[quad];
        __syncwarp();
        if (again && lane == 0) {
          flags[quad] = 0;
          redo_later(A.redo, redo_list, redo_slot(it.shard * A.nql + it.c, A.T, it.q0, quad), again);
        }
      }
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (warp >= 4 && redo_list->count > 0 && !*abort_flag) redo_rows<D>(A, *redo_list, warp - 4, kDqWarps, lane);
}

}  // namespace

int pack_attn_dq_launch(const PackArgs& A, const PackMaps& maps, int d, cudaStream_t stream) {
  DqParams P;
  P.a = A;
  P.m = maps;
  const int64_t qc = static_cast<int64_t>(A.nql) * d, kc = static_cast<int64_t>(A.nkvl) * d;
  int rc = TTL_OK;
  P.tiles = static_cast<int>((A.T + kTile - 1) / kTile);
  P.lanes = A.t * A.nql;
  P.timeout_ns = pack_wait_ns(P.tiles);
  const int64_t items = static_cast<int64_t>(P.tiles) * P.lanes;
  if (items >= (int64_t(1) << 30)) return set_error(TTL_ERR_SHAPE, "packed attention: too many query tiles");
  const int sms = num_sms();
  const unsigned grid = static_cast<unsigned>(items < sms ? items : sms);
  const double tri = static_cast<double>(A.T) * (A.T + 1) / 2.0;   // one document: the lengths are on the device
  TraceScope trace(stream, TTL_K_ATTN_CORE, 6.0 * tri * d * A.nql * A.t, 2.0 * A.T * (4.0 * qc + 2.0 * kc) * A.t);
  if (d == 128) {
    if ((rc = allow_smem<pack_dq_kernel<128>>(DqCfg<128>::SMEM, "cudaFuncSetAttribute(packed attention dQ)")))
      return rc;
    rc = cuda_check(launch_after(pack_dq_kernel<128>, dim3(grid), kDqThreads, DqCfg<128>::SMEM, stream, P), "pack_dq_kernel launch");
  } else {
    if ((rc = allow_smem<pack_dq_kernel<64>>(DqCfg<64>::SMEM, "cudaFuncSetAttribute(packed attention dQ)")))
      return rc;
    rc = cuda_check(launch_after(pack_dq_kernel<64>, dim3(grid), kDqThreads, DqCfg<64>::SMEM, stream, P), "pack_dq_kernel launch");
  }
  return rc;
}

}  // namespace ttl
