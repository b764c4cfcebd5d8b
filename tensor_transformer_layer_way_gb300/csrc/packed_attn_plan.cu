// Work lists of the packed attention kernels.
//
// A query tile's work is the number of key tiles it meets, a key tile's the number of (query tile, head) steps;
// both depend on the documents, which only the device knows.  One CTA sorts the tiles by work, heaviest first
// (a counting sort; tiles of equal work in any order), so that the persistent kernels, which take items in
// turn, end together, and cuts the longest key tiles into several items where there are few.  Worth it only
// when there are more items than SMs; below that every item starts at once.  The backward pass's launch also takes
// D = rowsum(dO o) of every row and head, in the other CTAs: the sort is hidden under it
// (8192 tokens, 32 heads of 128: 134 MB in 23 us, 86% of the copy rate; the sort alone takes 5).

#include "packed_attn.cuh"

namespace ttl {
namespace {

constexpr int kPlanThreads = 1024;

// First key tile that token tile `tile` meets, or -1.
__device__ __forceinline__ int first_key_tile(const PackArgs& A, int tile) {
  const int T = static_cast<int>(A.T);
  if (A.batch == 0 || static_cast<int64_t>(tile) * kTile >= A.T) return -1;
  const int q0 = tile * kTile, first = __ldg(A.cu), last = __ldg(A.cu + A.batch);
  const int v0 = q0 > first ? q0 : first;
  int v1 = q0 + kTile < last ? q0 + kTile : last;
  v1 = v1 < T ? v1 : T;
  return v0 < v1 ? doc_of(A.cu, A.batch, T, v0).lo / kTile : -1;
}

// Last query tile that key tile `tile` meets, or tile - 1.
__device__ __forceinline__ int last_query_tile(const PackArgs& A, int tile) {
  const int T = static_cast<int>(A.T);
  if (A.batch == 0) return tile - 1;
  const int k0 = tile * kTile, first = __ldg(A.cu), last = __ldg(A.cu + A.batch);
  const int v0 = k0 > first ? k0 : first;
  int v1 = k0 + kTile < last ? k0 + kTile : last;
  v1 = v1 < T ? v1 : T;
  if (v0 >= v1) return tile - 1;
  const int hi = doc_of(A.cu, A.batch, T, v1 - 1).hi;
  return (hi > v1 ? hi - 1 : v1 - 1) / kTile;
}

// hist[b] entries of work class b become places, the highest class first.  Every thread calls it.
__device__ __forceinline__ void to_places(int* hist, int* warp_tot) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  __syncthreads();
  const int mine = hist[kPlanThreads - 1 - threadIdx.x];
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warp_tot[w] = inc;
  __syncthreads();
  int base = inc - mine;
  for (int j = 0; j < w; ++j) base += warp_tot[j];
  hist[kPlanThreads - 1 - threadIdx.x] = base;
  __syncthreads();
}

__device__ __forceinline__ int work_class(int work, int shift) {
  const int c = work >> shift;
  return c < kPlanThreads ? c : kPlanThreads - 1;
}

// D of one token of one shard, all its heads, by a warp: 256 columns at a time, d / 8 lanes for each head.
template <int D>
__device__ __forceinline__ void row_dots(const PackArgs& A, int shard, int64_t i) {
  constexpr int kLanes = D / 8, kHeads = 256 / D;   // lanes of a head, heads of 256 columns
  const int lane = threadIdx.x & 31;
  const PackShard& S = A.s[shard];
  const __nv_bfloat16* a_at = S.dO + i * A.lddo + lane * 8;
  const __nv_bfloat16* b_at = S.o + i * A.ldo + lane * 8;
  int head = lane / kLanes;
  float* out = A.D + (static_cast<int64_t>(shard) * A.nql + head) * A.T + i;
#pragma unroll 2
  for (; head - lane / kLanes < A.nql; head += kHeads, a_at += 256, b_at += 256, out += kHeads * A.T) {
    float acc = 0.0f;
    if (head < A.nql) {
      const uint4 a = __ldcs(reinterpret_cast<const uint4*>(a_at)), b = __ldcs(reinterpret_cast<const uint4*>(b_at));
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) acc = fmaf(bf16_lo(aw[w]), bf16_lo(bw[w]), fmaf(bf16_hi(aw[w]), bf16_hi(bw[w]), acc));
    }
#pragma unroll
    for (int o = kLanes >> 1; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (head < A.nql && lane % kLanes == 0) *out = acc;
  }
}

__global__ void __launch_bounds__(kPlanThreads) pack_plan_kernel(const __grid_constant__ PackArgs A,
                                                                 const __grid_constant__ PackPlan P, int q_shift,
                                                                 int kv_shift, int d, unsigned blocks) {
  __shared__ int hist[kPlanThreads];
  __shared__ int warp_tot[32];
  __shared__ unsigned long long total;
  __shared__ int taken, joins, longest;
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    const unsigned shard = (blockIdx.x - 1) / blocks;
    const int64_t i = static_cast<int64_t>(blockIdx.x - 1 - shard * blocks) * (kPlanThreads / 32) + (tid >> 5);
    if (i < A.T) {
      if (d == 128) row_dots<128>(A, static_cast<int>(shard), i);
      else row_dots<64>(A, static_cast<int>(shard), i);
    }
    return;
  }
  if (P.q_list) {
    if (tid == 0) *P.q_taken = 0;
    hist[tid] = 0;
    __syncthreads();
    for (int pass = 0; pass < 2; ++pass) {
      for (int u = tid; u < P.q_units; u += kPlanThreads) {
        const int t0 = u * P.q_per;
        const int a = first_key_tile(A, t0), b = P.q_per == 2 ? first_key_tile(A, t0 + 1) : -1;
        const int work = (a < 0 ? 0 : t0 + 1 - a) + (b < 0 ? 0 : t0 + 2 - b);
        const int at = atomicAdd(&hist[work_class(work, q_shift)], 1);
        if (pass) P.q_list[at] = make_int4(u, a, b, 0);
      }
      if (pass == 0) to_places(hist, warp_tot);
    }
    __syncthreads();
  }
  if (P.kv_list) {
    hist[tid] = 0;
    if (tid == 0) {
      total = 0;
      taken = joins = longest = 0;
    }
    __syncthreads();
    unsigned long long sum = 0;
    int most_here = 0;
    for (int t = tid; t < P.tiles; t += kPlanThreads) {
      const int steps = (last_query_tile(A, t) - t + 1) * A.grp;
      sum += static_cast<unsigned long long>(steps);
      most_here = steps > most_here ? steps : most_here;
    }
    atomicAdd(&total, sum);
    atomicMax(&longest, most_here);
    __syncthreads();
    // Where a whole key tile would be more than an SM's share of all steps, no item is longer than a third of
    // that share.  (A part costs a write and a read of its fp32 sums: with every tile below the share,
    // cutting took 24 us and won nothing.)
    unsigned long long most = 0x7fffffffull;
    if (P.split && 3ull * static_cast<unsigned long long>(longest) * kSplitItems > 9ull * total * P.lanes) {
      most = (total * P.lanes + kSplitItems - 1) / kSplitItems;
      if (most < kSplitSteps) most = kSplitSteps;
    }
    for (int pass = 0; pass < 2; ++pass) {
      for (int t = tid; t < P.tiles; t += kPlanThreads) {
        const int last = last_query_tile(A, t);
        const int steps = (last - t + 1) * A.grp;
        const int parts = steps > 0 ? static_cast<int>((steps + most - 1) / most) : 1;
        const int len = (steps + parts - 1) / parts;
        const int at = atomicAdd(&hist[work_class(len, kv_shift)], parts);
        if (pass) {
          int slot = -1;
          if (parts > 1) {
            slot = atomicAdd(&taken, parts);
            P.join_list[atomicAdd(&joins, 1)] = make_int4(t, slot, parts, 0);
          }
          for (int p = 0; p < parts; ++p) {
            const int b = p * len, e = b + len < steps ? b + len : steps;
            P.kv_list[2 * (at + p)] = make_int4(t, last, b < steps ? b : steps, e);
            P.kv_list[2 * (at + p) + 1] = make_int4(slot < 0 ? -1 : slot + p, 0, 0, 0);
          }
        }
      }
      if (pass == 0) {
        to_places(hist, warp_tot);
      }
    }
    __syncthreads();
    if (tid == 0) P.kv_head[1] = joins;
    // the number of entries: all places given out
    int entries = 0;
    for (int t = tid; t < P.tiles; t += kPlanThreads) {
      const int steps = (last_query_tile(A, t) - t + 1) * A.grp;
      entries += steps > 0 ? static_cast<int>((steps + most - 1) / most) : 1;
    }
    if (tid == 0) taken = 0;
    __syncthreads();
    atomicAdd(&taken, entries);
    __syncthreads();
    if (tid == 0) {
      P.kv_head[0] = taken;
      *P.kv_taken = 0;
    }
  }
}

}  // namespace

int pack_attn_plan_launch(const PackArgs& A, const PackPlan& plan, int d, cudaStream_t stream) {
  const int tiles = static_cast<int>((A.T + kTile - 1) / kTile);
  int q_shift = 0, kv_shift = 0;
  while ((2 * static_cast<int64_t>(tiles) >> q_shift) >= kPlanThreads) ++q_shift;
  while ((static_cast<int64_t>(tiles) * A.grp >> kv_shift) >= kPlanThreads) ++kv_shift;
  // d > 0: with D, one warp per (shard, token) and `blocks` blocks a shard
  const int64_t rows = d > 0 ? A.t * A.T : 0;
  TraceScope trace(stream, TTL_K_OTHER, 0.0, 32.0 * tiles + 4.0 * rows * A.nql * d);
  const unsigned blocks = d > 0 ? static_cast<unsigned>((A.T + kPlanThreads / 32 - 1) / (kPlanThreads / 32)) : 0;
  const unsigned grid = 1 + blocks * A.t;
  pack_plan_kernel<<<grid, kPlanThreads, 0, stream>>>(A, plan, q_shift, kv_shift, d, blocks);
  return cuda_check(cudaGetLastError(), "pack_plan_kernel launch");
}

}  // namespace ttl
