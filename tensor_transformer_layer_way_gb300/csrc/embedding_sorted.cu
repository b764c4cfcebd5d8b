// Scaled vocab-parallel embedding lookup, and its table gradient summed by sorted tokens.
//
// Source: "v4:Tensor Parallel 与 Sequence Parallel", section "Embedding 和 LM head:按 vocab 切":
// shard i owns ids [i V/t, (i+1) V/t) and after the all-reduce every shard has every token's row.
//
// Forward:   out[tok] = bf16(scale E[id(tok)]), one rounding, into all t buffers.
// Backward:  dE[v] (+)= scale sum over the tokens of id v of dY[tok], in fp32.
// The token indices are sorted by id (a stable radix sort, so the tokens of one id stay in
// token order); a run of equal ids is then summed by whole CTAs in chunks of fixed length, and the
// partial sums of a run that crosses chunks are joined in a fixed order.  No atomic adds to the gradient: the
// same inputs give the same bits, and a row of the gradient is written once.
//
// What bounds it: the table's bytes where every row is written (8192 tokens, 151936 x 4096: 2.5 GB, 400 us, 94% of
// the copy rate), else the tokens' rows; the sort is latency.  Up to 16384 tokens it is one CTA in shared memory, and
// the other CTAs of the same launch write the zeros of the rows that no token has meanwhile; beyond that three
// launches per digit, and zeros everywhere first.  A few tokens of few columns need no sort: one launch.

#include "launch_after.cuh"
#include "operands.h"
#include "ttl_device.cuh"
#include "ttl_internal.h"

namespace ttl {
namespace {

struct ScaledTables {
  const uint4* e[kMaxShards];
};
struct ScaledOut {
  uint4* o[kMaxShards];
};
struct GradTables {
  float* g[kMaxShards];
};

__device__ __forceinline__ uint32_t scale2(uint32_t v, float s) { return pack_bf16x2(bf16_lo(v) * s, bf16_hi(v) * s); }

// grid T: token `tok`'s row, scaled, from its owning shard into every output buffer.
__global__ void __launch_bounds__(256) embed_scaled_kernel(const __grid_constant__ ScaledTables E,
                                                           const __grid_constant__ ScaledOut O, const int64_t* ids,
                                                           int t, int64_t h8, int64_t Vs, int64_t V, float scale,
                                                           int* status) {
  const int64_t tok = blockIdx.x;
  const int64_t id = ids[tok];
  const bool valid = id >= 0 && id < V;
  if (!valid && threadIdx.x == 0) atomicCAS(status, 0, TTL_ERR_DEVICE);
  const int owner = valid ? static_cast<int>(id / Vs) : 0;
  const uint4* src = E.e[owner] + (valid ? (id - owner * Vs) : 0) * h8;
  for (int64_t k = threadIdx.x; k < h8; k += blockDim.x) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (valid) {
      v = __ldg(src + k);
      v = make_uint4(scale2(v.x, scale), scale2(v.y, scale), scale2(v.z, scale), scale2(v.w, scale));
    }
    for (int j = 0; j < t; ++j) __stcs(O.o[j] + tok * h8 + k, v);
  }
}

// ------------------------------------------------------------------ stable radix sort of (id, token)

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortRounds = 8;                               // keys per lane
constexpr int kSortBlock = kSortThreads * kSortRounds;       // keys per CTA: 256 consecutive ones per warp
constexpr int kRadix = 256;

// The key of a token: its id, or V (sorted last, summed nowhere) for an id outside [0, V).
__device__ __forceinline__ uint32_t key_of(const int64_t* ids, const uint32_t* keys, int64_t k, int64_t V, int* status) {
  if (keys) return keys[k];
  const int64_t id = ids[k];
  if (id >= 0 && id < V) return static_cast<uint32_t>(id);
  atomicCAS(status, 0, TTL_ERR_DEVICE);
  return static_cast<uint32_t>(V);
}

// counts[digit * nb + block]: how many of the block's keys have the digit.  The first pass reads ids.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const int64_t* ids, const uint32_t* keys, int64_t T,
                                                                  int64_t V, int shift, uint32_t* counts, int nb,
                                                                  int* status) {
  __shared__ uint32_t hist[kRadix];
  hist[threadIdx.x] = 0;
  __syncthreads();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortBlock;
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t k = base + r * kSortThreads + threadIdx.x;
    if (k < T) atomicAdd(&hist[(key_of(ids, keys, k, V, status) >> shift) & (kRadix - 1)], 1u);
  }
  __syncthreads();
  counts[static_cast<int64_t>(threadIdx.x) * nb + blockIdx.x] = hist[threadIdx.x];
}

// Exclusive prefix sums of the n counts, in place; one CTA, each thread a contiguous range.
__global__ void __launch_bounds__(1024) sort_scan_kernel(uint32_t* counts, int64_t n, uint32_t* runs) {
  if (threadIdx.x < 2) runs[threadIdx.x] = 0;   // the lists of runs to be joined, filled by the sums
  __shared__ uint32_t warp_tot[32];
  const int64_t per = (n + 1023) / 1024;
  const int64_t lo = threadIdx.x * per < n ? threadIdx.x * per : n, hi = lo + per < n ? lo + per : n;
  uint32_t sum = 0;
  for (int64_t k = lo; k < hi; ++k) sum += counts[k];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warp_tot[w] = inc;
  __syncthreads();
  uint32_t run = inc - sum;
  for (int j = 0; j < w; ++j) run += warp_tot[j];
  for (int64_t k = lo; k < hi; ++k) {
    const uint32_t c = counts[k];
    counts[k] = run;
    run += c;
  }
}

// Moves each key and its token to its place.  A warp owns 256 consecutive keys and goes through
// them 32 at a time; lanes with the same digit are ranked by lane, so the order of equal digits
// is kept.
__global__ void __launch_bounds__(kSortThreads) sort_move_kernel(const int64_t* ids, const uint32_t* keys,
                                                                 const uint32_t* toks, int64_t T, int64_t V, int shift,
                                                                 const uint32_t* counts, int nb, uint32_t* keys_out,
                                                                 uint32_t* toks_out, int* status) {
  __shared__ uint32_t at[kSortWarps][kRadix];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (int d = lane; d < kRadix; d += 32) at[w][d] = 0;
  __syncwarp();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortBlock + w * (32 * kSortRounds);
  uint32_t key[kSortRounds];
  uint32_t peers[kSortRounds];
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t k = base + r * 32 + lane;
    const bool in = k < T;
    key[r] = in ? key_of(ids, keys, k, V, status) : 0xffffffffu;
    const uint32_t d = in ? (key[r] >> shift) & (kRadix - 1) : kRadix;   // past the end: a digit of its own
    peers[r] = __match_any_sync(0xffffffffu, d);
    if (in && lane == __ffs(peers[r]) - 1) at[w][d] += __popc(peers[r]);
    __syncwarp();
  }
  __syncthreads();
  {   // first place of each warp's keys of digit d = threadIdx.x
    uint32_t run = counts[static_cast<int64_t>(threadIdx.x) * nb + blockIdx.x];
#pragma unroll
    for (int j = 0; j < kSortWarps; ++j) {
      const uint32_t c = at[j][threadIdx.x];
      at[j][threadIdx.x] = run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t k = base + r * 32 + lane;
    const bool in = k < T;
    const uint32_t d = (key[r] >> shift) & (kRadix - 1);
    uint32_t place = 0;
    if (in) place = at[w][d] + __popc(peers[r] & ((1u << lane) - 1u));
    __syncwarp();
    if (in && lane == __ffs(peers[r]) - 1) at[w][d] += __popc(peers[r]);
    __syncwarp();
    if (in) {
      keys_out[place] = key[r];
      toks_out[place] = toks ? toks[k] : static_cast<uint32_t>(k);
    }
  }
}

// ------------------------------------------------------------------ sort in one CTA, zeros in the others

constexpr int kOneThreads = 1024;
constexpr int kOneWarps = kOneThreads / 32;
constexpr int kOneMost = 16384;      // tokens: two buffers of keys and of 16-bit tokens, and a count per warp and digit
constexpr size_t kOneSmem = 2 * kOneMost * 4 + 2 * kOneMost * 2 + kOneWarps * kRadix * 2;

// Lanes of the warp with the same `bits` low bits of d (one vote per bit), among the lanes of `in`.
__device__ __forceinline__ uint32_t same_digit(uint32_t d, int bits, uint32_t in) {
  uint32_t peers = in;
  for (int b = 0; b < bits; ++b) {
    const uint32_t m = __ballot_sync(0xffffffffu, (d >> b) & 1u);
    peers &= (d >> b) & 1u ? m : ~m;
  }
  return peers;
}

// CTA 0: the stable radix sort of the T <= 1024 R keys, `bits` bits at a time; a warp owns 32 R consecutive keys.
template <int R>
__device__ void sort_one(const int64_t* ids, int T, int64_t V, int passes, int bits, uint32_t* keys_out,
                         uint32_t* toks_out, int* status, uint8_t* smem) {
  uint32_t* key[2] = {reinterpret_cast<uint32_t*>(smem), reinterpret_cast<uint32_t*>(smem) + kOneMost};
  uint16_t* tok[2] = {reinterpret_cast<uint16_t*>(key[1] + kOneMost), reinterpret_cast<uint16_t*>(key[1] + kOneMost) + kOneMost};
  uint16_t* at = tok[1] + kOneMost;                          // [warp][digit]
  __shared__ uint32_t warp_tot[kRadix / 32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int base = w * (32 * R);
  const uint32_t mask = (1u << bits) - 1u;
  uint32_t k[R];
  uint16_t tk[R];
  {
    int64_t id[R];
#pragma unroll
    for (int r = 0; r < R; ++r) id[r] = base + r * 32 + lane < T ? __ldg(ids + base + r * 32 + lane) : 0;
    bool bad = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool in = base + r * 32 + lane < T, valid = id[r] >= 0 && id[r] < V;
      bad |= in && !valid;
      k[r] = static_cast<uint32_t>(valid ? id[r] : V);
      tk[r] = static_cast<uint16_t>(base + r * 32 + lane);
    }
    if (bad) atomicCAS(status, 0, TTL_ERR_DEVICE);
  }
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * bits;
    uint32_t* ko = key[pass & 1];
    uint16_t* to = tok[pass & 1];
    for (int d = lane; d < kRadix / 2; d += 32) reinterpret_cast<uint32_t*>(at + w * kRadix)[d] = 0;
    __syncwarp();
    uint32_t peers[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool in = base + r * 32 + lane < T;
      const uint32_t d = (k[r] >> shift) & mask;
      peers[r] = same_digit(d, bits, __ballot_sync(0xffffffffu, in));
      if (in && lane == __ffs(peers[r]) - 1) at[w * kRadix + d] += static_cast<uint16_t>(__popc(peers[r]));
      __syncwarp();
    }
    __syncthreads();
    // first place of warp w's keys of digit d: all smaller digits, then this digit's in the warps before
    uint32_t mine = 0, inc = 0;
    if (tid < kRadix) {
#pragma unroll
      for (int j = 0; j < kOneWarps; ++j) mine += at[j * kRadix + tid];
      inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) warp_tot[w] = inc;
    }
    __syncthreads();
    if (tid < kRadix) {
      uint32_t run = inc - mine;
      for (int j = 0; j < w; ++j) run += warp_tot[j];
#pragma unroll
      for (int j = 0; j < kOneWarps; ++j) {
        const uint32_t c = at[j * kRadix + tid];
        at[j * kRadix + tid] = static_cast<uint16_t>(run);
        run += c;
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool in = base + r * 32 + lane < T;
      const uint32_t d = (k[r] >> shift) & mask;
      uint32_t place = 0;
      if (in) place = at[w * kRadix + d] + __popc(peers[r] & ((1u << lane) - 1u));
      __syncwarp();
      if (in && lane == __ffs(peers[r]) - 1) at[w * kRadix + d] += static_cast<uint16_t>(__popc(peers[r]));
      __syncwarp();
      if (in) {
        if (pass + 1 == passes) {
          keys_out[place] = k[r];
          toks_out[place] = tk[r];
        } else {
          ko[place] = k[r];
          to[place] = tk[r];
        }
      }
    }
    if (pass + 1 < passes) {
      __syncthreads();
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int i = base + r * 32 + lane;
        if (i < T) {
          k[r] = ko[i];
          tk[r] = to[i];
        }
      }
    }
  }
}

// The other CTAs: zeros for the rows of a slice of the vocabulary that no token has.
__device__ void fill_slice(const GradTables& G, const int64_t* ids, int T, int64_t V, int64_t Vs, int64_t h, int cta,
                           int ctas, uint8_t* smem) {
  uint32_t* seen = reinterpret_cast<uint32_t*>(smem);
  const int64_t per = (V + ctas - 1) / ctas;
  const int64_t lo = cta * per < V ? cta * per : V, hi = lo + per < V ? lo + per : V;
  const int words = static_cast<int>((hi - lo + 31) / 32);
  for (int k = threadIdx.x; k < words; k += kOneThreads) seen[k] = 0;
  __syncthreads();
  for (int k = threadIdx.x; k < T; k += kOneThreads) {
    const int64_t id = ids[k];
    if (id >= lo && id < hi) atomicOr(&seen[(id - lo) >> 5], 1u << ((id - lo) & 31));
  }
  __syncthreads();
  // a warp per row
  const int64_t h4 = h / 4;
  for (int64_t v = lo + (threadIdx.x >> 5); v < hi; v += kOneWarps) {
    if ((seen[(v - lo) >> 5] >> ((v - lo) & 31)) & 1u) continue;
    const int i = static_cast<int>(v / Vs);
    float4* row = reinterpret_cast<float4*>(G.g[i] + (v - i * Vs) * h);
    for (int64_t k = threadIdx.x & 31; k < h4; k += 32) __stcs(row + k, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
  }
}

__global__ void __launch_bounds__(kOneThreads) sort_fill_kernel(const __grid_constant__ GradTables G,
                                                                const int64_t* ids, int T, int64_t V, int64_t Vs,
                                                                int64_t h, int passes, int bits, uint32_t* keys_out,
                                                                uint32_t* toks_out, uint32_t* runs, int* status) {
  extern __shared__ __align__(16) uint8_t one_smem[];
  if (blockIdx.x == 0) {
    if (threadIdx.x < 2) runs[threadIdx.x] = 0;
    if (T <= kOneThreads) sort_one<1>(ids, T, V, passes, bits, keys_out, toks_out, status, one_smem);
    else if (T <= 4 * kOneThreads) sort_one<4>(ids, T, V, passes, bits, keys_out, toks_out, status, one_smem);
    else if (T <= 8 * kOneThreads) sort_one<8>(ids, T, V, passes, bits, keys_out, toks_out, status, one_smem);
    else sort_one<16>(ids, T, V, passes, bits, keys_out, toks_out, status, one_smem);
  } else {
    fill_slice(G, ids, T, V, Vs, h, blockIdx.x - 1, gridDim.x - 1, one_smem);
  }
}

// ------------------------------------------------------------------ sums over runs of equal ids

constexpr int kSumThreads = 256;
constexpr int kMaxChunk = 1 << 20;   // places per chunk
constexpr int kShortRun = 4;         // further chunks of a run that one thread adds up alone

__device__ __forceinline__ float* row_of(const GradTables& G, uint32_t key, int64_t Vs, int64_t h) {
  const uint32_t i = key / static_cast<uint32_t>(Vs);
  return G.g[i] + static_cast<int64_t>(key - i * static_cast<uint32_t>(Vs)) * h;
}

// Eight columns of a finished row: 32 bytes, written (or added to) once.
__device__ __forceinline__ void row_out(float* dst, const float (&a)[8], float scale, int accumulate) {
  uint32_t w[8];
  float4 p = make_float4(0.0f, 0.0f, 0.0f, 0.0f), q = p;
  if (accumulate) {
    p = reinterpret_cast<const float4*>(dst)[0];
    q = reinterpret_cast<const float4*>(dst)[1];
  }
  const float old[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(accumulate ? fmaf(a[j], scale, old[j]) : a[j] * scale);
  if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
    st_global_v8(dst, w);
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Chunk b = sorted places [b C, (b + 1) C); each thread sums 8 columns, the rows of eight places loaded ahead of
// their sums.  A run that begins and ends in the chunk goes to its row of dE.  A run that began earlier leaves its
// sum in head[b]; one that begins here and goes on leaves its sum in tail[b], and the chunk in runs.
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const __grid_constant__ GradTables G,
                                                                const uint32_t* keys, const uint32_t* toks,
                                                                const __nv_bfloat16* dY, int64_t lddy, int64_t T,
                                                                int64_t h, int64_t Vs, int64_t V, int C, float scale,
                                                                int accumulate, float* head, float* tail,
                                                                uint32_t* runs) {
  constexpr int W = 128;                                     // places looked at together
  await_previous();
  __shared__ const __nv_bfloat16* src[W];
  __shared__ float* dst[W];                                  // where the run that ends at the place goes; null: it goes on
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * C, hi = lo + C < T ? lo + C : T;
  const int64_t col = (static_cast<int64_t>(blockIdx.y) * kSumThreads + threadIdx.x) * 8;
  const uint32_t first = keys[lo], last = keys[hi - 1];
  bool began = lo == 0 || keys[lo - 1] != first;
  if (blockIdx.y == 0 && threadIdx.x == 0 && last < V && hi < T && keys[hi] == last && (began || first != last)) {                                                          // (the lists' order does not matter)
    const int64_t far = (static_cast<int64_t>(blockIdx.x) + 1 + kShortRun) * C;
    if (far < T && keys[far] == last) runs[2 + gridDim.x - 1 - atomicAdd(runs + 1, 1u)] = blockIdx.x;
    else runs[2 + atomicAdd(runs, 1u)] = blockIdx.x;
  }
  float a[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) a[j] = 0.0f;
  for (int64_t w0 = lo; w0 < hi; w0 += W) {
    const int n = static_cast<int>(hi - w0 < W ? hi - w0 : W);
    if (w0 > lo) __syncthreads();
    if (static_cast<int>(threadIdx.x) < n) {
      const int64_t k = w0 + threadIdx.x;
      const uint32_t key = keys[k];
      const bool valid = key < V;                            // ids out of range are last
      src[threadIdx.x] = valid ? dY + static_cast<int64_t>(toks[k]) * lddy : nullptr;
      dst[threadIdx.x] = valid && (k + 1 == T || keys[k + 1] != key) ? row_of(G, key, Vs, h) : nullptr;
    }
    __syncthreads();
    if (col < h) {
      for (int k0 = 0; k0 < n; k0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const __nv_bfloat16* from = k0 + j < n ? src[k0 + j] : nullptr;
          v[j] = from ? __ldcs(reinterpret_cast<const uint4*>(from + col)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a[0] += bf16_lo(v[j].x); a[1] += bf16_hi(v[j].x); a[2] += bf16_lo(v[j].y); a[3] += bf16_hi(v[j].y);
          a[4] += bf16_lo(v[j].z); a[5] += bf16_hi(v[j].z); a[6] += bf16_lo(v[j].w); a[7] += bf16_hi(v[j].w);
          float* to = k0 + j < n ? dst[k0 + j] : nullptr;
          if (to) {
            if (began) {
              row_out(to + col, a, scale, accumulate);
            } else {
              float4* p = reinterpret_cast<float4*>(head + static_cast<int64_t>(blockIdx.x) * h + col);
              p[0] = make_float4(a[0], a[1], a[2], a[3]);
              p[1] = make_float4(a[4], a[5], a[6], a[7]);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) a[q] = 0.0f;
            began = true;
          }
        }
      }
    }
  }
  if (col < h && last < V && hi < T && keys[hi] == last) {   // a run goes on past the chunk
    float4* p = reinterpret_cast<float4*>((began ? tail : head) + static_cast<int64_t>(blockIdx.x) * h + col);
    p[0] = make_float4(a[0], a[1], a[2], a[3]);
    p[1] = make_float4(a[4], a[5], a[6], a[7]);
  }
}

// Joins the runs that go on past their chunk: first those that end within the next kShortRun chunks (eight columns per
// thread, the partial sums one after the other), then the longer ones, 128 columns of one run per CTA: sixteen
// lanes hold the columns, sixteen groups each every sixteenth partial sum, and the groups are added in order.
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(const __grid_constant__ GradTables G,
                                                                 const uint32_t* keys, int64_t T, int64_t h,
                                                                 int64_t Vs, int C, float scale, int accumulate,
                                                                 const float* head, const float* tail,
                                                                 const uint32_t* runs, int chunks) {
  __shared__ float red[16][16][9];
  await_previous();
  const int64_t wide = (h + kSumThreads * 8 - 1) / (kSumThreads * 8), narrow = (h + 127) / 128;
  const int64_t shorts = static_cast<int64_t>(runs[0]) * wide, items = shorts + static_cast<int64_t>(runs[1]) * narrow;
  auto add = [&](float (&a)[8], int64_t b, int64_t n, int64_t col) {
    const float4* p = reinterpret_cast<const float4*>((n == b ? tail : head) + n * h + col);
    const float4 u = p[0], v = p[1];
    a[0] += u.x; a[1] += u.y; a[2] += u.z; a[3] += u.w;
    a[4] += v.x; a[5] += v.y; a[6] += v.z; a[7] += v.w;
  };
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    float a[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = 0.0f;
    if (it < shorts) {
      const int64_t b = runs[2 + it / wide];
      const int64_t col = ((it % wide) * kSumThreads + threadIdx.x) * 8;
      if (col >= h) continue;
      const uint32_t key = keys[(b + 1) * C];
      bool in[kShortRun + 1];
#pragma unroll
      for (int n = 0; n <= kShortRun; ++n) in[n] = n < 2 || ((b + n) * C < T && keys[(b + n) * C] == key);
#pragma unroll
      for (int n = 0; n <= kShortRun; ++n)
        if (in[n]) add(a, b, b + n, col);
      row_out(row_of(G, key, Vs, h) + col, a, scale, accumulate);
      continue;
    }
    const int vec = threadIdx.x & 15, part = threadIdx.x >> 4;
    const int64_t b = runs[2 + chunks - 1 - (it - shorts) / narrow];
    const int64_t col = ((it - shorts) % narrow) * 128 + vec * 8;
    const uint32_t key = keys[(b + 1) * C];
    // the last chunk that the run enters: places are sorted, so by bisection
    int64_t l = b + 1, r = (T - 1) / C + 1;                  // keys[l C] == key; r: not, or past the end
    while (r - l > 1) {
      const int64_t m = (l + r) >> 1;
      if (keys[m * C] == key) l = m; else r = m;
    }
    if (col < h) {
#pragma unroll 4
      for (int64_t n = b + part; n <= l; n += 16) add(a, b, n, col);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) red[part][vec][j] = a[j];
    __syncthreads();
    if (part == 0 && col < h) {
      for (int p = 1; p < 16; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] += red[p][vec][j];
      row_out(row_of(G, key, Vs, h) + col, a, scale, accumulate);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ few tokens: no sort
// Each CTA owns a slice of the vocabulary and picks the tokens of its rows out of all ids, in token order.  A warp
// sums a row of few tokens, all warps one of many, each a part of the list, and the parts are added in order.  One launch
// where the sorted path takes three, but a slice's rows are one CTA's work: for calls whose tokens' rows are few
// bytes in all and the slices short.  Measured, this and the sorted path (us): 128 tokens x 256 columns, 2048 rows
// 5.2 and 11.3; 1024 x 256, half of them one id, 11.3 and 15.4; 1000 x 256, 65000 rows 19.6 and 22.1; 256 x
// 1024, half of them one id, 17.5 and 13.4; 1024 x 64, 200000 rows 33 and 27.

constexpr int kDirectThreads = 512;
constexpr int kDirectWarps = kDirectThreads / 32;
constexpr int kDirectMost = 1024;       // tokens
constexpr int kDirectWide = 512;        // columns
constexpr int kDirectRows = 65536;
constexpr int64_t kDirectWork = 1 << 18;   // tokens x columns
constexpr int kDirectFew = 8;           // tokens that one warp sums alone

// Adds columns [col, col + 8) of the row's tokens among entries [from, to) of the list, eight loads before their sums.
__device__ __forceinline__ void direct_sum(float (&a)[8], const uint32_t* list, int from, int to, uint32_t row,
                                           const __nv_bfloat16* dY, int64_t lddy, int64_t col, int64_t h) {
  const int lane = threadIdx.x & 31;
  for (int e0 = from; e0 < to; e0 += 32) {
    const uint32_t e = e0 + lane < to ? list[e0 + lane] : 0;
    unsigned m = __ballot_sync(0xffffffffu, e0 + lane < to && e / kDirectMost == row);
    while (m) {
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int at = m ? __ffs(m) - 1 : 32;
        m &= m - 1;
        const uint32_t tok = __shfl_sync(0xffffffffu, e, at & 31) % kDirectMost;
        v[u] = at < 32 && col < h ? __ldg(reinterpret_cast<const uint4*>(dY + static_cast<int64_t>(tok) * lddy + col))
                                  : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        a[0] += bf16_lo(v[u].x); a[1] += bf16_hi(v[u].x); a[2] += bf16_lo(v[u].y); a[3] += bf16_hi(v[u].y);
        a[4] += bf16_lo(v[u].z); a[5] += bf16_hi(v[u].z); a[6] += bf16_lo(v[u].w); a[7] += bf16_hi(v[u].w);
      }
    }
  }
}

__global__ void __launch_bounds__(kDirectThreads) embed_direct_kernel(const __grid_constant__ GradTables G,
                                                                      const int64_t* ids, int T, int64_t V, int64_t Vs,
                                                                      int64_t h, const __nv_bfloat16* dY, int64_t lddy,
                                                                      float scale, int accumulate, int* status) {
  __shared__ uint32_t list[kDirectMost];                   // row of the slice * kDirectMost + token
  __shared__ uint32_t many[kDirectMost / kDirectFew];      // rows of more than kDirectFew tokens
  __shared__ int found[kDirectWarps];
  __shared__ int many_n;
  __shared__ float4 part[kDirectWarps][2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t per = (V + gridDim.x - 1) / gridDim.x;
  const int64_t lo = blockIdx.x * per, hi = lo + per < V ? lo + per : V;
  if (threadIdx.x == 0) many_n = 0;
  int n = 0;                                               // entries
  for (int k0 = 0; k0 < T; k0 += kDirectThreads) {
    const int k = k0 + static_cast<int>(threadIdx.x);
    const int64_t id = k < T ? ids[k] : -1;
    if (blockIdx.x == 0 && k < T && (id < 0 || id >= V)) atomicCAS(status, 0, TTL_ERR_DEVICE);
    const bool mine = id >= lo && id < hi;
    const unsigned m = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) found[warp] = __popc(m);
    __syncthreads();
    int at = n;
#pragma unroll
    for (int w = 0; w < kDirectWarps; ++w) {
      at += w < warp ? found[w] : 0;
      n += found[w];
    }
    if (mine) list[at + __popc(m & ((1u << lane) - 1))] = static_cast<uint32_t>(id - lo) * kDirectMost + k;
    __syncthreads();
  }
  auto out = [&](int64_t r, int64_t col, const float (&a)[8]) {
    row_out(row_of(G, static_cast<uint32_t>(lo + r), Vs, h) + col, a, scale, accumulate);
  };
  for (int64_t r = warp; r < hi - lo; r += kDirectWarps) {
    int tokens = 0;
    for (int e0 = 0; e0 < n; e0 += 32)
      tokens += __popc(__ballot_sync(0xffffffffu, e0 + lane < n && list[e0 + lane] / kDirectMost == static_cast<uint32_t>(r)));
    if (tokens > kDirectFew) {
      if (lane == 0) many[atomicAdd(&many_n, 1)] = static_cast<uint32_t>(r);   // (their order does not matter)
      continue;
    }
    if (tokens == 0 && accumulate) continue;
    for (int64_t c0 = 0; c0 < h; c0 += 256) {
      const int64_t col = c0 + lane * 8;
      float a[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      if (tokens > 0) direct_sum(a, list, 0, n, static_cast<uint32_t>(r), dY, lddy, col, h);
      if (col < h) out(r, col, a);
    }
  }
  __syncthreads();
  const int share = (n + kDirectWarps - 1) / kDirectWarps, from = warp * share, to = min(n, from + share);
  for (int i = 0; i < many_n; ++i)
    for (int64_t c0 = 0; c0 < h; c0 += 256) {
      const int64_t col = c0 + lane * 8;
      float a[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      direct_sum(a, list, from, to, many[i], dY, lddy, col, h);
      part[warp][0][lane] = make_float4(a[0], a[1], a[2], a[3]);
      part[warp][1][lane] = make_float4(a[4], a[5], a[6], a[7]);
      __syncthreads();
      if (warp == 0 && col < h) {
#pragma unroll
        for (int w = 1; w < kDirectWarps; ++w) {
          const float4 p = part[w][0][lane], q = part[w][1][lane];
          a[0] += p.x; a[1] += p.y; a[2] += p.z; a[3] += p.w;
          a[4] += q.x; a[5] += q.y; a[6] += q.z; a[7] += q.w;
        }
        out(many[i], col, a);
      }
      __syncthreads();
    }
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

struct SortPlan {
  int64_t nb;        // sort blocks
  int C;             // sorted places per sum chunk
  int64_t chunks;
  size_t keys, counts, part, runs;   // bytes of one key array, of the counts, of one partial array, of the run list
};

// A chunk is 16 places, or longer so that there are at most 2048 of them up to kMaxChunk: with 8192 tokens of 4096
// columns that is 1024 CTAs of two batches of loads.
SortPlan plan_of(int64_t T, int64_t h) {
  SortPlan p;
  p.nb = (T + kSortBlock - 1) / kSortBlock;
  int64_t C = 16;
  while (C < kMaxChunk && (T + C - 1) / C > 2048) C *= 2;
  p.C = static_cast<int>(C);
  p.chunks = (T + C - 1) / C;
  p.keys = round256(static_cast<size_t>(T) * 4);
  p.counts = round256(static_cast<size_t>(kRadix) * p.nb * 4);
  p.part = round256(static_cast<size_t>(p.chunks) * h * 4);
  p.runs = round256(static_cast<size_t>(p.chunks + 2) * 4);
  return p;
}

int check_common(int t, int64_t T, int64_t h, int64_t V, const char* name) {
  if (t < 1 || t > kMaxShards) return set_error(TTL_ERR_ARG, "%s: t=%d outside [1,%d]", name, t, kMaxShards);
  if (T < 0 || h < 0 || V < 0) return set_error(TTL_ERR_ARG, "%s: negative shape", name);
  if (V % t) return set_error(TTL_ERR_SHAPE, "%s: t=%d must divide V=%lld", name, t, (long long)V);
  if (h % 8) return set_error(TTL_ERR_SHAPE, "%s: h must be a multiple of 8", name);
  if (T >= (int64_t(1) << 31) || V >= (int64_t(1) << 31) - 1 || h >= (int64_t(1) << 24))
    return set_error(TTL_ERR_SHAPE, "%s: extent too large", name);
  return TTL_OK;
}

int check_array(const void* const* a, int t, const char* what, const char* name) {
  if (!a) return set_error(TTL_ERR_ARG, "%s: %s: null shard array", name, what);
  for (int i = 0; i < t; ++i) {
    if (!a[i]) return set_error(TTL_ERR_ARG, "%s: %s[%d] is null", name, what, i);
    if (!aligned16(a[i])) return set_error(TTL_ERR_ALIGN, "%s: %s[%d] not 16-byte aligned", name, what, i);
  }
  return TTL_OK;
}

int check_ids(const int64_t* ids, const char* name) {
  if (!ids) return set_error(TTL_ERR_ARG, "%s: ids is null", name);
  if (reinterpret_cast<uintptr_t>(ids) & 7) return set_error(TTL_ERR_ALIGN, "%s: ids not 8-byte aligned", name);
  return TTL_OK;
}

}  // namespace
}  // namespace ttl

using namespace ttl;

extern "C" int ttl_vocab_parallel_embedding_scaled_fwd(int t, int64_t T, int64_t h, int64_t V, const int64_t* ids,
                                                       const ttl_bf16* const* E, float scale, ttl_bf16* const* out,
                                                       void* stream) {
  const char* name = "ttl_vocab_parallel_embedding_scaled_fwd";
  int rc = check_common(t, T, h, V, name);
  if (rc) return rc;
  if (T == 0 || h == 0) return TTL_OK;
  if (V == 0) return set_error(TTL_ERR_SHAPE, "%s: empty vocabulary", name);
  if ((rc = check_ids(ids, name)) || (rc = check_array(reinterpret_cast<const void* const*>(E), t, "E", name)) ||
      (rc = check_array(reinterpret_cast<const void* const*>(out), t, "out", name)))
    return rc;
  {
    bool one = true;   // the shards' outputs hold the same: they may be one buffer
    for (int i = 1; i < t; ++i) one &= out[i] == out[0];
    const void* tok = ids;
    const Operand outs = operand("out", reinterpret_cast<const void* const*>(out), one ? 1 : t, T * h * 2);
    const Operand ins[2] = {operand("E", reinterpret_cast<const void* const*>(E), t, V / t * h * 2),
                            operand("ids", &tok, 1, T * 8)};
    if ((rc = check_alias(&outs, 1, ins, 2, name))) return rc;
  }
  if ((rc = require_sm103())) return rc;
  int* status = device_status_ptr();
  if (!status) return TTL_ERR_CUDA;
  ScaledTables tab = {};
  ScaledOut o = {};
  for (int i = 0; i < t; ++i) {
    tab.e[i] = reinterpret_cast<const uint4*>(E[i]);
    o.o[i] = reinterpret_cast<uint4*>(out[i]);
  }
  const int64_t h8 = h / 8;
  const int threads = h8 >= 256 ? 256 : static_cast<int>((h8 + 31) / 32 * 32);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  TraceScope trace(s, TTL_K_EMBED, 0.0, static_cast<double>(T) * h * 2.0 * (1.0 + t));
  embed_scaled_kernel<<<static_cast<unsigned>(T), threads, 0, s>>>(tab, o, ids, t, h8, V / t, V, scale, status);
  return cuda_check(cudaGetLastError(), "embed_scaled_kernel launch");
}

extern "C" size_t ttl_vocab_parallel_embedding_sorted_bwd_workspace_size(int t, int64_t T, int64_t h, int64_t V) {
  if (check_common(t, T, h, V, "ttl_vocab_parallel_embedding_sorted_bwd_workspace_size")) return 0;
  const SortPlan p = plan_of(T, h);
  return 4 * p.keys + p.counts + 2 * p.part + p.runs;
}

extern "C" int ttl_vocab_parallel_embedding_sorted_bwd(int t, int64_t T, int64_t h, int64_t V, const int64_t* ids,
                                                       const ttl_bf16* dY, int64_t lddy, float scale,
                                                       float* const* dE, int accumulate, void* ws, size_t ws_bytes,
                                                       void* stream) {
  const char* name = "ttl_vocab_parallel_embedding_sorted_bwd";
  int rc = check_common(t, T, h, V, name);
  if (rc) return rc;
  if (accumulate != 0 && accumulate != 1) return set_error(TTL_ERR_ARG, "%s: accumulate must be 0 or 1", name);
  if (h == 0 || V == 0) return T > 0 && V == 0 ? set_error(TTL_ERR_SHAPE, "%s: empty vocabulary", name) : TTL_OK;
  if ((rc = check_array(reinterpret_cast<const void* const*>(dE), t, "dE", name))) return rc;
  const size_t need = ttl_vocab_parallel_embedding_sorted_bwd_workspace_size(t, T, h, V);
  if (T > 0) {
    if ((rc = check_ids(ids, name))) return rc;
    if (!dY) return set_error(TTL_ERR_ARG, "%s: dY is null", name);
    if (lddy < h) return set_error(TTL_ERR_SHAPE, "%s: dY's row stride is smaller than h", name);
    if (!aligned16(dY) || lddy % 8) return set_error(TTL_ERR_ALIGN, "%s: rows of dY not 16-byte aligned", name);
    if (!ws || ws_bytes < need)
      return set_error(TTL_ERR_ARG, "%s: workspace of %zu bytes needed, %zu given", name, need, ws_bytes);
    if (!aligned16(ws)) return set_error(TTL_ERR_ALIGN, "%s: workspace not 16-byte aligned", name);
  } else if (accumulate) {
    return TTL_OK;
  }
  {
    const void *tok = ids, *dy = dY, *space = ws;
    const int given = T > 0 ? 1 : 0;
    const Operand outs[2] = {operand("dE", reinterpret_cast<const void* const*>(dE), t, V / t * h * 4),
                             operand("the workspace", &space, given, static_cast<int64_t>(need))};
    const Operand ins[2] = {operand("dY", &dy, given, T, lddy * 2, h * 2), operand("ids", &tok, given, T * 8)};
    if ((rc = check_alias(outs, 2, ins, 2, name))) return rc;
  }
  if ((rc = require_sm103())) return rc;
  int* status = device_status_ptr();
  if (!status) return TTL_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t Vs = V / t;
  GradTables G = {};
  for (int i = 0; i < t; ++i) G.g[i] = dE[i];
  // one launch for the sort and the zeros, where the tokens fit one CTA and a slice's marks its shared memory
  const int sms = num_sms();
  const bool one = T > 0 && T <= kOneMost && sms > 1 && V / (sms - 1) / 8 + 64 < static_cast<int64_t>(kOneSmem);
  const bool direct = T <= kDirectMost && h <= kDirectWide && V <= kDirectRows && T * h <= kDirectWork;
  if (!accumulate && (T == 0 || !(one || direct))) {
    TraceScope trace(s, TTL_K_OTHER, 0.0, 4.0 * V * h);
    for (int i = 0; i < t; ++i)
      if ((rc = fill_zero(dE[i], static_cast<size_t>(Vs) * h * 4, s))) return rc;
  }
  if (T == 0) return TTL_OK;
  if (direct) {
    TraceScope trace(s, TTL_K_EMBED, 0.0, static_cast<double>(T) * h * 2.0 + (accumulate ? 0.0 : 4.0 * V * h));
    const int64_t most = (V + kDirectThreads / 32 - 1) / (kDirectThreads / 32);   // a row per warp at least
    const unsigned grid = static_cast<unsigned>(most < 2 * sms ? most : 2 * sms);
    embed_direct_kernel<<<grid, kDirectThreads, 0, s>>>(G, ids, static_cast<int>(T), V, Vs, h,
                                                        reinterpret_cast<const __nv_bfloat16*>(dY), lddy, scale,
                                                        accumulate, status);
    return cuda_check(cudaGetLastError(), "embed_direct_kernel launch");
  }

  const SortPlan p = plan_of(T, h);
  char* base = static_cast<char*>(ws);
  uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(base), reinterpret_cast<uint32_t*>(base + p.keys)};
  uint32_t* toks[2] = {reinterpret_cast<uint32_t*>(base + 2 * p.keys), reinterpret_cast<uint32_t*>(base + 3 * p.keys)};
  uint32_t* counts = reinterpret_cast<uint32_t*>(base + 4 * p.keys);
  float* head = reinterpret_cast<float*>(base + 4 * p.keys + p.counts);
  float* tail = reinterpret_cast<float*>(base + 4 * p.keys + p.counts + p.part);
  uint32_t* runs = reinterpret_cast<uint32_t*>(base + 4 * p.keys + p.counts + 2 * p.part);
  int width = 0;   // bits of the largest key, which is V
  while (width < 32 && (V >> width) > 0) ++width;
  const uint32_t* k_in = nullptr;
  const uint32_t* t_in = nullptr;
  if (one) {
    const int passes = (width + 7) / 8, bits = (width + passes - 1) / passes;
    TraceScope trace(s, TTL_K_EMBED, 0.0, 16.0 * T + (accumulate ? 0.0 : 4.0 * V * h));
    if ((rc = allow_smem<sort_fill_kernel>(kOneSmem, "cudaFuncSetAttribute(sort_fill_kernel)"))) return rc;
    sort_fill_kernel<<<accumulate ? 1 : sms, kOneThreads, kOneSmem, s>>>(
        G, ids, static_cast<int>(T), V, Vs, h, passes, bits, keys[0], toks[0], runs, status);
    if ((rc = cuda_check(cudaGetLastError(), "sort_fill_kernel launch"))) return rc;
    k_in = keys[0];
    t_in = toks[0];
  } else {
    TraceScope trace(s, TTL_K_EMBED, 0.0, 16.0 * T);
    int out = 0;
    for (int shift = 0; shift < width; shift += 8) {
      sort_count_kernel<<<static_cast<unsigned>(p.nb), kSortThreads, 0, s>>>(ids, k_in, T, V, shift, counts,
                                                                             static_cast<int>(p.nb), status);
      sort_scan_kernel<<<1, 1024, 0, s>>>(counts, kRadix * p.nb, runs);
      sort_move_kernel<<<static_cast<unsigned>(p.nb), kSortThreads, 0, s>>>(
          ids, k_in, t_in, T, V, shift, counts, static_cast<int>(p.nb), keys[out], toks[out], status);
      k_in = keys[out];
      t_in = toks[out];
      out ^= 1;
    }
    if ((rc = cuda_check(cudaGetLastError(), "token sort launch"))) return rc;
  }
  TraceScope trace(s, TTL_K_EMBED, 0.0, static_cast<double>(T) * h * 2.0);
  const dim3 grid(static_cast<unsigned>(p.chunks), static_cast<unsigned>((h / 8 + kSumThreads - 1) / kSumThreads));
  if ((rc = cuda_check(launch_after(embed_sum_kernel, grid, kSumThreads, 0, s, G, k_in, t_in,
                                    reinterpret_cast<const __nv_bfloat16*>(dY), lddy, T, h, Vs, V, p.C, scale,
                                    accumulate, head, tail, runs),
                       "embed_sum_kernel launch")))
    return rc;
  return cuda_check(launch_after(embed_join_kernel, dim3(static_cast<unsigned>(sms) * 2), kSumThreads, 0, s, G, k_in, T, h,
                                 Vs, p.C, scale, accumulate, static_cast<const float*>(head),
                                 static_cast<const float*>(tail), static_cast<const uint32_t*>(runs),
                                 static_cast<int>(p.chunks)),
                    "embed_join_kernel launch");
}
