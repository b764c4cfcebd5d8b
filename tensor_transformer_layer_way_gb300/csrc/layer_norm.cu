// Layer norm over the token slabs of a sequence-parallel block, forward and backward.
//
// Source: "v4:Tensor Parallel 与 Sequence Parallel", section "SP": between the tensor-parallel
// regions every shard keeps s/t tokens, and LayerNorm and the residual sum run on those slabs.
// The norm's weights are full on every shard, so their gradient is summed over all slabs.
//
// Row s = x (+ r, rounded to the stream's type), over h columns:
//   mean = sum(s) / h,  rstd = 1 / sqrt(sum((s - mean)^2) / h + eps),  xhat = (s - mean) rstd
//   y = xhat gamma + beta
// Backward, with g = dy gamma:
//   dx = rstd (g - sum(g) / h - xhat sum(g xhat) / h) (+ ds, the gradient that passes the block)
//   dgamma = sum over rows of dy xhat,  dbeta = sum over rows of dy
// All statistics and sums are fp32; the variance is taken about the mean (no E[x^2] - mean^2).

#include "launch_after.cuh"
#include "operands.h"
#include "ttl_device.cuh"
#include "ttl_internal.h"

namespace ttl {
namespace {

constexpr int kNormThreads = 512;
constexpr size_t kAnySums = 220000;   // bytes
constexpr int kNormParts = 456;   // partial sums of the weight gradients: at most three per SM of a 152-SM part

struct NormFwd {
  const void* x[kMaxShards];
  const void* r[kMaxShards];
  void* s[kMaxShards];
  void* y[kMaxShards];
  float* mean[kMaxShards];
  float* rstd[kMaxShards];
  const void* gamma;
  const void* beta;
  int64_t rows, h, ldx, ldr;   // rows per slab
  int64_t total;               // t rows
  float eps;
  int wtype;
  int* status;
};

struct NormBwd {
  const void* x[kMaxShards];
  const void* dy[kMaxShards];
  const void* ds[kMaxShards];
  void* dx[kMaxShards];
  const float* mean[kMaxShards];
  const float* rstd[kMaxShards];
  const void* gamma;
  float* part;                 // [grid][2][h]: dgamma then dbeta
  int64_t rows, h, ldx, lddy, ldds;
  int64_t total;
  int wtype;
  int* status;
};

__device__ __forceinline__ float load_w(const void* w, int wtype, int64_t i) {
  return wtype == TTL_T_F32 ? static_cast<const float*>(w)[i]
                            : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the CTA; every thread gets it.  `red` holds one float per warp and is reused by the next
// call only after the barrier at this one's start.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s += red[w];
  return s;
}

// A group's place: row k of slab i, moved on by a fixed number of rows (no division per row).
struct Cursor {
  int i;
  int64_t k;
  __device__ __forceinline__ Cursor(int64_t row, int64_t rows) {
    i = 0;
    k = row;
    fold(rows);
  }
  __device__ __forceinline__ void fold(int64_t rows) {
    while (k >= rows && i < kMaxShards) {   // past the last slab the place is not used
      k -= rows;
      ++i;
    }
  }
  __device__ __forceinline__ void move(int64_t step, int64_t rows) {
    k += step;
    fold(rows);
  }
};

// ------------------------------------------------------------------ rows held in registers
// Short rows (spread_of has the bounds): a row belongs to one warp or two; each thread holds NV words of B bytes of it (16 where every row
// starts on 16 bytes and holds whole words, else 4 or 2), so the row is read once and the weights stay in registers over
// the persistent loop.  The next row's words are loaded before this one's sums.  A CTA of narrow rows has
// several groups of warps, each with rows of its own.  Measured, 65536 rows of 256 bf16: forward 20 us (3.4 TB/s),
// backward 39 us (2.6 TB/s); bound by a row's chain of loads, sums and stores.

template <int B> struct Word;
template <> struct Word<16> { using type = uint4; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<2> { using type = uint16_t; };

template <typename T, int B>
__device__ __forceinline__ void unpack(const typename Word<B>::type& w, float* f) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (B == 16) {
      f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y); f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
    } else {
      f[0] = __uint_as_float(w);
    }
  } else if constexpr (B == 16) {
    f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
    f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
  } else if constexpr (B == 4) {
    f[0] = bf16_lo(w); f[1] = bf16_hi(w);
  } else {
    f[0] = __uint_as_float(static_cast<uint32_t>(w) << 16);
  }
}

template <typename T, int B>
__device__ __forceinline__ typename Word<B>::type pack(const float* f) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (B == 16)
      return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    else
      return __float_as_uint(f[0]);
  } else if constexpr (B == 16) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  } else if constexpr (B == 4) {
    return pack_bf16x2(f[0], f[1]);
  } else {
    return static_cast<uint16_t>(pack_bf16x2(f[0], 0.0f) & 0xffffu);
  }
}

constexpr int kMaxWarps = 16;    // warps per row

// The W warps of a group meet (each group has its own hardware barrier; all its warps take the same rows).
__device__ __forceinline__ void group_sync(int group, int W) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(W * 32) : "memory");
}

template <typename T, int B, int NV>
__global__ void __launch_bounds__(kMaxWarps * 32) norm_fwd_kernel(const __grid_constant__ NormFwd P, int G) {
  using Wd = typename Word<B>::type;
  constexpr int E = B / sizeof(T);
  const int group = threadIdx.x >> 5, v0 = threadIdx.x & 31;
  const int words = static_cast<int>(P.h / E);
  constexpr int vs = 32;                           // this thread's words: v0 + u vs
  float ga[NV * E], be[NV * E];
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool in = v0 + u * vs < words;
      const int64_t c = static_cast<int64_t>(v0 + u * vs) * E + e;
      ga[u * E + e] = in ? load_w(P.gamma, P.wtype, c) : 0.0f;
      be[u * E + e] = in && P.beta ? load_w(P.beta, P.wtype, c) : 0.0f;
    }
  const float inv_h = 1.0f / static_cast<float>(P.h);
  Wd xw[NV], rw[NV];
  auto fetch = [&](const Cursor& at) {
    const int i = at.i;
    const int64_t k = at.k;
    const Wd* x = reinterpret_cast<const Wd*>(static_cast<const T*>(P.x[i]) + k * P.ldx);
    const Wd* r = P.r[i] ? reinterpret_cast<const Wd*>(static_cast<const T*>(P.r[i]) + k * P.ldr) : nullptr;
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (v0 + u * vs < words) {
        xw[u] = __ldcs(x + v0 + u * vs);
        if (r) rw[u] = __ldcs(r + v0 + u * vs);
      }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  int64_t row = static_cast<int64_t>(blockIdx.x) * G + group;
  Cursor ahead(row, P.rows);
  if (row < P.total) fetch(ahead);
  for (; row < P.total; row += step) {
    const int i = ahead.i;
    const int64_t k = ahead.k;
    ahead.move(step, P.rows);
    const bool res = P.r[i] != nullptr;
    float x[NV * E];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const bool in = v0 + u * vs < words;
      if (in) {
        unpack<T, B>(xw[u], x + u * E);
        if (res) {
          float r[E];
          unpack<T, B>(rw[u], r);
#pragma unroll
          for (int e = 0; e < E; ++e) x[u * E + e] += r[e];
          const Wd w = pack<T, B>(x + u * E);      // the stream's type: what is normalised is what is kept
          unpack<T, B>(w, x + u * E);
          __stcs(reinterpret_cast<Wd*>(static_cast<T*>(P.s[i]) + k * P.h) + v0 + u * vs, w);
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) x[u * E + e] = 0.0f;
      }
    }
    if (row + step < P.total) fetch(ahead);
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < NV * E; ++e) sum += x[e];
    sum = warp_sum(sum);
    const float mean = sum / static_cast<float>(P.h);   // divided, so that a row of one value has exactly that mean
    float sq = 0.0f;
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (v0 + u * vs < words) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float d = x[u * E + e] - mean;
          sq = fmaf(d, d, sq);
        }
      }
    sq = warp_sum(sq);
    const float rstd = rsqrtf(fmaf(sq, inv_h, P.eps));
    Wd* y = reinterpret_cast<Wd*>(static_cast<T*>(P.y[i]) + k * P.h);
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (v0 + u * vs < words) {
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf((x[u * E + e] - mean) * rstd, ga[u * E + e], be[u * E + e]);
        __stcs(y + v0 + u * vs, pack<T, B>(o));
      }
    if (v0 == 0) {
      P.mean[i][k] = mean;
      P.rstd[i][k] = rstd;
    }
  }
}

// The backward pass: each thread also keeps its columns' sums of dgamma and dbeta over the CTA's rows;
// the groups of a CTA join theirs in shared memory, the CTAs in norm_join_kernel.
template <typename T, int B, int NV>
__global__ void __launch_bounds__(kMaxWarps * 32) norm_bwd_kernel(const __grid_constant__ NormBwd P, int W, int G) {
  using Wd = typename Word<B>::type;
  constexpr int E = B / sizeof(T);
  __shared__ float2 red[2][kMaxWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / W, gw = warp % W;
  const int words = static_cast<int>(P.h / E);
  const int v0 = gw * 32 + lane, vs = W * 32;
  float ga[NV * E], dg[NV * E], db[NV * E];
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool in = v0 + u * vs < words;
      ga[u * E + e] = in ? load_w(P.gamma, P.wtype, static_cast<int64_t>(v0 + u * vs) * E + e) : 0.0f;
      dg[u * E + e] = db[u * E + e] = 0.0f;
    }
  const float inv_h = 1.0f / static_cast<float>(P.h);
  Wd xw[NV], dw[NV];
  float mean = 0.0f, rstd = 0.0f;
  auto fetch = [&](const Cursor& at) {
    const int i = at.i;
    const int64_t k = at.k;
    const Wd* x = reinterpret_cast<const Wd*>(static_cast<const T*>(P.x[i]) + k * P.ldx);
    const Wd* d = reinterpret_cast<const Wd*>(static_cast<const T*>(P.dy[i]) + k * P.lddy);
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (v0 + u * vs < words) {
        xw[u] = __ldcs(x + v0 + u * vs);
        dw[u] = __ldcs(d + v0 + u * vs);
      }
    mean = __ldg(P.mean[i] + k);
    rstd = __ldg(P.rstd[i] + k);
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  int64_t row = static_cast<int64_t>(blockIdx.x) * G + group;
  Cursor ahead(row, P.rows);
  if (row < P.total) fetch(ahead);
  for (int it = 0; row < P.total; row += step, it ^= 1) {
    const int i = ahead.i;
    const int64_t k = ahead.k;
    ahead.move(step, P.rows);
    const bool more = P.ds[i] != nullptr;
    const Wd* ds = more ? reinterpret_cast<const Wd*>(static_cast<const T*>(P.ds[i]) + k * P.ldds) : nullptr;
    Wd sw[NV];
    if (more) {
#pragma unroll
      for (int u = 0; u < NV; ++u)
        if (v0 + u * vs < words) sw[u] = __ldcs(ds + v0 + u * vs);
    }
    float xh[NV * E], g[NV * E];
    float s1 = 0.0f, s2 = 0.0f;
    const float rs = rstd;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (v0 + u * vs < words) {
        float d[E];
        unpack<T, B>(xw[u], xh + u * E);
        unpack<T, B>(dw[u], d);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int c = u * E + e;
          xh[c] = (xh[c] - mean) * rs;
          dg[c] = fmaf(d[e], xh[c], dg[c]);
          db[c] += d[e];
          g[c] = d[e] * ga[c];
          s1 += g[c];
          s2 = fmaf(g[c], xh[c], s2);
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) xh[u * E + e] = g[u * E + e] = 0.0f;
      }
    }
    if (row + step < P.total) fetch(ahead);
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (W > 1) {
      if (lane == 0) red[it][warp] = make_float2(s1, s2);
      group_sync(group, W);
      s1 = s2 = 0.0f;
      for (int w = 0; w < W; ++w) {
        const float2 o = red[it][group * W + w];
        s1 += o.x;
        s2 += o.y;
      }
    }
    const float c1 = s1 * inv_h, c2 = s2 * inv_h;
    Wd* dx = reinterpret_cast<Wd*>(static_cast<T*>(P.dx[i]) + k * P.h);
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (v0 + u * vs < words) {
        float o[E], d[E];
        if (more) unpack<T, B>(sw[u], d);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int c = u * E + e;
          o[e] = rs * (g[c] - c1 - xh[c] * c2);
          if (more) o[e] += d[e];
        }
        __stcs(dx + v0 + u * vs, pack<T, B>(o));
      }
  }
  // ---- the CTA's partial sums: group 0 first, the others added in order
  extern __shared__ float sums[];                      // [2][h], only with several groups
  float* pg = G > 1 ? sums : P.part + static_cast<int64_t>(blockIdx.x) * 2 * P.h;
  for (int q = 0; q < G; ++q) {
    if (q == group) {
#pragma unroll
      for (int u = 0; u < NV; ++u)
        if (v0 + u * vs < words) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int64_t c = static_cast<int64_t>(v0 + u * vs) * E + e;
            pg[c] = q ? pg[c] + dg[u * E + e] : dg[u * E + e];
            pg[P.h + c] = q ? pg[P.h + c] + db[u * E + e] : db[u * E + e];
          }
        }
    }
    if (G > 1) __syncthreads();
  }
  if (G > 1) {
    float* out = P.part + static_cast<int64_t>(blockIdx.x) * 2 * P.h;
    for (int64_t c = threadIdx.x; c < 2 * P.h; c += blockDim.x) out[c] = sums[c];
  }
}

// ------------------------------------------------------------------ rows through shared memory
// Longer rows: a ring of whole rows in shared memory, filled by bulk copies that run several rows ahead,
// so the bytes in flight do not depend on how many registers the sums take.  A bulk copy moves whole 16-byte
// pieces, so a row that does not start on one is copied with its neighbours' bytes (they belong to the same
// slab; at the slab's own ends the copy is cut and the few elements outside it are stored beside it by hand), and
// its words are read from shared memory at the row's own offset.
// Measured, 8192 rows of 4096: fp32 forward 44 us (6.1 TB/s, 90% of the copy rate), backward 71 us (83%); bf16
// with a residual 50 us (5.3 TB/s, 79%) and 61 us (4.4 TB/s, 65%), 7 of them the join of the weight gradients.
// Rows of 4001 bf16, whose words are single values: 81 and 95 us.

constexpr int kMaxStages = 6;
constexpr uint64_t kNormTimeout = 2000000000ull;

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// One input's row in shared memory.
struct RowSpan {
  const uint8_t* row;        // global address of the row
  int skip;                  // bytes from the row's 16-byte piece to its start
  int lo, hi;                // bytes of the row that the copy brings: [lo, hi)
};

// Row k of a slab of `rows` rows of row_bytes bytes every ld_bytes.
template <int B>
__device__ __forceinline__ RowSpan span_of(const void* slab, int64_t rows, int64_t ld_bytes, int row_bytes, int64_t k) {
  RowSpan s;
  const uint8_t* base = static_cast<const uint8_t*>(slab);
  s.row = base + k * ld_bytes;
  s.skip = B == 16 ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(s.row) & 15);
  s.lo = 0;
  s.hi = row_bytes;
  if constexpr (B != 16) {
    if (s.skip && k * ld_bytes < s.skip) s.lo = 16 - s.skip;              // the piece would begin before the slab
    const int over = (s.skip + row_bytes) & 15;
    if (over && (rows - 1 - k) * ld_bytes < 16 - over) s.hi = row_bytes - over;   // or end after it
  }
  return s;
}

// The whole pieces that hold bytes [lo, hi) of the row, to the place that its first piece has at dst.
template <int B>
__device__ __forceinline__ uint32_t span_bytes(const RowSpan& s) {
  if constexpr (B == 16) return static_cast<uint32_t>(s.hi);
  const int from = s.lo ? s.skip + s.lo : 0, to = (s.skip + s.hi + 15) & ~15;
  return static_cast<uint32_t>(to - from);
}
template <int B>
__device__ __forceinline__ void span_load(const RowSpan& s, uint8_t* dst, uint64_t* bar) {
  const int from = B != 16 && s.lo ? s.skip + s.lo : 0;
  bulk_load(dst + from, s.row - s.skip + from, span_bytes<B>(s), bar);
}
// Bytes that an input's row takes in a stage.
template <int B>
__host__ __device__ __forceinline__ uint32_t span_room(int64_t row_bytes) {
  return static_cast<uint32_t>(B == 16 ? row_bytes : (row_bytes + 15 + 15) / 16 * 16);
}

// Whether the copy left bytes of the row out, and those bytes by hand (fewer than 16 at either end, by one warp).
template <int B>
__device__ __forceinline__ bool span_cut(const RowSpan& s, int row_bytes) {
  return B != 16 && (s.lo > 0 || s.hi < row_bytes);
}
template <int B>
__device__ __forceinline__ void span_mend(const RowSpan& s, uint8_t* at, int row_bytes) {
  using Wd = typename Word<B>::type;
  const int lane = threadIdx.x & 31;
  const int c = lane < 16 ? lane * B : s.hi + (lane - 16) * B;
  if (lane < 16 ? c < s.lo : c < row_bytes)
    *reinterpret_cast<Wd*>(at + s.skip + c) = *reinterpret_cast<const Wd*>(s.row + c);
  fence_proxy_async_smem();   // a later copy writes the same bytes
}

// Word v of the row.
template <int B>
__device__ __forceinline__ typename Word<B>::type span_word(const RowSpan& s, const uint8_t* at, int v) {
  return *reinterpret_cast<const typename Word<B>::type*>(at + s.skip + v * B);
}

// The arithmetic runs on pairs of values (two fp32 operations per instruction): neither issue (45 to 52%) nor DRAM (53 to
// 54%) is full, and fewer instructions shorten the chain of loads, sums, exchange and stores that a row is.  A value
// past the row's end is 0.

template <typename T, int B, int NV>
__global__ void __launch_bounds__(kMaxWarps * 32) norm_fwd_ring_kernel(const __grid_constant__ NormFwd P, int W, int G,
                                                                       int stages) {
  using Wd = typename Word<B>::type;
  constexpr int E = B / sizeof(T);
  extern __shared__ __align__(16) uint8_t ring[];     // [G][stages][x, r]
  __shared__ float2 red[2][kMaxWarps];
  __shared__ float own_mean[2][kMaxWarps];
  __shared__ float count[kMaxWarps];
  __shared__ uint64_t full[8][kMaxStages];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / W, gw = warp % W;
  const int words = static_cast<int>(P.h / E), row_bytes = words * B;
  const int v0 = gw * 32 + lane, vs = W * 32;
  const bool res = P.r[0] != nullptr;
  const int64_t ldx = P.ldx * static_cast<int64_t>(sizeof(T)), ldr = P.ldr * static_cast<int64_t>(sizeof(T));
  const uint32_t room = span_room<B>(row_bytes), stage_bytes = room * (res ? 2 : 1);
  uint8_t* mine = ring + static_cast<size_t>(group) * stages * stage_bytes;
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * G + group;
  volatile int* ab = &abort_flag;
  Cursor ahead(first, P.rows);      // the next row to be copied (used by the group's first thread)
  auto start = [&](int st) {
    const RowSpan sx = span_of<B>(P.x[ahead.i], P.rows, ldx, row_bytes, ahead.k);
    uint32_t bytes = span_bytes<B>(sx);
    if (res) {
      const RowSpan sr = span_of<B>(P.r[ahead.i], P.rows, ldr, row_bytes, ahead.k);
      mbar_arrive_expect_tx(&full[group][st], bytes + span_bytes<B>(sr));
      span_load<B>(sr, mine + st * stage_bytes + room, &full[group][st]);
    } else {
      mbar_arrive_expect_tx(&full[group][st], bytes);
    }
    span_load<B>(sx, mine + st * stage_bytes, &full[group][st]);
    ahead.move(step, P.rows);
  };
  if (gw == 0 && lane == 0) {
    for (int st = 0; st < stages; ++st) mbar_init(&full[group][st], 1);
    if (group == 0) abort_flag = 0;
    fence_mbarrier_init();
  }
  __syncthreads();
  if (gw == 0 && lane == 0)
    for (int st = 0; st < stages; ++st)
      if (first + st * step < P.total) start(st);
  float ga[NV * E], be[NV * E];
  float n_mine = 0.0f;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int left = words - (gw * 32 + u * vs);
    n_mine += static_cast<float>(left <= 0 ? 0 : (left < 32 ? left : 32) * E);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool in = v0 + u * vs < words;
      const int64_t c = static_cast<int64_t>(v0 + u * vs) * E + e;
      ga[u * E + e] = in ? load_w(P.gamma, P.wtype, c) : 0.0f;
      be[u * E + e] = in && P.beta ? load_w(P.beta, P.wtype, c) : 0.0f;
    }
  }
  if (lane == 0) count[warp] = n_mine;
  __syncthreads();
  const float hf = static_cast<float>(P.h), inv_h = 1.0f / hf;
  int st = 0, it = 0;
  uint32_t ph = 0;
  Cursor at(first, P.rows);
  for (int64_t row = first; row < P.total; row += step, it ^= 1, at.move(step, P.rows)) {
    const int i = at.i;
    const int64_t k = at.k;
    const RowSpan sx = span_of<B>(P.x[i], P.rows, ldx, row_bytes, k);
    const RowSpan sr = span_of<B>(res ? P.r[i] : P.x[i], P.rows, res ? ldr : ldx, row_bytes, k);
    // (a wait that runs out is in the status word; the group goes on, so that all its warps keep meeting)
    mbar_wait(&full[group][st], ph, ab, P.status, kNormTimeout);
    uint8_t* px = mine + st * stage_bytes;
    if (span_cut<B>(sx, row_bytes) || span_cut<B>(sr, row_bytes)) {
      if (gw == 0) {
        span_mend<B>(sx, px, row_bytes);
        if (res) span_mend<B>(sr, px + room, row_bytes);
      }
      if (W > 1) group_sync(group, W); else __syncwarp();
    }
    constexpr int N = NV * E;
    float x[N];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (v0 + u * vs < words) {
        unpack<T, B>(span_word<B>(sx, px, v0 + u * vs), x + u * E);
        if (res) {
          float r[E];
          unpack<T, B>(span_word<B>(sr, px + room, v0 + u * vs), r);
#pragma unroll
          for (int e = 0; e < E; ++e) x[u * E + e] += r[e];
          const Wd w = pack<T, B>(x + u * E);          // the stream's type: what is normalised is what is kept
          unpack<T, B>(w, x + u * E);
          __stcs(reinterpret_cast<Wd*>(static_cast<T*>(P.s[i]) + k * P.h) + v0 + u * vs, w);
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) x[u * E + e] = 0.0f;
      }
    }
    uint64_t acc0 = f2_pack(x[0], x[1]), acc1 = f2_pack(x[2], x[3]);
#pragma unroll
    for (int c = 4; c < N; c += 4) {
      acc0 = fadd2(acc0, f2_pack(x[c], x[c + 1]));
      acc1 = fadd2(acc1, f2_pack(x[c + 2], x[c + 3]));
    }
    const float2 pair = f2_unpack(fadd2(acc0, acc1));
    const float sum = warp_sum(pair.x + pair.y);
    // The warp's own mean and the squares about it; the warps are joined with the exact shift
    // sum (s - mean)^2 = sum (s - mean_w)^2 + n_w (mean_w - mean)^2, so one exchange is enough.
    float mean = n_mine > 0.0f ? sum / n_mine : 0.0f;
    acc0 = acc1 = 0;
    const uint64_t nm2 = f2_pack(-mean, -mean);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      // (a value past the end takes no part)
      const bool in0 = v0 + (c / E) * vs < words, in1 = v0 + ((c + 1) / E) * vs < words;
      uint64_t d = fadd2(f2_pack(x[c], x[c + 1]), nm2);
      if (!in0 || !in1) {
        const float2 f = f2_unpack(d);
        d = f2_pack(in0 ? f.x : 0.0f, in1 ? f.y : 0.0f);
      }
      if (c & 2) acc1 = ffma2(d, d, acc1);
      else acc0 = ffma2(d, d, acc0);
    }
    const float2 sqp = f2_unpack(fadd2(acc0, acc1));
    float sq = sqp.x + sqp.y;
    sq = warp_sum(sq);
    if (W > 1) {
      if (lane == 0) {
        red[it][warp] = make_float2(sum, sq);
        own_mean[it][warp] = mean;
      }
      group_sync(group, W);
      // lane w takes warp w's, the lanes join by shuffles
      const bool has = lane < W;
      const float2 o = has ? red[it][group * W + lane] : make_float2(0.0f, 0.0f);
      const float n = has ? count[group * W + lane] : 0.0f, mw = has ? own_mean[it][group * W + lane] : 0.0f;
      float tot = o.x;
#pragma unroll
      for (int q = kMaxWarps / 2; q > 0; q >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, q);
      mean = __shfl_sync(0xffffffffu, tot, 0) / hf;   // divided: a row of one value has exactly that mean
      const float d = mw - mean;
      sq = fmaf(n * d, d, o.y);
#pragma unroll
      for (int q = kMaxWarps / 2; q > 0; q >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, q);
      sq = __shfl_sync(0xffffffffu, sq, 0);
    } else {
      __syncwarp();
    }
    // every thread of the group holds its words: the buffer is free
    if (gw == 0 && lane == 0 && row + stages * step < P.total) start(st);
    if (++st == stages) {
      st = 0;
      ph ^= 1;
    }
    const float rstd = rsqrtf(fmaf(sq, inv_h, P.eps));
    Wd* y = reinterpret_cast<Wd*>(static_cast<T*>(P.y[i]) + k * P.h);
    const uint64_t m2 = f2_pack(-mean, -mean), r2 = f2_pack(rstd, rstd);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const float2 f = f2_unpack(ffma2(fmul2(fadd2(f2_pack(x[c], x[c + 1]), m2), r2), f2_pack(ga[c], ga[c + 1]),
                                       f2_pack(be[c], be[c + 1])));
      x[c] = f.x;
      x[c + 1] = f.y;
    }
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (v0 + u * vs < words) __stcs(y + v0 + u * vs, pack<T, B>(x + u * E));
    if (gw == 0 && lane == 0) {
      P.mean[i][k] = mean;
      P.rstd[i][k] = rstd;
    }
  }
}

// The backward pass.  Up to 16 values a thread, xhat and g stay in registers between the sums and dx (KEEP) and the
// row's buffer is free with the sums' exchange; with more, the words are read again, and the buffer is free once
// the group has met over the next row's sums.
template <typename T, int B, int NV>
__global__ void __launch_bounds__(kMaxWarps * 32) norm_bwd_ring_kernel(const __grid_constant__ NormBwd P, int W, int G,
                                                                       int stages) {
  constexpr bool KEEP = NV * B / sizeof(T) <= 16;
  using Wd = typename Word<B>::type;
  constexpr int E = B / sizeof(T);
  extern __shared__ __align__(16) uint8_t ring[];     // [G][stages][x, dy, ds], and then [2][h] sums
  __shared__ float2 red[2][kMaxWarps];
  __shared__ uint64_t full[8][kMaxStages];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / W, gw = warp % W;
  const int words = static_cast<int>(P.h / E), row_bytes = words * B;
  const int v0 = gw * 32 + lane, vs = W * 32;
  const bool more = P.ds[0] != nullptr;
  const int64_t ldx = P.ldx * static_cast<int64_t>(sizeof(T)), ldd = P.lddy * static_cast<int64_t>(sizeof(T)),
                lds = P.ldds * static_cast<int64_t>(sizeof(T));
  const uint32_t room = span_room<B>(row_bytes), stage_bytes = room * (more ? 3 : 2);
  uint8_t* mine = ring + static_cast<size_t>(group) * stages * stage_bytes;
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * G + group;
  volatile int* ab = &abort_flag;
  Cursor ahead(first, P.rows);      // the next row to be copied (used by the group's first thread)
  int64_t ahead_row = first;
  auto start = [&](int st) {
    if (ahead_row < P.total) {
      uint8_t* dst = mine + st * stage_bytes;
      uint64_t* bar = &full[group][st];
      const RowSpan sx = span_of<B>(P.x[ahead.i], P.rows, ldx, row_bytes, ahead.k);
      const RowSpan sd = span_of<B>(P.dy[ahead.i], P.rows, ldd, row_bytes, ahead.k);
      const uint32_t bytes = span_bytes<B>(sx) + span_bytes<B>(sd);
      if (more) {
        const RowSpan ss = span_of<B>(P.ds[ahead.i], P.rows, lds, row_bytes, ahead.k);
        mbar_arrive_expect_tx(bar, bytes + span_bytes<B>(ss));
        span_load<B>(ss, dst + 2 * room, bar);
      } else {
        mbar_arrive_expect_tx(bar, bytes);
      }
      span_load<B>(sx, dst, bar);
      span_load<B>(sd, dst + room, bar);
      ahead.move(step, P.rows);
    }
    ahead_row += step;
  };
  if (gw == 0 && lane == 0) {
    for (int st = 0; st < stages; ++st) mbar_init(&full[group][st], 1);
    if (group == 0) abort_flag = 0;
    fence_mbarrier_init();
  }
  __syncthreads();
  if (gw == 0 && lane == 0)
    for (int st = 0; st < stages; ++st) start(st);
  float ga[NV * E], dg[NV * E], db[NV * E];
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool in = v0 + u * vs < words;
      ga[u * E + e] = in ? load_w(P.gamma, P.wtype, static_cast<int64_t>(v0 + u * vs) * E + e) : 0.0f;
      dg[u * E + e] = db[u * E + e] = 0.0f;
    }
  const float inv_h = 1.0f / static_cast<float>(P.h);
  int st = 0, it = 0;
  uint32_t ph = 0;
  Cursor at(first, P.rows);
  float next_mean = 0.0f, next_rstd = 0.0f;   // of the coming row: loaded a row early
  if (first < P.total) {
    next_mean = __ldg(P.mean[at.i] + at.k);
    next_rstd = __ldg(P.rstd[at.i] + at.k);
  }
  for (int64_t row = first; row < P.total; row += step, it ^= 1) {
    const int i = at.i;
    const int64_t k = at.k;
    const float mean = next_mean, rs = next_rstd;
    at.move(step, P.rows);
    if (row + step < P.total) {
      next_mean = __ldg(P.mean[at.i] + at.k);
      next_rstd = __ldg(P.rstd[at.i] + at.k);
    }
    const RowSpan sx = span_of<B>(P.x[i], P.rows, ldx, row_bytes, k);
    const RowSpan sd = span_of<B>(P.dy[i], P.rows, ldd, row_bytes, k);
    mbar_wait(&full[group][st], ph, ab, P.status, kNormTimeout);
    uint8_t* px = mine + st * stage_bytes;
    const RowSpan ss = span_of<B>(more ? P.ds[i] : P.x[i], P.rows, more ? lds : ldx, row_bytes, k);
    if (span_cut<B>(sx, row_bytes) || span_cut<B>(sd, row_bytes) || span_cut<B>(ss, row_bytes)) {
      if (gw == 0) {
        span_mend<B>(sx, px, row_bytes);
        span_mend<B>(sd, px + room, row_bytes);
        if (more) span_mend<B>(ss, px + 2 * room, row_bytes);
      }
      if (W > 1) group_sync(group, W); else __syncwarp();
    }
    constexpr int N = NV * E;
    // xhat = (x - mean) rstd, the difference first: it is exact near the mean, where x rstd - round(mean rstd) leaves half
    // a step of the product in every xhat of the row (a row of one value has xhat 0).  g = dy gamma, 0 past the row's end.
    const uint64_t rs2 = f2_pack(rs, rs), nm2 = f2_pack(-mean, -mean);
    float n[KEEP ? N : 2], q[KEEP ? N : 2];
    // xhat and g of word u of this thread; E is 1 only where words are read in pairs
    constexpr int U = E == 1 ? 2 : 1;            // words taken together
    auto read = [&](int u, float (&nn)[U * E], float (&qq)[U * E], bool sums_too, uint64_t& a1, uint64_t& a2) {
#pragma unroll
      for (int w = 0; w < U; ++w) {
        if (v0 + (u + w) * vs < words) {
          unpack<T, B>(span_word<B>(sx, px, v0 + (u + w) * vs), nn + w * E);
          unpack<T, B>(span_word<B>(sd, px + room, v0 + (u + w) * vs), qq + w * E);
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) nn[w * E + e] = qq[w * E + e] = 0.0f;
        }
      }
#pragma unroll
      for (int e = 0; e < U * E; e += 2) {
        const int c = u * E + e;
        const uint64_t d2 = f2_pack(qq[e], qq[e + 1]), n2 = fmul2(fadd2(f2_pack(nn[e], nn[e + 1]), nm2), rs2);
        const uint64_t g2 = fmul2(d2, f2_pack(ga[c], ga[c + 1]));
        if (sums_too) {
          const float2 fg = f2_unpack(ffma2(d2, n2, f2_pack(dg[c], dg[c + 1])));
          const float2 fb = f2_unpack(fadd2(d2, f2_pack(db[c], db[c + 1])));
          dg[c] = fg.x;
          dg[c + 1] = fg.y;
          db[c] = fb.x;
          db[c + 1] = fb.y;
          a1 = fadd2(a1, g2);
          a2 = ffma2(g2, n2, a2);
        }
        const float2 fn = f2_unpack(n2), fq = f2_unpack(g2);
        nn[e] = fn.x;
        nn[e + 1] = fn.y;
        qq[e] = fq.x;
        qq[e + 1] = fq.y;
      }
    };
    uint64_t a1 = 0, a2 = 0;
#pragma unroll
    for (int u = 0; u < NV; u += U) {
      float nn[U * E], qq[U * E];
      read(u, nn, qq, true, a1, a2);
      if constexpr (KEEP) {
#pragma unroll
        for (int e = 0; e < U * E; ++e) {
          n[u * E + e] = nn[e];
          q[u * E + e] = qq[e];
        }
      }
    }
    Wd sw[KEEP ? NV : 1];
    if (KEEP && more) {
#pragma unroll
      for (int u = 0; u < NV; ++u)
        if (v0 + u * vs < words) sw[KEEP ? u : 0] = span_word<B>(ss, px + 2 * room, v0 + u * vs);
    }
    const float2 f1 = f2_unpack(a1), f2 = f2_unpack(a2);
    float s1 = warp_sum(f1.x + f1.y), s2 = warp_sum(f2.x + f2.y);
    if (W > 1) {
      if (lane == 0) red[it][warp] = make_float2(s1, s2);
      group_sync(group, W);
      const float2 o = lane < W ? red[it][group * W + lane] : make_float2(0.0f, 0.0f);
      s1 = o.x;
      s2 = o.y;
#pragma unroll
      for (int q = kMaxWarps / 2; q > 0; q >>= 1) {
        s1 += __shfl_xor_sync(0xffffffffu, s1, q);
        s2 += __shfl_xor_sync(0xffffffffu, s2, q);
      }
      s1 = __shfl_sync(0xffffffffu, s1, 0);
      s2 = __shfl_sync(0xffffffffu, s2, 0);
    } else {
      __syncwarp();
    }
    // the group is done with this row's buffer (or, without KEEP, with the one before): it is filled again
    if (gw == 0 && lane == 0 && (KEEP || row > first)) start(KEEP ? st : (st == 0 ? stages - 1 : st - 1));
    const float c1 = s1 * inv_h, c2 = s2 * inv_h;
    Wd* dx = reinterpret_cast<Wd*>(static_cast<T*>(P.dx[i]) + k * P.h);
    const uint64_t k1 = f2_pack(-rs * c1, -rs * c1), k2 = f2_pack(-rs * c2, -rs * c2);
#pragma unroll
    for (int u = 0; u < NV; u += U) {
      float nn[U * E], qq[U * E];
      if constexpr (KEEP) {
#pragma unroll
        for (int e = 0; e < U * E; ++e) {
          nn[e] = n[u * E + e];
          qq[e] = q[u * E + e];
        }
      } else {
        read(u, nn, qq, false, a1, a2);
      }
#pragma unroll
      for (int e = 0; e < U * E; e += 2) {
        const float2 f = f2_unpack(ffma2(f2_pack(nn[e], nn[e + 1]), k2, ffma2(f2_pack(qq[e], qq[e + 1]), rs2, k1)));
        qq[e] = f.x;
        qq[e + 1] = f.y;
      }
#pragma unroll
      for (int w = 0; w < U; ++w)
        if (v0 + (u + w) * vs < words) {
          if (more) {
            float d[E];
            unpack<T, B>(KEEP ? sw[KEEP ? u + w : 0] : span_word<B>(ss, px + 2 * room, v0 + (u + w) * vs), d);
#pragma unroll
            for (int e = 0; e < E; ++e) qq[w * E + e] += d[e];
          }
          __stcs(dx + v0 + (u + w) * vs, pack<T, B>(qq + w * E));
        }
    }
    if (++st == stages) {
      st = 0;
      ph ^= 1;
    }
  }
  // ---- the CTA's partial sums: group 0 first, the others added in order
  float* sums = reinterpret_cast<float*>(ring + static_cast<size_t>(G) * stages * stage_bytes);
  float* pg = G > 1 ? sums : P.part + static_cast<int64_t>(blockIdx.x) * 2 * P.h;
  for (int q = 0; q < G; ++q) {
    if (q == group) {
#pragma unroll
      for (int u = 0; u < NV; ++u)
        if (v0 + u * vs < words) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int64_t c = static_cast<int64_t>(v0 + u * vs) * E + e;
            pg[c] = q ? pg[c] + dg[u * E + e] : dg[u * E + e];
            pg[P.h + c] = q ? pg[P.h + c] + db[u * E + e] : db[u * E + e];
          }
        }
    }
    if (G > 1) __syncthreads();
  }
  if (G > 1) {
    float* out = P.part + static_cast<int64_t>(blockIdx.x) * 2 * P.h;
    for (int64_t c = threadIdx.x; c < 2 * P.h; c += blockDim.x) out[c] = sums[c];
  }
}

// ------------------------------------------------------------------ rows of any width

// E weights from column c on (a multiple of E), in wide loads where they start on 16 bytes.
template <int E>
__device__ __forceinline__ void load_weights(const void* w, int wtype, int64_t c, float (&f)[E]) {
  const bool wide = (reinterpret_cast<uintptr_t>(w) & 15) == 0;
  if constexpr (E >= 4) {
    if (wide && wtype == TTL_T_F32) {
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + c + e);
        f[e] = v.x; f[e + 1] = v.y; f[e + 2] = v.z; f[e + 3] = v.w;
      }
      return;
    }
    if (wide) {
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + c + e);
        f[e] = bf16_lo(v.x); f[e + 1] = bf16_hi(v.x); f[e + 2] = bf16_lo(v.y); f[e + 3] = bf16_hi(v.y);
      }
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) f[e] = load_w(w, wtype, c + e);
}

// One row per CTA at a time, any width, stride and alignment; the row is read again for each step (from L1 / L2), by
// words of 16 bytes where every row is made of them, else value by value.  Measured, 2048 rows of 20000 bf16: forward
// 52 us (3.2 TB/s), backward 132 us (1.9 TB/s; 241 with its sums value by value); 2730 rows of 12288 fp32 with ds,
// too wide for the ring's three rows: 129 us (4.2 TB/s), of 12287: 277.
template <typename T, int B>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_any_kernel(const __grid_constant__ NormFwd P) {
  using Wd = typename Word<B>::type;
  constexpr int E = B / sizeof(T);
  __shared__ float red[kNormThreads / 32];
  const int64_t words = P.h / E;
  for (int64_t row = blockIdx.x; row < P.total; row += gridDim.x) {
    const int i = static_cast<int>(row / P.rows);
    const int64_t k = row - i * P.rows;
    const Wd* x = reinterpret_cast<const Wd*>(static_cast<const T*>(P.x[i]) + k * P.ldx);
    const Wd* r = P.r[i] ? reinterpret_cast<const Wd*>(static_cast<const T*>(P.r[i]) + k * P.ldr) : nullptr;
    Wd* s = r ? reinterpret_cast<Wd*>(static_cast<T*>(P.s[i]) + k * P.h) : nullptr;
    Wd* y = reinterpret_cast<Wd*>(static_cast<T*>(P.y[i]) + k * P.h);
    float sum = 0.0f;
#pragma unroll 4
    for (int64_t v = threadIdx.x; v < words; v += kNormThreads) {
      float f[E];
      unpack<T, B>(x[v], f);
      if (r) {
        float g[E];
        unpack<T, B>(r[v], g);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] += g[e];
        const Wd w = pack<T, B>(f);                        // the stream's type: what is normalised is what is kept
        unpack<T, B>(w, f);
        s[v] = w;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) sum += f[e];
    }
    const Wd* in = r ? s : x;                              // (each thread reads the words that it wrote)
    const float mean = block_sum(sum, red) / static_cast<float>(P.h);
    float sq = 0.0f;
#pragma unroll 4
    for (int64_t v = threadIdx.x; v < words; v += kNormThreads) {
      float f[E];
      unpack<T, B>(in[v], f);
#pragma unroll
      for (int e = 0; e < E; ++e) sq = fmaf(f[e] - mean, f[e] - mean, sq);
    }
    const float rstd = 1.0f / sqrtf(block_sum(sq, red) / static_cast<float>(P.h) + P.eps);
#pragma unroll 2
    for (int64_t v = threadIdx.x; v < words; v += kNormThreads) {
      float f[E];
      unpack<T, B>(in[v], f);
      float ga[E], be[E];
      load_weights<E>(P.gamma, P.wtype, v * E, ga);
#pragma unroll
      for (int e = 0; e < E; ++e) be[e] = 0.0f;
      if (P.beta) load_weights<E>(P.beta, P.wtype, v * E, be);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = fmaf((f[e] - mean) * rstd, ga[e], be[e]);
      y[v] = pack<T, B>(f);
    }
    if (threadIdx.x == 0) {
      P.mean[i][k] = mean;
      P.rstd[i][k] = rstd;
    }
  }
}

// The same for the backward pass.  CTA b takes rows b, b + grid, ...; each thread owns its columns' sums of dgamma
// and dbeta, in shared memory where they fit (`near`), else in the CTA's slice of the workspace.
template <typename T, int B>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_any_kernel(const __grid_constant__ NormBwd P, int near) {
  using Wd = typename Word<B>::type;
  constexpr int E = B / sizeof(T);
  extern __shared__ __align__(16) float any_sums[];        // [2][h]
  __shared__ float red[kNormThreads / 32];
  const int64_t words = P.h / E;
  float* part = P.part + static_cast<int64_t>(blockIdx.x) * 2 * P.h;
  float* pg = near ? any_sums : part;
  float* pb = pg + P.h;
  for (int64_t v = threadIdx.x; v < words; v += kNormThreads)
#pragma unroll
    for (int e = 0; e < E; ++e) pg[v * E + e] = pb[v * E + e] = 0.0f;
  for (int64_t row = blockIdx.x; row < P.total; row += gridDim.x) {
    const int i = static_cast<int>(row / P.rows);
    const int64_t k = row - i * P.rows;
    const Wd* x = reinterpret_cast<const Wd*>(static_cast<const T*>(P.x[i]) + k * P.ldx);
    const Wd* dy = reinterpret_cast<const Wd*>(static_cast<const T*>(P.dy[i]) + k * P.lddy);
    const Wd* ds = P.ds[i] ? reinterpret_cast<const Wd*>(static_cast<const T*>(P.ds[i]) + k * P.ldds) : nullptr;
    Wd* dx = reinterpret_cast<Wd*>(static_cast<T*>(P.dx[i]) + k * P.h);
    const float mean = P.mean[i][k], rstd = P.rstd[i][k];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll 2
    for (int64_t v = threadIdx.x; v < words; v += kNormThreads) {
      float f[E], d[E];
      unpack<T, B>(x[v], f);
      unpack<T, B>(dy[v], d);
      float ga[E];
      load_weights<E>(P.gamma, P.wtype, v * E, ga);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float g = d[e] * ga[e];
        f[e] = (f[e] - mean) * rstd;
        s1 += g;
        s2 = fmaf(g, f[e], s2);
      }
      if constexpr (E >= 4) {
        float4* a = reinterpret_cast<float4*>(pg + v * E);
        float4* b = reinterpret_cast<float4*>(pb + v * E);
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          float4 p = a[e / 4], q = b[e / 4];
          p.x = fmaf(d[e], f[e], p.x);
          p.y = fmaf(d[e + 1], f[e + 1], p.y);
          p.z = fmaf(d[e + 2], f[e + 2], p.z);
          p.w = fmaf(d[e + 3], f[e + 3], p.w);
          q.x += d[e];
          q.y += d[e + 1];
          q.z += d[e + 2];
          q.w += d[e + 3];
          a[e / 4] = p;
          b[e / 4] = q;
        }
      } else {
        pg[v] = fmaf(d[0], f[0], pg[v]);
        pb[v] += d[0];
      }
    }
    const float c1 = block_sum(s1, red) / static_cast<float>(P.h);
    const float c2 = block_sum(s2, red) / static_cast<float>(P.h);
#pragma unroll 2
    for (int64_t v = threadIdx.x; v < words; v += kNormThreads) {
      float f[E], d[E];
      unpack<T, B>(x[v], f);
      unpack<T, B>(dy[v], d);
      float ga[E];
      load_weights<E>(P.gamma, P.wtype, v * E, ga);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float xh = (f[e] - mean) * rstd;
        f[e] = rstd * (d[e] * ga[e] - c1 - xh * c2);
      }
      if (ds) {
        unpack<T, B>(ds[v], d);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] += d[e];
      }
      dx[v] = pack<T, B>(f);
    }
  }
  if (near) {
    __syncthreads();
    for (int64_t c = threadIdx.x; c < 2 * P.h; c += kNormThreads) part[c] = any_sums[c];
  }
}

// dgamma and dbeta: the partial sums joined in the order of the CTAs.  One warp per 32 columns of
// one of the two, 32 warps of a CTA each taking every 32nd part.
__global__ void __launch_bounds__(1024) norm_join_kernel(const float* part, int nparts, int64_t h, float* dgamma,
                                                         float* dbeta, int accumulate) {
  __shared__ float red[32][33];
  await_previous();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  float s = 0.0f;
  if (c < h)
#pragma unroll 8
    for (int p = w; p < nparts; p += 32) s += part[(static_cast<int64_t>(p) * 2 + blockIdx.y) * h + c];
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < h) {
    float v = red[0][lane];
#pragma unroll
    for (int j = 1; j < 32; ++j) v += red[j][lane];
    out[c] = accumulate ? out[c] + v : v;
  }
}

int elem_bytes(int type) { return type == TTL_T_F32 ? 4 : 2; }

int check_common(int t, int64_t rows, int64_t h, int x_type, int w_type, const char* name) {
  if (t < 1 || t > kMaxShards) return set_error(TTL_ERR_ARG, "%s: t=%d outside [1,%d]", name, t, kMaxShards);
  if (rows < 0 || h < 1) return set_error(TTL_ERR_ARG, "%s: rows < 0 or h < 1", name);
  if ((x_type != TTL_T_BF16 && x_type != TTL_T_F32) || (w_type != TTL_T_BF16 && w_type != TTL_T_F32))
    return set_error(TTL_ERR_ARG, "%s: unknown element type", name);
  if (h >= (int64_t(1) << 31) || rows >= (int64_t(1) << 40)) return set_error(TTL_ERR_SHAPE, "%s: extent too large", name);
  return TTL_OK;
}

int check_ptr(const void* p, int bytes, const char* what, const char* name) {
  if (!p) return set_error(TTL_ERR_ARG, "%s: %s is null", name, what);
  if (reinterpret_cast<uintptr_t>(p) % bytes)
    return set_error(TTL_ERR_ALIGN, "%s: %s not aligned to its elements", name, what);
  return TTL_OK;
}

int check_slabs(const void* const* a, int t, int bytes, const char* what, const char* name) {
  if (!a) return set_error(TTL_ERR_ARG, "%s: %s: null slab array", name, what);
  for (int i = 0; i < t; ++i)
    if (int rc = check_ptr(a[i], bytes, what, name)) return rc;
  return TTL_OK;
}

// How a row of h elements is spread: B bytes per word, NV words per thread, W warps per row, G rows at a
// time per CTA, `ctas` CTAs on an SM; stages > 0: through the ring, with that many rows of a group in shared memory
// (smem bytes in all).  W = 0: wider than all of these, the kernel that reads its row again takes it.
struct Spread {
  int B, NV, W, G, stages, ctas;
  size_t smem;
};

// `inputs` rows (x, r, or x, dy, ds) come in for each row.
Spread spread_of(int64_t h, int elem, int B, bool bwd, int inputs) {
  Spread s = {B, 0, 0, 1, 0, 2, 0};
  const int64_t words = h * elem / B;
  const int E = B / elem;
  auto fit = [&](int nv, int warps) {
    if (s.W || words > static_cast<int64_t>(nv) * 32 * warps) return;
    s.NV = nv;
    s.W = static_cast<int>((words + nv * 32 - 1) / (nv * 32));
  };
  // (32768 rows, forward: 800 bytes fp32 with a residual 20 us through the ring, 31 in registers; 602 bytes of single
  // values 36 and 77; 512 bytes, 65536 rows, 30 and 21.  Backward: 800 bytes 29 and 26, 602 bytes 52 and 40)
  if (h * elem > (bwd ? 1023 : 512)) {
    // 16 values a thread: fewer leave too little work between the row's exchanges, more hold the registers
    // that other rows need (8192 x 4096: fp32 forward 45 us with 16 values, 53 with eight).  The backward pass
    // holds five registers a value: eight where the words are fp32 or short (fp32 80 us with eight values, 83 with
    // 16; 4099 x 1001 fp32 19 and 35).
    if (bwd && (elem == 4 || B < 16)) fit(8 / E, kMaxWarps);
    fit(16 / E, 8);
    fit(16 / E, kMaxWarps);
    fit(24 / E, kMaxWarps);
    if (!bwd || elem == 2) fit(32 / E, kMaxWarps);            // (fp32 rows that wide do not fit below)
    if (!s.W) return s;
    if (s.W < 8) s.G = 8 / s.W;
    s.ctas = s.W * s.G <= 8 ? 2 : 1;
    const size_t room = B == 16 ? h * elem : (h * elem + 30) / 16 * 16;
    const size_t stage = room * inputs * s.G;
    const size_t sums = bwd && s.G > 1 ? static_cast<size_t>(h) * 8 : 0;
    const size_t budget = 226000 / s.ctas - 2048;
    size_t n = sums < budget ? (budget - sums) / stage : 0;
    n = n < 2 ? 2 : (n > kMaxStages ? kMaxStages : n);
    if (bwd && s.NV * E > 16 && n < 3) n = 3;                 // one of them is the row that is being stored
    if (n * stage + sums > 224000) {
      s.W = 0;
      return s;
    }
    s.stages = static_cast<int>(n);
    s.smem = n * stage + sums;
    return s;
  }
  fit(B == 16 ? 1 : (bwd ? 4 : 16 / B), 1);
  if (bwd) {
    fit(B == 16 ? 2 : 8, 1);
    if (B < 16) fit(8, 2);
  }
  if (s.W < 8) s.G = 8 / s.W;
  // (65536 rows of 256 bf16: forward 28 us with two CTAs an SM, 21 with four, 24 with six; the backward pass has
  // registers for two, with four values a thread for three: 32768 rows of 77 fp32 26 and 23 us)
  if (!bwd) s.ctas = 4;
  else if (s.NV * E <= 4) s.ctas = 3;
  if (bwd && s.G > 1) s.smem = static_cast<size_t>(h) * 8;
  return s;
}

unsigned fwd_grid(const NormFwd& P, const Spread& sp) {
  const int64_t ctas = (P.total + sp.G - 1) / sp.G;
  const int64_t cap = static_cast<int64_t>(num_sms()) * sp.ctas;
  return static_cast<unsigned>(ctas < cap ? ctas : cap);
}

template <typename T, int B, int NV>
int fwd_ring(const NormFwd& P, const Spread& sp, cudaStream_t s) {
  if (int rc = allow_smem<norm_fwd_ring_kernel<T, B, NV>>(sp.smem, "cudaFuncSetAttribute(layer norm)")) return rc;
  norm_fwd_ring_kernel<T, B, NV><<<fwd_grid(P, sp), sp.W * sp.G * 32, sp.smem, s>>>(P, sp.W, sp.G, sp.stages);
  return TTL_OK;
}

template <typename T, int B, int NV>
int fwd_regs(const NormFwd& P, const Spread& sp, cudaStream_t s) {
  norm_fwd_kernel<T, B, NV><<<fwd_grid(P, sp), sp.G * 32, 0, s>>>(P, sp.G);
  return TTL_OK;
}

template <typename T, int B, int NV>
int bwd_ring(const NormBwd& P, const Spread& sp, int parts, cudaStream_t s) {
  if (int rc = allow_smem<norm_bwd_ring_kernel<T, B, NV>>(sp.smem, "cudaFuncSetAttribute(layer norm)")) return rc;
  norm_bwd_ring_kernel<T, B, NV><<<parts, sp.W * sp.G * 32, sp.smem, s>>>(P, sp.W, sp.G, sp.stages);
  return TTL_OK;
}

template <typename T, int B, int NV>
int bwd_regs(const NormBwd& P, const Spread& sp, int parts, cudaStream_t s) {
  norm_bwd_kernel<T, B, NV><<<parts, sp.W * sp.G * 32, sp.smem, s>>>(P, sp.W, sp.G);
  return TTL_OK;
}

// Up to 220 KB of sums stay in shared memory; the partial rows are as many as the CTAs that fit then.
template <typename T, int B>
int bwd_any(const NormBwd& P, int parts, cudaStream_t s) {
  const size_t sums = static_cast<size_t>(P.h) * 8;
  const int near = sums <= kAnySums;
  if (near)
    if (int rc = allow_smem<norm_bwd_any_kernel<T, B>>(sums, "cudaFuncSetAttribute(layer norm)")) return rc;
  norm_bwd_any_kernel<T, B><<<parts, kNormThreads, near ? sums : 0, s>>>(P, near);
  return TTL_OK;
}

template <typename T, int B>
int pick_fwd(const NormFwd& P, const Spread& sp, cudaStream_t s) {
  constexpr int E = B / sizeof(T);
  if (sp.stages > 0) {
    if (sp.NV == 16 / E) return fwd_ring<T, B, 16 / E>(P, sp, s);
    return sp.NV == 24 / E ? fwd_ring<T, B, 24 / E>(P, sp, s) : fwd_ring<T, B, 32 / E>(P, sp, s);
  }
  return fwd_regs<T, B, B == 16 ? 1 : 16 / B>(P, sp, s);   // (16 / B words of 32 lanes: 512 bytes)
}

template <typename T, int B>
int pick_bwd(const NormBwd& P, const Spread& sp, int parts, cudaStream_t s) {
  constexpr int E = B / sizeof(T);
  if (sp.stages > 0) {
    if constexpr (sizeof(T) == 4 || B < 16)
      if (sp.NV == 8 / E) return bwd_ring<T, B, 8 / E>(P, sp, parts, s);
    if constexpr (sizeof(T) == 2)
      if (sp.NV == 32 / E) return bwd_ring<T, B, 32 / E>(P, sp, parts, s);
    return sp.NV == 24 / E ? bwd_ring<T, B, 24 / E>(P, sp, parts, s) : bwd_ring<T, B, 16 / E>(P, sp, parts, s);
  }
  if constexpr (B == 16) return sp.NV == 1 ? bwd_regs<T, B, 1>(P, sp, parts, s) : bwd_regs<T, B, 2>(P, sp, parts, s);
  else return sp.NV == 4 ? bwd_regs<T, B, 4>(P, sp, parts, s) : bwd_regs<T, B, 8>(P, sp, parts, s);
}

// The widest word that every row is made of: 16 bytes, or 4, or the element.
int word_of(uintptr_t ptrs, int64_t strides, int64_t h, int elem) {
  const uintptr_t all = ptrs | static_cast<uintptr_t>(strides * elem) | static_cast<uintptr_t>(h * elem);
  return all % 16 == 0 ? 16 : (all % 4 == 0 ? 4 : elem);
}

int parts_of(int64_t total) { return static_cast<int>(total < kNormParts ? total : kNormParts); }

}  // namespace
}  // namespace ttl

using namespace ttl;

extern "C" int ttl_layer_norm_fwd(int t, int64_t rows, int64_t h, int x_type, int w_type, const void* const* X,
                                  int64_t ldx, const void* const* R, int64_t ldr, const void* gamma, const void* beta,
                                  float eps, void* const* S, void* const* Y, float* const* mean, float* const* rstd,
                                  void* stream) {
  const char* name = "ttl_layer_norm_fwd";
  int rc = check_common(t, rows, h, x_type, w_type, name);
  if (rc) return rc;
  if (!(eps >= 0.0f)) return set_error(TTL_ERR_ARG, "%s: eps must not be negative", name);
  if (ldx < h || (R && ldr < h)) return set_error(TTL_ERR_SHAPE, "%s: a row stride is smaller than h", name);
  if (!R != !S) return set_error(TTL_ERR_ARG, "%s: the residual R and the sum S come together", name);
  if (rows == 0) return TTL_OK;
  const int xb = elem_bytes(x_type), wb = elem_bytes(w_type);
  using CP = const void* const*;
  if ((rc = check_slabs(X, t, xb, "X", name)) || (rc = check_slabs(reinterpret_cast<CP>(Y), t, xb, "Y", name)) ||
      (R && (rc = check_slabs(R, t, xb, "R", name))) ||
      (S && (rc = check_slabs(reinterpret_cast<CP>(S), t, xb, "S", name))) ||
      (rc = check_slabs(reinterpret_cast<CP>(mean), t, 4, "mean", name)) ||
      (rc = check_slabs(reinterpret_cast<CP>(rstd), t, 4, "rstd", name)) ||
      (rc = check_ptr(gamma, wb, "gamma", name)) || (beta && (rc = check_ptr(beta, wb, "beta", name))))
    return rc;
  {
    const int64_t w = h * xb;
    Operand outs[4] = {operand("Y", reinterpret_cast<CP>(Y), t, rows, w, w),
                       operand("mean", reinterpret_cast<CP>(mean), t, rows * 4),
                       operand("rstd", reinterpret_cast<CP>(rstd), t, rows * 4),
                       operand("S", reinterpret_cast<CP>(S), t, rows, w, w)};
    const Operand ins[4] = {operand("X", X, t, rows, ldx * xb, w), operand("gamma", &gamma, 1, h * wb),
                            operand("beta", &beta, beta ? 1 : 0, h * wb), operand("R", R, R ? t : 0, rows, ldr * xb, w)};
    if ((rc = check_alias(outs, S ? 4 : 3, ins, 4, name))) return rc;
  }
  if ((rc = require_sm103())) return rc;
  NormFwd P = {};
  P.status = device_status_ptr();
  if (!P.status) return TTL_ERR_CUDA;
  for (int i = 0; i < t; ++i) {
    P.x[i] = X[i];
    P.r[i] = R ? R[i] : nullptr;
    P.s[i] = S ? S[i] : nullptr;
    P.y[i] = Y[i];
    P.mean[i] = mean[i];
    P.rstd[i] = rstd[i];
  }
  P.gamma = gamma;
  P.beta = beta;
  P.rows = rows;
  P.h = h;
  P.ldx = ldx;
  P.ldr = ldr;
  P.total = rows * t;
  P.eps = eps;
  P.wtype = w_type;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const double n = static_cast<double>(P.total) * h;
  TraceScope trace(s, TTL_K_NORM, 0.0, n * xb * (R ? 4.0 : 2.0));
  uintptr_t ptrs = 0;
  for (int i = 0; i < t; ++i)
    ptrs |= reinterpret_cast<uintptr_t>(X[i]) | reinterpret_cast<uintptr_t>(Y[i]) |
            (R ? reinterpret_cast<uintptr_t>(R[i]) | reinterpret_cast<uintptr_t>(S[i]) : 0);
  const Spread sp = spread_of(h, xb, word_of(ptrs, ldx | (R ? ldr : 0), h, xb), false, R ? 2 : 1);
  if (sp.W == 0) {
    const int64_t cap = static_cast<int64_t>(num_sms()) * 8;
    const unsigned grid = static_cast<unsigned>(P.total < cap ? P.total : cap);
    if (x_type == TTL_T_F32) {
      if (sp.B == 16) norm_fwd_any_kernel<float, 16><<<grid, kNormThreads, 0, s>>>(P);
      else norm_fwd_any_kernel<float, 4><<<grid, kNormThreads, 0, s>>>(P);
    } else {
      if (sp.B == 16) norm_fwd_any_kernel<__nv_bfloat16, 16><<<grid, kNormThreads, 0, s>>>(P);
      else norm_fwd_any_kernel<__nv_bfloat16, 2><<<grid, kNormThreads, 0, s>>>(P);
    }
  } else if (x_type == TTL_T_F32) {
    if (sp.B == 16) rc = pick_fwd<float, 16>(P, sp, s);
    else rc = pick_fwd<float, 4>(P, sp, s);
  } else {
    if (sp.B == 16) rc = pick_fwd<__nv_bfloat16, 16>(P, sp, s);
    else if (sp.B == 4) rc = pick_fwd<__nv_bfloat16, 4>(P, sp, s);
    else rc = pick_fwd<__nv_bfloat16, 2>(P, sp, s);
  }
  if (rc) return rc;
  return cuda_check(cudaGetLastError(), "layer norm forward launch");
}

extern "C" size_t ttl_layer_norm_bwd_workspace_size(int t, int64_t rows, int64_t h) {
  if (check_common(t, rows, h, TTL_T_BF16, TTL_T_BF16, "ttl_layer_norm_bwd_workspace_size")) return 0;
  return static_cast<size_t>(parts_of(rows * t)) * 2 * h * sizeof(float);
}

extern "C" int ttl_layer_norm_bwd(int t, int64_t rows, int64_t h, int x_type, int w_type, const void* const* X,
                                  int64_t ldx, const void* const* dY, int64_t lddy, const void* const* dS,
                                  int64_t ldds, const void* gamma, const float* const* mean,
                                  const float* const* rstd, void* const* dX, float* dgamma, float* dbeta,
                                  int accumulate, void* ws, size_t ws_bytes, void* stream) {
  const char* name = "ttl_layer_norm_bwd";
  int rc = check_common(t, rows, h, x_type, w_type, name);
  if (rc) return rc;
  if (accumulate != 0 && accumulate != 1) return set_error(TTL_ERR_ARG, "%s: accumulate must be 0 or 1", name);
  if (ldx < h || lddy < h || (dS && ldds < h))
    return set_error(TTL_ERR_SHAPE, "%s: a row stride is smaller than h", name);
  if ((rc = check_ptr(dgamma, 4, "dgamma", name)) || (dbeta && (rc = check_ptr(dbeta, 4, "dbeta", name)))) return rc;
  const int xb = elem_bytes(x_type), wb = elem_bytes(w_type);
  using CP = const void* const*;
  if (rows > 0) {
    if ((rc = check_slabs(X, t, xb, "X", name)) || (rc = check_slabs(dY, t, xb, "dY", name)) ||
        (dS && (rc = check_slabs(dS, t, xb, "dS", name))) ||
        (rc = check_slabs(reinterpret_cast<CP>(dX), t, xb, "dX", name)) ||
        (rc = check_slabs(reinterpret_cast<CP>(mean), t, 4, "mean", name)) ||
        (rc = check_slabs(reinterpret_cast<CP>(rstd), t, 4, "rstd", name)) ||
        (rc = check_ptr(gamma, wb, "gamma", name)))
      return rc;
    const size_t need = ttl_layer_norm_bwd_workspace_size(t, rows, h);
    if (!ws || ws_bytes < need)
      return set_error(TTL_ERR_ARG, "%s: workspace of %zu bytes needed, %zu given", name, need, ws_bytes);
    if (!aligned16(ws)) return set_error(TTL_ERR_ALIGN, "%s: workspace not 16-byte aligned", name);
    const int64_t w = h * xb;
    const void *dg = dgamma, *db = dbeta, *space = ws;
    const Operand outs[4] = {operand("dX", reinterpret_cast<CP>(dX), t, rows, w, w), operand("dgamma", &dg, 1, h * 4),
                             operand("dbeta", &db, dbeta ? 1 : 0, h * 4),
                             operand("the workspace", &space, 1, static_cast<int64_t>(need))};
    const Operand ins[6] = {operand("X", X, t, rows, ldx * xb, w), operand("dY", dY, t, rows, lddy * xb, w),
                            operand("gamma", &gamma, 1, h * wb), operand("mean", reinterpret_cast<CP>(mean), t, rows * 4),
                            operand("rstd", reinterpret_cast<CP>(rstd), t, rows * 4),
                            operand("dS", dS, dS ? t : 0, rows, ldds * xb, w)};
    if ((rc = check_alias(outs, 4, ins, 6, name))) return rc;
  }
  if (rows == 0 && accumulate) return TTL_OK;
  if ((rc = require_sm103())) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int parts = 0;
  if (rows > 0) {
    NormBwd P = {};
    P.status = device_status_ptr();
    if (!P.status) return TTL_ERR_CUDA;
    for (int i = 0; i < t; ++i) {
      P.x[i] = X[i];
      P.dy[i] = dY[i];
      P.ds[i] = dS ? dS[i] : nullptr;
      P.dx[i] = dX[i];
      P.mean[i] = mean[i];
      P.rstd[i] = rstd[i];
    }
    P.gamma = gamma;
    P.part = static_cast<float*>(ws);
    P.rows = rows;
    P.h = h;
    P.ldx = ldx;
    P.lddy = lddy;
    P.ldds = ldds;
    P.total = rows * t;
    P.wtype = w_type;
    parts = parts_of(P.total);
    const double n = static_cast<double>(P.total) * h;
    TraceScope trace(s, TTL_K_NORM, 0.0, n * xb * (dS ? 4.0 : 3.0));
    uintptr_t ptrs = 0;
    for (int i = 0; i < t; ++i)
      ptrs |= reinterpret_cast<uintptr_t>(X[i]) | reinterpret_cast<uintptr_t>(dY[i]) |
              reinterpret_cast<uintptr_t>(dX[i]) | (dS ? reinterpret_cast<uintptr_t>(dS[i]) : 0);
    const Spread sp = spread_of(h, xb, word_of(ptrs, ldx | lddy | (dS ? ldds : 0), h, xb), true, dS ? 3 : 2);
    if (sp.W > 0) {
      const int64_t ctas = (P.total + sp.G - 1) / sp.G, cap = sp.ctas * (kNormParts / 3);
      parts = static_cast<int>(ctas < cap ? ctas : cap);
    }
    if (sp.W == 0) {
      // one CTA per SM where its sums take more than half of the shared memory, else two, or three without sums in it
      const size_t sums = static_cast<size_t>(h) * 8;
      const int cap = (sums > kAnySums ? 3 : (sums > kAnySums / 2 ? 1 : 2)) * (kNormParts / 3);
      parts = static_cast<int>(P.total < cap ? P.total : cap);
      if (x_type == TTL_T_F32) rc = sp.B == 16 ? bwd_any<float, 16>(P, parts, s) : bwd_any<float, 4>(P, parts, s);
      else rc = sp.B == 16 ? bwd_any<__nv_bfloat16, 16>(P, parts, s) : bwd_any<__nv_bfloat16, 2>(P, parts, s);
    } else if (x_type == TTL_T_F32) {
      if (sp.B == 16) rc = pick_bwd<float, 16>(P, sp, parts, s);
      else rc = pick_bwd<float, 4>(P, sp, parts, s);
    } else {
      if (sp.B == 16) rc = pick_bwd<__nv_bfloat16, 16>(P, sp, parts, s);
      else if (sp.B == 4) rc = pick_bwd<__nv_bfloat16, 4>(P, sp, parts, s);
      else rc = pick_bwd<__nv_bfloat16, 2>(P, sp, parts, s);
    }
    if (rc || (rc = cuda_check(cudaGetLastError(), "layer norm backward launch"))) return rc;
  }
  TraceScope trace(s, TTL_K_NORM, 0.0, 8.0 * h * parts);
  return cuda_check(launch_after(norm_join_kernel, dim3(static_cast<unsigned>((h + 31) / 32), 2), 1024, 0, s,
                                 static_cast<const float*>(ws), parts, h, dgamma, dbeta, accumulate),
                    "norm_join_kernel launch");
}
