// Norm of every head of Q and K and its rotation by position, in one pass, and the backward pass.
//
// Source: "v4:Tensor Parallel 与 Sequence Parallel", section "Attention:按 head 切": what happens to a head
// between the projection and the scores happens on the shard that holds it.
//
// For one head x of a token, d values:  r = 1 / sqrt(mean(x^2) + eps), n = x r, y = n gamma (y = x without
// weights), and each pair (a, b) of y's first rot columns turns by the angle f = pos[axis] freq of the pair:
//   (a cos f - b sin f, b cos f + a sin f)
// Backward, g = the incoming gradient turned back:  dgamma = sum g n, h = g gamma, dx = r (h - n mean(h n)).
//
// Angles.  A position times a frequency needs more than 32 bits before its whole turns are dropped.  The host
// gives turns per position as a 64-bit fraction of a turn; the integer product with the position wraps at whole turns
// by itself, exactly, for positions of either sign, and its upper 32 bits are the angle to 2^-32 turns.
//
// Layout.  A lane holds 16 columns of a head as two 16-byte words whose columns pair up (columns c.. and rot/2 + c..,
// or 16 neighbours), so a rotation exchanges nothing; the 1 to 16 lanes of a head share a token and join their squares
// by shuffles.  A warp's tokens stay while it walks over a range of heads of all shards: the sines are taken once for
// the range.
//
// What bounds it: bytes.

#include <cmath>

#include "launch_after.cuh"
#include "operands.h"
#include "pack_docs.h"
#include "ttl_device.cuh"
#include "ttl_internal.h"

namespace ttl {
namespace {

constexpr int kMaxHead = 256;
constexpr int kMaxPairs = kMaxHead / 2;
constexpr int kMaxAxes = 8;
constexpr int kWarps = 8;

enum Mode : int {
  kTurn = 0,      // the rotation alone (backward: by the angles' negatives)
  kForward = 1,
  kBackward = 2,  // of the norm and the rotation
};

struct HeadArgs {
  const __nv_bfloat16* in[2][kMaxShards];    // Q and K; backward: their outputs' gradients
  const __nv_bfloat16* x[2][kMaxShards];     // kBackward: Q and K
  __nv_bfloat16* out[2][kMaxShards];
  int64_t ld_in[2], ld_x[2], ld_out[2];
  uint64_t turns[kMaxPairs];                 // per position, in units of 2^-64 turns
  uint8_t axis[kMaxPairs];
  int heads[2];                              // of Q and K on a shard
  uint32_t magic[2];                         // shard of head h of a kind: h magic >> 32 (0: h itself)
  int t, d, rot;
  int64_t T;
  const int32_t* pos;                        // [axes, T]; null: a token's place in its document, or in the pack
  const int32_t* cu;                         // null: every token counts
  int batch;
  const void* gamma[2];
  int w_type;
  float eps;
  float sign;                                // kTurn: -1 turns back
  float* part;                               // kBackward: [blocks][2][d]
  int chunks, chunk;                         // ranges of heads a token group is cut into, heads of one
  int64_t items;                             // token groups x chunks
  int* status;
};

__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }

// The 16 columns of two words as pairs (a[e], b[e]).
template <bool NEIGHBOURS>
__device__ __forceinline__ void to_pairs(const uint4& u, const uint4& v, float (&a)[8], float (&b)[8]) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (NEIGHBOURS) {
      a[e] = bf16_lo(w[e]);
      b[e] = bf16_hi(w[e]);
    } else {
      a[e] = e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
      b[e] = e & 1 ? bf16_hi(w[4 + (e >> 1)]) : bf16_lo(w[4 + (e >> 1)]);
    }
  }
}
template <bool NEIGHBOURS>
__device__ __forceinline__ void store_pairs(__nv_bfloat16* p0, __nv_bfloat16* p1, const float (&a)[8], const float (&b)[8]) {
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (NEIGHBOURS) w[e] = pack_bf16x2(a[e], b[e]);
    else w[e] = e < 4 ? pack_bf16x2(a[2 * e], a[2 * e + 1]) : pack_bf16x2(b[2 * e - 8], b[2 * e - 7]);
  }
  *reinterpret_cast<uint4*>(p0) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(p1) = make_uint4(w[4], w[5], w[6], w[7]);
}

// Reports document bounds that do not start at 0 or above, decrease, or end beyond T.
__device__ __forceinline__ void check_bounds(const HeadArgs& A) {
  bool bad = false;
  for (int b = threadIdx.x; b <= A.batch; b += blockDim.x) {
    const int c = __ldg(A.cu + b);
    bad |= c < 0 || c > A.T || (b > 0 && __ldg(A.cu + b - 1) > c);
  }
  if (bad) atomicCAS(A.status, 0, TTL_ERR_DEVICE);
}

// LANES lanes to a head, each with two words of eight columns.
template <int LANES, bool NEIGHBOURS, int MODE>
__global__ void __launch_bounds__(kWarps * 32, 2) head_rotary_kernel(const __grid_constant__ HeadArgs A) {
  constexpr int kTokens = 32 / LANES;
  __shared__ uint64_t turns[kMaxPairs];
  __shared__ uint8_t axis[kMaxPairs];
  __shared__ float gamma[MODE == kTurn ? 1 : 2][kMaxHead];
  __shared__ float sums[MODE == kBackward ? kWarps : 1][2][kMaxHead];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < A.rot / 2; i += kWarps * 32) {
    turns[i] = A.turns[i];
    axis[i] = A.axis[i];
  }
  if constexpr (MODE != kTurn) {
    for (int i = threadIdx.x; i < 2 * A.d; i += kWarps * 32) {
      const int kind = i >= A.d, c = i - kind * A.d;
      gamma[kind][c] = A.w_type == TTL_T_F32 ? static_cast<const float*>(A.gamma[kind])[c]
                                             : __bfloat162float(static_cast<const __nv_bfloat16*>(A.gamma[kind])[c]);
    }
  }
  if (A.cu && blockIdx.x == 0) check_bounds(A);
  __syncthreads();

  const int slot = lane % LANES;
  const bool mine = slot < A.d / 16;              // (a head whose 16-column slots are no power of two leaves lanes idle)
  // the slot's columns, and its pairs
  int c0 = slot * 16, c1 = c0 + 8;
  if (!NEIGHBOURS && slot < A.rot / 16) {
    c0 = slot * 8;
    c1 = A.rot / 2 + c0;
  }
  const float inv_d = 1.0f / static_cast<float>(A.d);
  float acc[2][16];
  if constexpr (MODE == kBackward) {
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[0][e] = acc[1][e] = 0.0f;
  }

  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp; item < A.items;
       item += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t group = item / A.chunks;
    const int h0 = static_cast<int>(item - group * A.chunks) * A.chunk;
    const int all = A.t * (A.heads[0] + A.heads[1]);
    const int h1 = h0 + A.chunk < all ? h0 + A.chunk : all;
    const int64_t tok = group * kTokens + lane / LANES;
    const bool there = tok < A.T;
    DocRange doc{0, static_cast<int>(A.T)};
    if (A.cu) doc = doc_of(A.cu, A.batch, static_cast<int>(A.T), there ? static_cast<int>(tok) : -1);
    const bool counts = there && doc.hi > doc.lo;
    float co[8], si[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int pair = slot * 8 + e;
      co[e] = 1.0f;
      si[e] = 0.0f;
      if (pair < A.rot / 2 && counts) {
        const int64_t p = A.pos ? __ldg(A.pos + axis[pair] * A.T + tok) : tok - doc.lo;
        const uint64_t turn = turns[pair] * static_cast<uint64_t>(p);
        sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &si[e], &co[e]);
      }
      if constexpr (MODE == kTurn) si[e] *= A.sign;
    }
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const int base = kind ? A.t * A.heads[0] : 0;
      const int begin = (h0 > base ? h0 : base) - base;
      const int last = kind ? all : A.t * A.heads[0];
      const int end = (h1 < last ? h1 : last) - base;
      if (begin >= end) continue;
      float ga[8], gb[8];
      if constexpr (MODE != kTurn) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ga[e] = mine ? gamma[kind][NEIGHBOURS ? c0 + 2 * e : c0 + e] : 0.0f;
          gb[e] = mine ? gamma[kind][NEIGHBOURS ? c0 + 2 * e + 1 : c1 + e] : 0.0f;
        }
      }
      constexpr int kAtOnce = MODE == kBackward ? 1 : 2;   // heads whose words are loaded before the first is worked on
#pragma unroll 1
      for (int h = begin; h < end; h += kAtOnce) {
        uint4 u[kAtOnce], v[kAtOnce], xu[kAtOnce], xv[kAtOnce];
        int shard[kAtOnce], col[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const int hk = h + k < end ? h + k : h;
          shard[k] = A.magic[kind] ? static_cast<int>(__umulhi(static_cast<uint32_t>(hk), A.magic[kind])) : hk;
          col[k] = (hk - shard[k] * A.heads[kind]) * A.d;
          u[k] = v[k] = xu[k] = xv[k] = make_uint4(0, 0, 0, 0);
          if (mine && counts) {
            const __nv_bfloat16* p = A.in[kind][shard[k]] + tok * A.ld_in[kind] + col[k];
            u[k] = load16(p + c0);
            v[k] = load16(p + c1);
            if constexpr (MODE == kBackward) {
              const __nv_bfloat16* q = A.x[kind][shard[k]] + tok * A.ld_x[kind] + col[k];
              xu[k] = load16(q + c0);
              xv[k] = load16(q + c1);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          float a[8], b[8], ya[8], yb[8];
          to_pairs<NEIGHBOURS>(u[k], v[k], a, b);
          if constexpr (MODE == kForward) {
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
#pragma unroll
            for (int o = LANES >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = rsqrtf(fmaf(ss, inv_d, A.eps));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              a[e] *= r * ga[e];
              b[e] *= r * gb[e];
            }
          }
          if constexpr (MODE != kBackward) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              ya[e] = fmaf(a[e], co[e], -b[e] * si[e]);
              yb[e] = fmaf(b[e], co[e], a[e] * si[e]);
            }
          } else {
            float na[8], nb[8];
            to_pairs<NEIGHBOURS>(xu[k], xv[k], na, nb);
            float ss = 0.0f, dot = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float g0 = fmaf(a[e], co[e], b[e] * si[e]), g1 = fmaf(b[e], co[e], -a[e] * si[e]);
              ss = fmaf(na[e], na[e], fmaf(nb[e], nb[e], ss));
              a[e] = g0;
              b[e] = g1;
              dot = fmaf(g0 * ga[e], na[e], fmaf(g1 * gb[e], nb[e], dot));
            }
#pragma unroll
            for (int o = LANES >> 1; o > 0; o >>= 1) {
              ss += __shfl_xor_sync(0xffffffffu, ss, o);
              dot += __shfl_xor_sync(0xffffffffu, dot, o);
            }
            const float r = rsqrtf(fmaf(ss, inv_d, A.eps));
            const float m = dot * r * inv_d;      // mean of h n
            const bool add = counts && h + k < end;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              na[e] *= r;
              nb[e] *= r;
              acc[kind][e] += add ? a[e] * na[e] : 0.0f;
              acc[kind][8 + e] += add ? b[e] * nb[e] : 0.0f;
              ya[e] = r * fmaf(a[e], ga[e], -na[e] * m);
              yb[e] = r * fmaf(b[e], gb[e], -nb[e] * m);
            }
          }
          if (!counts) {
#pragma unroll
            for (int e = 0; e < 8; ++e) ya[e] = yb[e] = 0.0f;
          }
          if (mine && there && h + k < end) {
            __nv_bfloat16* p = A.out[kind][shard[k]] + tok * A.ld_out[kind] + col[k];
            store_pairs<NEIGHBOURS>(p + c0, p + c1, ya, yb);
          }
        }
      }
    }
  }

  if constexpr (MODE == kBackward) {
    // the block's sums: over the warp's tokens, then over its warps in their order
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float a = acc[kind][e], b = acc[kind][8 + e];
#pragma unroll
        for (int o = 16; o >= LANES; o >>= 1) {
          a += __shfl_xor_sync(0xffffffffu, a, o);
          b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if (lane < LANES && mine) {
          sums[warp][kind][NEIGHBOURS ? c0 + 2 * e : c0 + e] = a;
          sums[warp][kind][NEIGHBOURS ? c0 + 2 * e + 1 : c1 + e] = b;
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * A.d; i += kWarps * 32) {
      const int kind = i >= A.d, c = i - kind * A.d;
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sums[w][kind][c];
      A.part[static_cast<int64_t>(blockIdx.x) * 2 * A.d + i] = s;
    }
  }
}

// dgamma from the blocks' sums, in their order: 32 columns a block, eight warps on every eighth row.
__global__ void __launch_bounds__(256) head_join_kernel(const float* part, int rows, int d, float* dq, float* dk, int accumulate) {
  __shared__ float sums[8][32];
  await_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < 2 * d)
#pragma unroll 8
    for (int r = warp; r < rows; r += 8) s += part[static_cast<int64_t>(r) * 2 * d + c];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < 2 * d) {
    for (int w = 1; w < 8; ++w) s += sums[w][lane];
    float* out = c < d ? dq + c : dk + (c - d);
    *out = accumulate ? *out + s : s;
  }
}

int lanes_of(int d) {
  int l = 1;
  while (l * 16 < d) l *= 2;
  return l;
}

// Blocks of the backward launch, at most: what its workspace holds partial sums for.
constexpr int kMaxBlocks = 2 * 152;

int blocks_of(int64_t items) {
  const int64_t need = (items + kWarps - 1) / kWarps;
  return static_cast<int>(need < kMaxBlocks ? need : kMaxBlocks);
}

// How the heads of a token group are cut: into ranges of no fewer than eight, more where the groups alone are too few
// warps for the card.
void cut_heads(HeadArgs& A) {
  const int all = A.t * (A.heads[0] + A.heads[1]);
  const int64_t groups = (A.T + 32 / lanes_of(A.d) - 1) / (32 / lanes_of(A.d));
  const int64_t want = 152 * 2 * kWarps;
  int64_t chunk = all * groups / want;
  chunk = chunk < 2 ? 2 : (chunk > 8 ? 8 : chunk);
  A.chunk = static_cast<int>(chunk < all ? chunk : all);
  A.chunks = (all + A.chunk - 1) / A.chunk;
  A.items = groups * A.chunks;
}

template <int MODE>
int launch(const HeadArgs& A, bool neighbours, unsigned grid, cudaStream_t s) {
  const double size = static_cast<double>(A.T) * A.t * (A.heads[0] + A.heads[1]) * A.d;
  TraceScope trace(s, TTL_K_NORM, 0.0, size * (MODE == kBackward ? 6.0 : 4.0));
  auto go = [&](auto kernel) { return cuda_check(launch_first(kernel, dim3(grid), kWarps * 32, 0, s, A), "head_rotary_kernel launch"); };
  switch (lanes_of(A.d)) {
    case 1: return neighbours ? go(head_rotary_kernel<1, true, MODE>) : go(head_rotary_kernel<1, false, MODE>);
    case 2: return neighbours ? go(head_rotary_kernel<2, true, MODE>) : go(head_rotary_kernel<2, false, MODE>);
    case 4: return neighbours ? go(head_rotary_kernel<4, true, MODE>) : go(head_rotary_kernel<4, false, MODE>);
    case 8: return neighbours ? go(head_rotary_kernel<8, true, MODE>) : go(head_rotary_kernel<8, false, MODE>);
    default: return neighbours ? go(head_rotary_kernel<16, true, MODE>) : go(head_rotary_kernel<16, false, MODE>);
  }
}

int check_shape(int t, int64_t T, int n_q, int n_kv, int d, const char* name) {
  if (t < 1 || t > kMaxShards) return set_error(TTL_ERR_ARG, "%s: t=%d outside [1,%d]", name, t, kMaxShards);
  if (T < 0 || n_q < 1 || n_kv < 1 || d < 1) return set_error(TTL_ERR_ARG, "%s: bad shape", name);
  if (n_q % t || n_kv % t)
    return set_error(TTL_ERR_SHAPE, "%s: t=%d must divide the head counts %d and %d", name, t, n_q, n_kv);
  if (d % 16 || d > kMaxHead)
    return set_error(TTL_ERR_SHAPE, "%s: head dimension %d is not a multiple of 16 up to %d", name, d, kMaxHead);
  if (T >= (int64_t(1) << 31) - 1 || n_q > 32768 || n_kv > 32768) return set_error(TTL_ERR_SHAPE, "%s: extent too large", name);
  return TTL_OK;
}

// What both directions say about positions: fills A.
int check_rotary(HeadArgs& A, int rot, int neighbours, const double* freqs, const int32_t* pair_axis, int axes,
                 const int32_t* positions, int batch, const int32_t* cu, const char* name) {
  if (rot < 0 || rot > A.d || rot % 16)
    return set_error(TTL_ERR_SHAPE, "%s: %d rotated columns: not a multiple of 16 up to d=%d", name, rot, A.d);
  if (neighbours != 0 && neighbours != 1) return set_error(TTL_ERR_ARG, "%s: interleaved must be 0 or 1", name);
  if (axes < 1 || axes > kMaxAxes) return set_error(TTL_ERR_ARG, "%s: axes=%d outside [1,%d]", name, axes, kMaxAxes);
  if (!positions && axes != 1) return set_error(TTL_ERR_ARG, "%s: %d axes need positions", name, axes);
  if (rot && !freqs) return set_error(TTL_ERR_ARG, "%s: freqs is null", name);
  if (reinterpret_cast<uintptr_t>(positions) & 3) return set_error(TTL_ERR_ALIGN, "%s: positions not 4-byte aligned", name);
  if (batch < 0) return set_error(TTL_ERR_ARG, "%s: bad shape", name);
  if (reinterpret_cast<uintptr_t>(cu) & 3) return set_error(TTL_ERR_ALIGN, "%s: cu_seqlens not 4-byte aligned", name);
  for (int i = 0; i < rot / 2; ++i) {
    // (2^20 radians a position: beyond any use, and small enough for the fraction below)
    if (!(std::fabs(freqs[i]) <= 1048576.0)) return set_error(TTL_ERR_ARG, "%s: freqs[%d] is not a frequency", name, i);
    const double turns = std::fabs(freqs[i]) / 6.283185307179586476925;
    const uint64_t part = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64));   // (below 2^64: both steps are exact)
    A.turns[i] = freqs[i] < 0.0 ? 0 - part : part;
    const int axis = pair_axis ? pair_axis[i] : 0;
    if (axis < 0 || axis >= axes) return set_error(TTL_ERR_ARG, "%s: pair %d is on axis %d of %d", name, i, axis, axes);
    A.axis[i] = static_cast<uint8_t>(axis);
  }
  A.rot = rot;
  A.pos = positions;
  A.cu = cu;
  A.batch = batch;
  return TTL_OK;
}

int check_mats(const ttl_bf16* const* a, int t, int64_t cols, int64_t ld, const char* what, const char* name) {
  if (!a) return set_error(TTL_ERR_ARG, "%s: %s: null shard array", name, what);
  if (ld < cols) return set_error(TTL_ERR_SHAPE, "%s: %s: row stride smaller than its columns", name, what);
  if (ld % 8) return set_error(TTL_ERR_ALIGN, "%s: %s: row stride not a multiple of 8", name, what);
  if (ld >= (int64_t(1) << 31)) return set_error(TTL_ERR_SHAPE, "%s: %s: row stride too large", name, what);
  for (int i = 0; i < t; ++i) {
    if (!a[i]) return set_error(TTL_ERR_ARG, "%s: %s[%d] is null", name, what, i);
    if (!aligned16(a[i])) return set_error(TTL_ERR_ALIGN, "%s: %s[%d] not 16-byte aligned", name, what, i);
  }
  return TTL_OK;
}

int check_weights(HeadArgs& A, int w_type, const void* gamma_q, const void* gamma_k, float eps, const char* name) {
  if (!gamma_q != !gamma_k) return set_error(TTL_ERR_ARG, "%s: gamma_q and gamma_k go together", name);
  if (!gamma_q) return TTL_OK;
  if (w_type != TTL_T_BF16 && w_type != TTL_T_F32) return set_error(TTL_ERR_ARG, "%s: unknown weight type %d", name, w_type);
  const uintptr_t mask = w_type == TTL_T_F32 ? 3 : 1;
  if ((reinterpret_cast<uintptr_t>(gamma_q) | reinterpret_cast<uintptr_t>(gamma_k)) & mask)
    return set_error(TTL_ERR_ALIGN, "%s: gamma not aligned to its elements", name);
  if (!(eps >= 0.0f && eps < INFINITY)) return set_error(TTL_ERR_ARG, "%s: eps must be finite and not negative", name);
  A.gamma[0] = gamma_q;
  A.gamma[1] = gamma_k;
  A.w_type = w_type;
  A.eps = eps;
  return TTL_OK;
}

Operand mats(const char* name, const ttl_bf16* const* at, int t, int64_t T, int64_t ld, int64_t cols) {
  return operand(name, reinterpret_cast<const void* const*>(at), t, T, ld * 2, cols * 2);
}

// Whether the outputs are the inputs themselves, shard by shard: every word is read and written by one thread.
bool in_place(const ttl_bf16* const* in, int64_t ld_in, ttl_bf16* const* out, int64_t ld_out, int t) {
  if (ld_in != ld_out) return false;
  for (int i = 0; i < t; ++i)
    if (in[i] != out[i]) return false;
  return true;
}

uint32_t magic_of(int n) { return n == 1 ? 0u : static_cast<uint32_t>((uint64_t(1) << 32) / n + 1); }

void fill_mats(HeadArgs& A, int kind, const ttl_bf16* const* in, int64_t ld_in, ttl_bf16* const* out, int64_t ld_out) {
  for (int i = 0; i < A.t; ++i) {
    A.in[kind][i] = reinterpret_cast<const __nv_bfloat16*>(in[i]);
    A.out[kind][i] = reinterpret_cast<__nv_bfloat16*>(out[i]);
  }
  A.ld_in[kind] = ld_in;
  A.ld_out[kind] = ld_out;
}

}  // namespace
}  // namespace ttl

using namespace ttl;

extern "C" int ttl_head_norm_rotary_fwd(int t, int64_t T, int n_q, int n_kv, int d, int rot, int interleaved,
                                        const double* freqs, const int32_t* pair_axis, int axes,
                                        const int32_t* positions, int batch, const int32_t* cu_seqlens, int w_type,
                                        const void* gamma_q, const void* gamma_k, float eps, const ttl_bf16* const* Q,
                                        int64_t ldq, const ttl_bf16* const* K, int64_t ldk, ttl_bf16* const* Qo,
                                        int64_t ldqo, ttl_bf16* const* Ko, int64_t ldko, void* stream) {
  const char* name = "ttl_head_norm_rotary_fwd";
  HeadArgs A = {};
  int rc = check_shape(t, T, n_q, n_kv, d, name);
  if (rc) return rc;
  A.t = t; A.T = T; A.d = d; A.heads[0] = n_q / t; A.heads[1] = n_kv / t;
  A.magic[0] = magic_of(A.heads[0]); A.magic[1] = magic_of(A.heads[1]);
  if ((rc = check_rotary(A, rot, interleaved, freqs, pair_axis, axes, positions, batch, cu_seqlens, name)) ||
      (rc = check_weights(A, w_type, gamma_q, gamma_k, eps, name)))
    return rc;
  if (T == 0) return TTL_OK;
  const int64_t qc = static_cast<int64_t>(A.heads[0]) * d, kc = static_cast<int64_t>(A.heads[1]) * d;
  if ((rc = check_mats(Q, t, qc, ldq, "Q", name)) || (rc = check_mats(K, t, kc, ldk, "K", name)) ||
      (rc = check_mats(Qo, t, qc, ldqo, "the output Q", name)) || (rc = check_mats(Ko, t, kc, ldko, "the output K", name)))
    return rc;
  {
    const Operand outs[2] = {mats("Q", Qo, t, T, ldqo, qc), mats("K", Ko, t, T, ldko, kc)};
    const int64_t w = d * (w_type == TTL_T_F32 ? 4 : 2);
    const void *pos = positions, *cu = cu_seqlens;
    Operand ins[6];
    int n = 0;
    if (!in_place(Q, ldq, Qo, ldqo, t)) ins[n++] = mats("the input Q", Q, t, T, ldq, qc);
    if (!in_place(K, ldk, Ko, ldko, t)) ins[n++] = mats("the input K", K, t, T, ldk, kc);
    if (positions) ins[n++] = operand("positions", &pos, 1, axes * T * 4);
    if (cu_seqlens) ins[n++] = operand("cu_seqlens", &cu, 1, (int64_t(batch) + 1) * 4);
    if (gamma_q) {
      ins[n++] = operand("gamma_q", &gamma_q, 1, w);
      ins[n++] = operand("gamma_k", &gamma_k, 1, w);
    }
    if ((rc = check_alias(outs, 2, ins, n, name))) return rc;
  }
  if ((rc = require_sm103())) return rc;
  A.status = device_status_ptr();
  if (!A.status) return TTL_ERR_CUDA;
  fill_mats(A, 0, Q, ldq, Qo, ldqo);
  fill_mats(A, 1, K, ldk, Ko, ldko);
  A.sign = 1.0f;
  cut_heads(A);
  const int64_t need = (A.items + kWarps - 1) / kWarps;
  const unsigned grid = static_cast<unsigned>(need < (1 << 30) ? need : (1 << 30));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return gamma_q ? launch<kForward>(A, interleaved, grid, s) : launch<kTurn>(A, interleaved, grid, s);
}

extern "C" size_t ttl_head_norm_rotary_bwd_workspace_size(int t, int64_t T, int n_q, int n_kv, int d) {
  if (check_shape(t, T, n_q, n_kv, d, "ttl_head_norm_rotary_bwd_workspace_size")) return 0;
  return static_cast<size_t>(kMaxBlocks) * 2 * d * 4;
}

extern "C" int ttl_head_norm_rotary_bwd(int t, int64_t T, int n_q, int n_kv, int d, int rot, int interleaved,
                                        const double* freqs, const int32_t* pair_axis, int axes,
                                        const int32_t* positions, int batch, const int32_t* cu_seqlens, int w_type,
                                        const void* gamma_q, const void* gamma_k, float eps, const ttl_bf16* const* dY_q,
                                        int64_t lddyq, const ttl_bf16* const* dY_k, int64_t lddyk,
                                        const ttl_bf16* const* Q, int64_t ldq, const ttl_bf16* const* K, int64_t ldk,
                                        ttl_bf16* const* dQ, int64_t lddq, ttl_bf16* const* dK, int64_t lddk,
                                        float* dgamma_q, float* dgamma_k, int accumulate, void* ws, size_t ws_bytes,
                                        void* stream) {
  const char* name = "ttl_head_norm_rotary_bwd";
  HeadArgs A = {};
  int rc = check_shape(t, T, n_q, n_kv, d, name);
  if (rc) return rc;
  A.t = t; A.T = T; A.d = d; A.heads[0] = n_q / t; A.heads[1] = n_kv / t;
  A.magic[0] = magic_of(A.heads[0]); A.magic[1] = magic_of(A.heads[1]);
  if ((rc = check_rotary(A, rot, interleaved, freqs, pair_axis, axes, positions, batch, cu_seqlens, name)) ||
      (rc = check_weights(A, w_type, gamma_q, gamma_k, eps, name)))
    return rc;
  if (accumulate != 0 && accumulate != 1) return set_error(TTL_ERR_ARG, "%s: accumulate must be 0 or 1", name);
  const bool norm = gamma_q != nullptr;
  if (norm) {
    if (!dgamma_q || !dgamma_k) return set_error(TTL_ERR_ARG, "%s: dgamma is null", name);
    if ((reinterpret_cast<uintptr_t>(dgamma_q) | reinterpret_cast<uintptr_t>(dgamma_k)) & 3)
      return set_error(TTL_ERR_ALIGN, "%s: dgamma not 4-byte aligned", name);
  } else if (dgamma_q || dgamma_k) {
    return set_error(TTL_ERR_ARG, "%s: dgamma without gamma", name);
  }
  const int64_t qc = static_cast<int64_t>(A.heads[0]) * d, kc = static_cast<int64_t>(A.heads[1]) * d;
  const size_t need_ws = norm && T > 0 ? ttl_head_norm_rotary_bwd_workspace_size(t, T, n_q, n_kv, d) : 0;
  if (T > 0) {
    if ((rc = check_mats(dY_q, t, qc, lddyq, "the gradient of Q", name)) ||
        (rc = check_mats(dY_k, t, kc, lddyk, "the gradient of K", name)) ||
        (norm && ((rc = check_mats(Q, t, qc, ldq, "Q", name)) || (rc = check_mats(K, t, kc, ldk, "K", name)))) ||
        (rc = check_mats(dQ, t, qc, lddq, "dQ", name)) || (rc = check_mats(dK, t, kc, lddk, "dK", name)))
      return rc;
    if (need_ws) {
      if (!ws || ws_bytes < need_ws)
        return set_error(TTL_ERR_ARG, "%s: workspace of %zu bytes needed, %zu given", name, need_ws, ws_bytes);
      if (!aligned16(ws)) return set_error(TTL_ERR_ALIGN, "%s: workspace not 16-byte aligned", name);
    }
  }
  {
    Operand outs[5], ins[8];
    int no = 0, ni = 0;
    const int64_t w = d * (w_type == TTL_T_F32 ? 4 : 2);
    const void *pos = positions, *cu = cu_seqlens, *gq = dgamma_q, *gk = dgamma_k, *space = ws;
    if (T > 0) {
      outs[no++] = mats("dQ", dQ, t, T, lddq, qc);
      outs[no++] = mats("dK", dK, t, T, lddk, kc);
      if (!in_place(dY_q, lddyq, dQ, lddq, t)) ins[ni++] = mats("the gradient of Q", dY_q, t, T, lddyq, qc);
      if (!in_place(dY_k, lddyk, dK, lddk, t)) ins[ni++] = mats("the gradient of K", dY_k, t, T, lddyk, kc);
      if (norm) {
        ins[ni++] = mats("Q", Q, t, T, ldq, qc);
        ins[ni++] = mats("K", K, t, T, ldk, kc);
      }
      if (positions) ins[ni++] = operand("positions", &pos, 1, axes * T * 4);
      if (cu_seqlens) ins[ni++] = operand("cu_seqlens", &cu, 1, (int64_t(batch) + 1) * 4);
    }
    if (norm) {
      outs[no++] = operand("dgamma_q", &gq, 1, d * 4);
      outs[no++] = operand("dgamma_k", &gk, 1, d * 4);
      if (need_ws) outs[no++] = operand("the workspace", &space, 1, static_cast<int64_t>(need_ws));
      ins[ni++] = operand("gamma_q", &gamma_q, 1, w);
      ins[ni++] = operand("gamma_k", &gamma_k, 1, w);
    }
    if ((rc = check_alias(outs, no, ins, ni, name))) return rc;
  }
  if (T == 0 && (!norm || accumulate)) return TTL_OK;
  if ((rc = require_sm103())) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned grid = 0;
  if (T > 0) {
    A.status = device_status_ptr();
    if (!A.status) return TTL_ERR_CUDA;
    fill_mats(A, 0, dY_q, lddyq, dQ, lddq);
    fill_mats(A, 1, dY_k, lddyk, dK, lddk);
    cut_heads(A);
    if (!norm) {
      A.sign = -1.0f;
      const int64_t need = (A.items + kWarps - 1) / kWarps;
      grid = static_cast<unsigned>(need < (1 << 30) ? need : (1 << 30));
      return launch<kTurn>(A, interleaved, grid, s);
    }
    for (int i = 0; i < t; ++i) {
      A.x[0][i] = reinterpret_cast<const __nv_bfloat16*>(Q[i]);
      A.x[1][i] = reinterpret_cast<const __nv_bfloat16*>(K[i]);
    }
    A.ld_x[0] = ldq;
    A.ld_x[1] = ldk;
    A.part = static_cast<float*>(ws);
    grid = static_cast<unsigned>(blocks_of(A.items));
    if ((rc = launch<kBackward>(A, interleaved, grid, s))) return rc;
  }
  TraceScope trace(s, TTL_K_NORM, 0.0, 8.0 * d * grid);
  // (T = 0 has no kernel before it of its own)
  const unsigned cols = static_cast<unsigned>((2 * d + 31) / 32);
  const float* part = A.part;
  const int rows = static_cast<int>(grid);
  return cuda_check(grid ? launch_after(head_join_kernel, dim3(cols), 256, 0, s, part, rows, d, dgamma_q, dgamma_k, accumulate)
                         : launch_first(head_join_kernel, dim3(cols), 256, 0, s, part, rows, d, dgamma_q, dgamma_k, accumulate),
                    "head_join_kernel launch");
}
