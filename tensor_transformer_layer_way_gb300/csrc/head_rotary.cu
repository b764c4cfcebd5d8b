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
// gives turns per position as a 64-bit fraction of a turn, to 2^-64; the integer product with the position wraps at whole turns
// by itself, for positions of either sign, and its upper 32 bits are the angle to 2^-31 turns.
//
// Layout.  A lane holds 16 columns of a head as two 16-byte words whose columns pair up (columns c.. and rot/2 + c..,
// or 16 neighbours), so a rotation exchanges nothing; the 1 to 16 lanes of a head share a token and join their squares
// by shuffles.  A warp walks over an even share of all (token group, head) pairs, a group's heads of all shards in turn:
// sines are taken once for a group.  A lane copies its words to a ring in shared memory, places ahead, and
// reads there what it copied itself: no barrier, and the copies' depth costs no registers.  The arithmetic is on pairs
// of values.
//
// What bounds it: bytes, of which it moves 86% (forward) and 80% (backward) of what a plain copy of as many does.
// Measured: 8192 tokens, 32 and 8 heads of 128 over 8 shards, forward 33 us (5.0 TB/s; one head's words a lane at a time
// through registers took 51), backward with the weights' gradients 51 us, 4 of them the join of the blocks' sums (alone on an idle
// card it takes 6.6).  A
// look-up of a token's document in memory cost each token group microseconds: the bounds are in shared memory.

#include <cmath>
#include <type_traits>

#include "head_deal.h"
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
constexpr int kNearDocs = 512;   // document bounds that a block keeps in shared memory
constexpr int kWarps = kHeadWarps;

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
  float sign;                                // -1: the turns go back
  float* part;                               // kBackward: [blocks][2][d]
  int64_t groups;                            // of the tokens that a warp works on together
  int64_t warps;                             // that share the pairs of a group and a head
  int* status;
};

// Eight pairs (a, b), two of them to a register pair: a[i] holds the a of pairs 2 i and 2 i + 1.
struct Pairs {
  uint64_t a[4], b[4];
};
__device__ __forceinline__ uint64_t widen(uint32_t w) { return f2_pack(bf16_lo(w), bf16_hi(w)); }
// The 16 columns of two words.
template <bool NEIGHBOURS>
__device__ __forceinline__ Pairs to_pairs(const uint4& u, const uint4& v) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  Pairs p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (NEIGHBOURS) {
      p.a[i] = f2_pack(bf16_lo(w[2 * i]), bf16_lo(w[2 * i + 1]));
      p.b[i] = f2_pack(bf16_hi(w[2 * i]), bf16_hi(w[2 * i + 1]));
    } else {
      p.a[i] = widen(w[i]);
      p.b[i] = widen(w[4 + i]);
    }
  }
  return p;
}
template <bool NEIGHBOURS>
__device__ __forceinline__ void to_words(const Pairs& p, uint4& u, uint4& v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = f2_unpack(p.a[i]), b = f2_unpack(p.b[i]);
    if constexpr (NEIGHBOURS) {
      w[2 * i] = pack_bf16x2(a.x, b.x);
      w[2 * i + 1] = pack_bf16x2(a.y, b.y);
    } else {
      w[i] = pack_bf16x2(a.x, a.y);
      w[4 + i] = pack_bf16x2(b.x, b.y);
    }
  }
  u = make_uint4(w[0], w[1], w[2], w[3]);
  v = make_uint4(w[4], w[5], w[6], w[7]);
}
// Sum of the lanes of a head.
template <int LANES>
__device__ __forceinline__ float head_sum(uint64_t x) {
  const float2 f = f2_unpack(x);
  float s = f.x + f.y;
#pragma unroll
  for (int o = LANES >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// cos and sin of two angles, given as fractions of a turn in units of 2^-32: Taylor's series about the nearest quarter turn
// (|x| <= pi / 4: up to x^9 for the sine, x^8 for the cosine, whose next terms are below 2^-29 and 2^-25).
__device__ __forceinline__ void turn_of(uint32_t f0, uint32_t f1, float (&c)[2], float (&s)[2]) {
  const uint32_t q[2] = {(f0 + 0x20000000u) >> 30, (f1 + 0x20000000u) >> 30};
  const float unit = 1.4629180792671596e-9f;      // 2 pi / 2^32
  const float x0 = static_cast<float>(static_cast<int32_t>(f0 - (q[0] << 30))) * unit;
  const float x1 = static_cast<float>(static_cast<int32_t>(f1 - (q[1] << 30))) * unit;
  auto both = [](float v) { return f2_pack(v, v); };
  const uint64_t x = f2_pack(x0, x1), x2 = fmul2(x, x);
  uint64_t p = ffma2(x2, both(1.0f / 362880.0f), both(-1.0f / 5040.0f));
  p = ffma2(p, x2, both(1.0f / 120.0f));
  p = ffma2(p, x2, both(-1.0f / 6.0f));
  const float2 sn = f2_unpack(ffma2(fmul2(p, x2), x, x));
  p = ffma2(x2, both(1.0f / 40320.0f), both(-1.0f / 720.0f));
  p = ffma2(p, x2, both(1.0f / 24.0f));
  p = ffma2(p, x2, both(-0.5f));
  const float2 cs = f2_unpack(ffma2(p, x2, both(1.0f)));
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float sv = u ? sn.y : sn.x, cv = u ? cs.y : cs.x;
    const float ps = q[u] & 1 ? cv : sv, pc = q[u] & 1 ? sv : cv;
    s[u] = __uint_as_float(__float_as_uint(ps) ^ ((q[u] & 2u) << 30));
    c[u] = __uint_as_float(__float_as_uint(pc) ^ (((q[u] + 1) & 2u) << 30));
  }
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

// 16 bytes to shared memory, in the group that the thread commits next.
__device__ __forceinline__ void copy16(void* dst, const __nv_bfloat16* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void await_copies() {   // all but the last N groups
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Places of a warp's ring: all but one of them hold heads on their way.  Blocks of an SM: with three (80 registers a thread) the
// forward kernel spilled and took 37 us where two take 33; the backward kernel's one, whose sums leave half as many
// rows to join, 51 where two took 53.  (8192 tokens, 40 heads of 128.)
template <int MODE>
constexpr int kStages = MODE == kBackward ? 4 : 5;
template <int MODE>
constexpr int kResident = MODE == kBackward ? 1 : 2;
template <int MODE>
constexpr int kWords = MODE == kBackward ? 4 : 2;   // of a lane and head
template <int MODE>
constexpr int kRingBytes = kWarps * kStages<MODE> * kWords<MODE> * 512;

// LANES lanes to a head, each with two words of eight columns.
template <int LANES, bool NEIGHBOURS, int MODE>
__global__ void __launch_bounds__(kWarps * 32, kResident<MODE>) head_rotary_kernel(const __grid_constant__ HeadArgs A) {
  constexpr int kTokens = 32 / LANES, S = kStages<MODE>;
  extern __shared__ __align__(16) uint4 ring[];   // [warp][stage][word][lane]: a lane reads what it copied
  __shared__ __align__(16) uint64_t turns[kMaxPairs];
  __shared__ __align__(8) uint8_t axis[kMaxPairs];
  __shared__ int32_t bounds[kNearDocs + 1];       // (looked up in memory they cost each token group a few microseconds)
  __shared__ __align__(16) float gamma[MODE == kTurn ? 1 : 2][kMaxHead];
  __shared__ float sums[MODE == kBackward ? kWarps : 1][2][kMaxHead];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if constexpr (MODE == kBackward) launch_next();   // (the join, which waits for all of this kernel)
  uint4* mine_at = ring + warp * (S * kWords<MODE> * 32) + lane;
  for (int i = threadIdx.x; i < kMaxPairs; i += kWarps * 32) {
    turns[i] = A.turns[i];                        // (0 behind the rotated columns' pairs: no turn)
    axis[i] = A.axis[i];
  }
  const bool near = A.cu && A.batch <= kNearDocs;
  if (near) {
    for (int i = threadIdx.x; i <= A.batch; i += kWarps * 32) bounds[i] = __ldg(A.cu + i);
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
  const bool turns_here = slot < A.rot / 16;
  int c0 = slot * 16, step = 8;
  if (!NEIGHBOURS && turns_here) {
    c0 = slot * 8;
    step = A.rot / 2;
  }
  auto column = [&](bool second, int e) { return NEIGHBOURS ? c0 + 2 * e + second : c0 + e + (second ? step : 0); };
  if (!mine) {                                    // idle lanes read zeros, which their heads' sums take in
    for (int k = 0; k < S * kWords<MODE>; ++k) mine_at[k * 32] = make_uint4(0, 0, 0, 0);
  }
  const float inv_d = 1.0f / static_cast<float>(A.d);
  const int q_heads = A.t * A.heads[0], all = q_heads + A.t * A.heads[1];
  Pairs acc[2];
  if constexpr (MODE == kBackward) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[0].a[i] = acc[0].b[i] = acc[1].a[i] = acc[1].b[i] = 0;
  }

  // The warp's share of all (token group, head) pairs: a group's heads of Q, shard by shard, then those of K.
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t total = A.groups * all, share = total / A.warps, more = total - share * A.warps;
  // (an int: the results, 32 bytes a pair at least, share no memory, and a launch of many pairs has thousands of warps)
  int left = w < A.warps ? static_cast<int>(share + (w < more)) : 0;
  const int64_t from = w < A.warps ? w * share + (w < more ? w : more) : 0;
  const int64_t group = from / all;
  int h0 = static_cast<int>(from - group * all);
  int tok = static_cast<int>(group) * kTokens + lane / LANES;
  // Shard of head h of Q (kind 0) or K, counted from the kind's first; h becomes the head on the shard.
  auto shard_of = [&](int kind, int& h) {
    const int shard = A.magic[kind] ? static_cast<int>(__umulhi(static_cast<uint32_t>(h), A.magic[kind])) : h;
    h -= shard * A.heads[kind];
    return shard;
  };
  // What is fetched next: head `f_head` of shard f_shard, at f_in (and f_x), f_left of them in all.
  int f_left = left, f_tok = tok;
  int f_kind = h0 >= q_heads, f_head = f_kind ? h0 - q_heads : h0, f_shard = shard_of(f_kind, f_head);
  int put = 0, get = 0;                           // places of the ring
  const __nv_bfloat16 *f_in, *f_x;
  auto locate = [&]() {
    f_in = A.in[f_kind][f_shard] + static_cast<int64_t>(f_tok) * A.ld_in[f_kind] + f_head * A.d + c0;
    if constexpr (MODE == kBackward) f_x = A.x[f_kind][f_shard] + static_cast<int64_t>(f_tok) * A.ld_x[f_kind] + f_head * A.d + c0;
  };
  locate();
  auto fetch = [&]() {
    if (f_left > 0) {
      uint4* to = mine_at + put * (kWords<MODE> * 32);
      if (mine && f_tok < A.T) {
        copy16(to, f_in);
        copy16(to + 32, f_in + step);
        if constexpr (MODE == kBackward) {
          copy16(to + 64, f_x);
          copy16(to + 96, f_x + step);
        }
      }
      --f_left;
      put = put + 1 == S ? 0 : put + 1;
      f_in += A.d;
      if constexpr (MODE == kBackward) f_x += A.d;
      if (++f_head == A.heads[f_kind]) {
        f_head = 0;
        if (++f_shard == A.t) {
          f_shard = 0;
          f_kind ^= 1;
          if (f_kind == 0) f_tok += kTokens;
        }
        locate();
      }
    }
    commit_copies();
  };
#pragma unroll
  for (int k = 0; k < S - 1; ++k) fetch();

  for (; left > 0; tok += kTokens, h0 = 0) {
    const int h1 = left < all - h0 ? h0 + left : all;
    left -= h1 - h0;
    const bool there = tok < A.T;
    DocRange doc{0, static_cast<int>(A.T)};
    if (near) doc = doc_among([&](int b) { return bounds[b]; }, A.batch, static_cast<int>(A.T), there ? tok : -1);
    else if (A.cu) doc = doc_of(A.cu, A.batch, static_cast<int>(A.T), there ? tok : -1);
    const bool counts = there && doc.hi > doc.lo;
    const bool all_count = __all_sync(0xffffffffu, counts);
    uint64_t co[4], si[4];
    {
      const uint2 on = *reinterpret_cast<const uint2*>(axis + slot * 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const ulonglong2 per = *reinterpret_cast<const ulonglong2*>(turns + slot * 8 + i * 2);
        const uint32_t two = ((i & 2) ? on.y : on.x) >> ((i & 1) * 16);
        int p[2] = {tok - doc.lo, tok - doc.lo};
        if (A.pos) {
          p[0] = counts ? __ldg(A.pos + (two & 255u) * A.T + tok) : 0;
          p[1] = counts ? __ldg(A.pos + (two >> 8 & 255u) * A.T + tok) : 0;
        }
        float c[2], s[2];
        turn_of(static_cast<uint32_t>((per.x * static_cast<uint64_t>(static_cast<int64_t>(p[0]))) >> 32),
                static_cast<uint32_t>((per.y * static_cast<uint64_t>(static_cast<int64_t>(p[1]))) >> 32), c, s);
        co[i] = f2_pack(c[0], c[1]);
        si[i] = f2_pack(s[0] * A.sign, s[1] * A.sign);
      }
    }
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      int at = kind ? (h0 > q_heads ? h0 - q_heads : 0) : h0;
      int n = (kind ? h1 - q_heads : (h1 < q_heads ? h1 : q_heads)) - at;   // heads of this kind
      if (n <= 0) continue;
      Pairs ga;
      if constexpr (MODE != kTurn) {
        float g[16];                              // (idle lanes: 0, as of their zeros a weight that is infinite would make NaN)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(g + i * 4) =
              mine ? *reinterpret_cast<const float4*>(gamma[kind] + c0 + (i & 1) * 4 + (i >> 1) * step) : make_float4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ga.a[i] = NEIGHBOURS ? f2_pack(g[4 * i], g[4 * i + 2]) : f2_pack(g[2 * i], g[2 * i + 1]);
          ga.b[i] = NEIGHBOURS ? f2_pack(g[4 * i + 1], g[4 * i + 3]) : f2_pack(g[8 + 2 * i], g[8 + 2 * i + 1]);
        }
      }
      for (int shard = shard_of(kind, at); n > 0; ++shard, at = 0) {
        __nv_bfloat16* out = A.out[kind][shard] + static_cast<int64_t>(tok) * A.ld_out[kind] + at * A.d + c0;
        int here = A.heads[kind] - at;
        here = here < n ? here : n;
        n -= here;
        // (Two copies: from one, with the branch, heads that turn whole take 18.5 us in place of 17.5, 8192 tokens, 32 heads of 80.  The
        // backward pass does without the second: 51.5 us either way, and short ones 17.5 in place of 18.4.)
        auto walk = [&](auto whole) {
#pragma unroll 1
          for (; here > 0; --here, out += A.d) {
            const uint4* ring_at = mine_at + get * (kWords<MODE> * 32);
            get = get + 1 == S ? 0 : get + 1;
            await_copies<S - 2>();
            uint4 u = ring_at[0], v = ring_at[32];
            const bool hide = !all_count && !counts;
            if (MODE == kBackward && hide) u = v = make_uint4(0, 0, 0, 0);
            Pairs y = to_pairs<NEIGHBOURS>(u, v);
            if constexpr (MODE == kForward) {
              uint64_t ss = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) ss = ffma2(y.a[i], y.a[i], ffma2(y.b[i], y.b[i], ss));
              const float r = rsqrtf(fmaf(head_sum<LANES>(ss), inv_d, A.eps));
              const uint64_t r2 = f2_pack(r, r);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                y.a[i] = fmul2(fmul2(y.a[i], r2), ga.a[i]);
                y.b[i] = fmul2(fmul2(y.b[i], r2), ga.b[i]);
              }
            }
            // the turn (backward: A.sign turned it back); columns that stay are not turned by 0, which an infinite or NaN
            // neighbour would make NaN
            if (decltype(whole)::value || turns_here) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint64_t a = y.a[i], b = y.b[i];
                y.a[i] = ffma2(a, co[i], fmul2(b, si[i] ^ 0x8000000080000000ull));
                y.b[i] = ffma2(b, co[i], fmul2(a, si[i]));
              }
            }
            if constexpr (MODE == kBackward) {
              // y is g; with k = -r^2 mean(h n):  dx = (g r) gamma + x k,  dgamma += (g r) x
              u = ring_at[64];
              v = ring_at[96];
              if (hide) u = v = make_uint4(0, 0, 0, 0);
              const Pairs x = to_pairs<NEIGHBOURS>(u, v);
              uint64_t ss = 0, dot = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                ss = ffma2(x.a[i], x.a[i], ffma2(x.b[i], x.b[i], ss));
                dot = ffma2(fmul2(y.a[i], ga.a[i]), x.a[i], ffma2(fmul2(y.b[i], ga.b[i]), x.b[i], dot));
              }
              float r = rsqrtf(fmaf(head_sum<LANES>(ss), inv_d, A.eps));
              if (hide) r = 0.0f;
              const float k = -(head_sum<LANES>(dot) * inv_d) * r * r * r;
              const uint64_t r2 = f2_pack(r, r), k2 = f2_pack(k, k);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint64_t a = fmul2(y.a[i], r2), b = fmul2(y.b[i], r2);
                acc[kind].a[i] = ffma2(a, x.a[i], acc[kind].a[i]);
                acc[kind].b[i] = ffma2(b, x.b[i], acc[kind].b[i]);
                y.a[i] = ffma2(a, ga.a[i], fmul2(x.a[i], k2));
                y.b[i] = ffma2(b, ga.b[i], fmul2(x.b[i], k2));
              }
            }
            fetch();                                // (into the place that was read a head ago)
            to_words<NEIGHBOURS>(y, u, v);
            if (hide) u = v = make_uint4(0, 0, 0, 0);
            if (mine && there) {
              *reinterpret_cast<uint4*>(out) = u;
              *reinterpret_cast<uint4*>(out + step) = v;
            }
          }
        };
        if (MODE != kBackward && A.rot == A.d) walk(std::true_type{});
        else walk(std::false_type{});
      }
    }
  }

  if constexpr (MODE == kBackward) {
    // the block's sums: over the warp's tokens, then over its warps in their order
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float2 f = f2_unpack(i < 4 ? acc[kind].a[i] : acc[kind].b[i - 4]);
#pragma unroll
        for (int o = 16; o >= LANES; o >>= 1) {
          f.x += __shfl_xor_sync(0xffffffffu, f.x, o);
          f.y += __shfl_xor_sync(0xffffffffu, f.y, o);
        }
        if (lane < LANES && mine) {
          sums[warp][kind][column(i >= 4, i % 4 * 2)] = f.x;
          sums[warp][kind][column(i >= 4, i % 4 * 2 + 1)] = f.y;
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * A.d; i += kWarps * 32) {
      const int kind = i >= A.d, c = i - kind * A.d;
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) s += sums[k][kind][c];
      A.part[static_cast<int64_t>(blockIdx.x) * 2 * A.d + i] = s;
    }
  }
}

// dgamma from the blocks' sums: 32 columns a block, a warp on every 32nd row, the warps' sums in their order.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(kJoinWarps * 32) head_join_kernel(const float* part, int rows, int d, float* dq, float* dk,
                                                                     int accumulate) {
  __shared__ float sums[kJoinWarps][32];
  await_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < 2 * d) {
#pragma unroll 10
    for (int r = warp; r < rows; r += kJoinWarps) s += part[static_cast<int64_t>(r) * 2 * d + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < 2 * d) {
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) s += sums[w][lane];
    float* out = c < d ? dq + c : dk + (c - d);
    *out = accumulate ? *out + s : s;
  }
}

template <int MODE>
int launch(HeadArgs& A, bool neighbours, unsigned& grid, cudaStream_t s) {
  const HeadDeal deal = head_deal(A.T, static_cast<int64_t>(A.t) * (A.heads[0] + A.heads[1]), A.d, kResident<MODE>, num_sms());
  A.groups = deal.groups;
  A.warps = deal.warps;
  grid = deal.blocks;
  const double size = static_cast<double>(A.T) * A.t * (A.heads[0] + A.heads[1]) * A.d;
  TraceScope trace(s, TTL_K_NORM, 0.0, size * (MODE == kBackward ? 6.0 : 4.0));
  auto go = [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    auto run = [&](auto kernel) { return cuda_check(launch_first(kernel, dim3(grid), kWarps * 32, kRingBytes<MODE>, s, A), "head_rotary_kernel launch"); };
    const char* what = "cudaFuncSetAttribute(head rotation)";
    int rc = neighbours ? allow_smem<head_rotary_kernel<L, true, MODE>>(kRingBytes<MODE>, what)
                        : allow_smem<head_rotary_kernel<L, false, MODE>>(kRingBytes<MODE>, what);
    if (rc) return rc;
    return neighbours ? run(head_rotary_kernel<L, true, MODE>) : run(head_rotary_kernel<L, false, MODE>);
  };
  switch (head_lanes(A.d)) {
    case 1: return go(std::integral_constant<int, 1>{});
    case 2: return go(std::integral_constant<int, 2>{});
    case 4: return go(std::integral_constant<int, 4>{});
    case 8: return go(std::integral_constant<int, 8>{});
    default: return go(std::integral_constant<int, 16>{});
  }
}

int check_shape(int t, int64_t T, int n_q, int n_kv, int d, const char* name) {
  if (t < 1 || t > kMaxShards) return set_error(TTL_ERR_ARG, "%s: t=%d outside [1,%d]", name, t, kMaxShards);
  if (T < 0 || n_q < 1 || n_kv < 1 || d < 1) return set_error(TTL_ERR_ARG, "%s: bad shape", name);
  if (n_q % t || n_kv % t)
    return set_error(TTL_ERR_SHAPE, "%s: t=%d must divide the head counts %d and %d", name, t, n_q, n_kv);
  if (d % 16 || d > kMaxHead)
    return set_error(TTL_ERR_SHAPE, "%s: head dimension %d is not a multiple of 16 up to %d", name, d, kMaxHead);
  if (T >= (int64_t(1) << 31) - 64 || n_q > 32768 || n_kv > 32768) return set_error(TTL_ERR_SHAPE, "%s: extent too large", name);
  return TTL_OK;
}

// f / 2 pi without its whole turns, in units of 2^-64 turns, to one of them (0 <= f <= 2^20): a position of 2^31 leaves
// 2^-33 turns of that.  The quotient in doubles alone is off by up to 2^-36 turns, which such a position makes a thirtieth
// of a turn; so the division's remainder is divided too, by 2 pi as a sum of two doubles.
uint64_t turns_of(double f) {
  constexpr double kTwoPi = 0x1.921fb54442d18p+2, kTwoPiRest = 0x1.1a62633145c07p-52;
  const double q = f / kTwoPi;
  const double rest = std::fma(-q, kTwoPiRest, std::fma(-q, kTwoPi, f)) / kTwoPi;   // (the inner one is exact)
  const double fraction = q - static_cast<double>(static_cast<int64_t>(q));
  // (2^64; the first product is exact but for what lies below a unit)
  return static_cast<uint64_t>(fraction * 18446744073709551616.0) + static_cast<uint64_t>(std::llrint(rest * 18446744073709551616.0));
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
    const uint64_t part = turns_of(std::fabs(freqs[i]));
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
  unsigned grid;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return gamma_q ? launch<kForward>(A, interleaved, grid, s) : launch<kTurn>(A, interleaved, grid, s);
}

extern "C" size_t ttl_head_norm_rotary_bwd_workspace_size(int t, int64_t T, int n_q, int n_kv, int d) {
  if (check_shape(t, T, n_q, n_kv, d, "ttl_head_norm_rotary_bwd_workspace_size")) return 0;
  return static_cast<size_t>(kResident<kBackward> * kHeadMostSms) * 2 * d * 4;
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
    A.sign = -1.0f;
    if (!norm) {
      return launch<kTurn>(A, interleaved, grid, s);
    }
    for (int i = 0; i < t; ++i) {
      A.x[0][i] = reinterpret_cast<const __nv_bfloat16*>(Q[i]);
      A.x[1][i] = reinterpret_cast<const __nv_bfloat16*>(K[i]);
    }
    A.ld_x[0] = ldq;
    A.ld_x[1] = ldk;
    A.part = static_cast<float*>(ws);
    if ((rc = launch<kBackward>(A, interleaved, grid, s))) return rc;
  }
  TraceScope trace(s, TTL_K_NORM, 0.0, 8.0 * d * grid);
  // (T = 0 has no kernel before it of its own)
  const unsigned cols = static_cast<unsigned>((2 * d + 31) / 32);
  const float* part = A.part;
  const int rows = static_cast<int>(grid);
  return cuda_check(grid ? launch_after(head_join_kernel, dim3(cols), kJoinWarps * 32, 0, s, part, rows, d, dgamma_q, dgamma_k, accumulate)
                         : launch_first(head_join_kernel, dim3(cols), kJoinWarps * 32, 0, s, part, rows, d, dgamma_q, dgamma_k, accumulate),
                    "head_join_kernel launch");
}
