// Scaled vocab-parallel embedding lookup, and its table gradient summed by sorted tokens.
//
// Source: "v4:Tensor Parallel 与 Sequence Parallel", section "Embedding 和 LM head:按 vocab 切":
// shard i owns ids [i V/t, (i+1) V/t) and after the all-reduce every shard has every token's row.
//
// Forward:   out[tok] = bf16(scale E[id(tok)]), one rounding, into all t buffers.
// Backward:  dE[v] (+)= scale sum over the tokens of id v of dY[tok], in fp32.
// The token indices are sorted by id (a stable radix sort, so the tokens of one id stay in
// token order); a run of equal ids is then summed by whole CTAs in chunks of fixed length, and the
// partial sums of a run that crosses chunks are joined in chunk order.  No atomic adds: the same
// inputs give the same bits, and a row of the gradient is written once.

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
__global__ void __launch_bounds__(1024) sort_scan_kernel(uint32_t* counts, int64_t n) {
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

// ------------------------------------------------------------------ sums over runs of equal ids

constexpr int kSumThreads = 256;

__device__ __forceinline__ void row_out(const GradTables& G, uint32_t key, int64_t Vs, int64_t h, int64_t col,
                                        const float (&a)[8], float scale, int accumulate) {
  const int i = static_cast<int>(key / Vs);
  float4* dst = reinterpret_cast<float4*>(G.g[i] + (key - i * Vs) * h + col);
  float4 u = make_float4(a[0] * scale, a[1] * scale, a[2] * scale, a[3] * scale);
  float4 v = make_float4(a[4] * scale, a[5] * scale, a[6] * scale, a[7] * scale);
  if (accumulate) {
    const float4 p = dst[0], q = dst[1];
    u = make_float4(u.x + p.x, u.y + p.y, u.z + p.z, u.w + p.w);
    v = make_float4(v.x + q.x, v.y + q.y, v.z + q.z, v.w + q.w);
  }
  dst[0] = u;
  dst[1] = v;
}

// Chunk b = sorted places [b C, (b + 1) C); each thread sums 8 columns.  A run that begins and ends in
// the chunk goes to its row of dE.  A run that began earlier leaves its sum in head[b]; one that
// begins here and goes on leaves its sum in tail[b].
__global__ void __launch_bounds__(kSumThreads) embed_sum_kernel(const __grid_constant__ GradTables G,
                                                                const uint32_t* keys, const uint32_t* toks,
                                                                const __nv_bfloat16* dY, int64_t lddy, int64_t T,
                                                                int64_t h, int64_t Vs, int64_t V, int C, float scale,
                                                                int accumulate, float* head, float* tail) {
  const int64_t col = (static_cast<int64_t>(blockIdx.y) * kSumThreads + threadIdx.x) * 8;
  if (col >= h) return;
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * C, hi = lo + C < T ? lo + C : T;
  float a[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) a[j] = 0.0f;
  bool began = lo == 0 || keys[lo - 1] != keys[lo];
  for (int64_t k = lo; k < hi; ++k) {
    const uint32_t key = keys[k];
    if (key >= V) break;   // ids out of range are last
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(dY + static_cast<int64_t>(toks[k]) * lddy + col));
    a[0] += bf16_lo(v.x); a[1] += bf16_hi(v.x); a[2] += bf16_lo(v.y); a[3] += bf16_hi(v.y);
    a[4] += bf16_lo(v.z); a[5] += bf16_hi(v.z); a[6] += bf16_lo(v.w); a[7] += bf16_hi(v.w);
    const bool ends = k + 1 == T || keys[k + 1] != key;
    if (ends || k + 1 == hi) {
      if (began && ends) {
        row_out(G, key, Vs, h, col, a, scale, accumulate);
      } else {
        float4* p = reinterpret_cast<float4*>((began ? tail : head) + static_cast<int64_t>(blockIdx.x) * h + col);
        p[0] = make_float4(a[0], a[1], a[2], a[3]);
        p[1] = make_float4(a[4], a[5], a[6], a[7]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = 0.0f;
      began = true;
    }
  }
}

// Joins the runs that go on past their chunk: the chunk in which the run began adds the heads of the
// following ones, in order.
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(const __grid_constant__ GradTables G,
                                                                 const uint32_t* keys, int64_t T, int64_t h,
                                                                 int64_t Vs, int64_t V, int C, float scale,
                                                                 int accumulate, const float* head, const float* tail) {
  const int64_t b = blockIdx.x, lo = b * C, hi = lo + C;
  if (hi >= T) return;                                     // the last chunk goes on nowhere
  const uint32_t key = keys[hi - 1];
  if (key >= V || keys[hi] != key) return;                 // ends with the chunk
  if (keys[lo] == key && lo > 0 && keys[lo - 1] == key) return;   // began in an earlier chunk
  const int64_t col = (static_cast<int64_t>(blockIdx.y) * kSumThreads + threadIdx.x) * 8;
  if (col >= h) return;
  float a[8];
  auto add = [&](const float* p, bool first) {
    const float4 u = reinterpret_cast<const float4*>(p)[0], v = reinterpret_cast<const float4*>(p)[1];
    const float w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = first ? w[j] : a[j] + w[j];
  };
  add(tail + b * h + col, true);
  for (int64_t n = b + 1; n * C < T && keys[n * C] == key; ++n) add(head + n * h + col, false);
  row_out(G, key, Vs, h, col, a, scale, accumulate);
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

struct SortPlan {
  int64_t nb;        // sort blocks
  int C;             // sorted places per sum chunk
  int64_t chunks;
  size_t keys, counts, part;   // bytes of one key array, of the counts, of one partial array
};

// A chunk is 32 places, or longer so that there are at most 2048 of them: a run of any length is
// then joined from at most 2048 partial sums.
SortPlan plan_of(int64_t T, int64_t h) {
  SortPlan p;
  p.nb = (T + kSortBlock - 1) / kSortBlock;
  int64_t C = 32;
  while ((T + C - 1) / C > 2048) C *= 2;
  p.C = static_cast<int>(C);
  p.chunks = (T + C - 1) / C;
  p.keys = round256(static_cast<size_t>(T) * 4);
  p.counts = round256(static_cast<size_t>(kRadix) * p.nb * 4);
  p.part = round256(static_cast<size_t>(p.chunks) * h * 4);
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
  return 4 * p.keys + p.counts + 2 * p.part;
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
  if ((rc = require_sm103())) return rc;
  int* status = device_status_ptr();
  if (!status) return TTL_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t Vs = V / t;
  GradTables G = {};
  for (int i = 0; i < t; ++i) G.g[i] = dE[i];
  if (!accumulate) {
    TraceScope trace(s, TTL_K_OTHER, 0.0, 4.0 * V * h);
    for (int i = 0; i < t; ++i)
      if ((rc = fill_zero(dE[i], static_cast<size_t>(Vs) * h * 4, s))) return rc;
  }
  if (T == 0) return TTL_OK;

  const SortPlan p = plan_of(T, h);
  char* base = static_cast<char*>(ws);
  uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(base), reinterpret_cast<uint32_t*>(base + p.keys)};
  uint32_t* toks[2] = {reinterpret_cast<uint32_t*>(base + 2 * p.keys), reinterpret_cast<uint32_t*>(base + 3 * p.keys)};
  uint32_t* counts = reinterpret_cast<uint32_t*>(base + 4 * p.keys);
  float* head = reinterpret_cast<float*>(base + 4 * p.keys + p.counts);
  float* tail = reinterpret_cast<float*>(base + 4 * p.keys + p.counts + p.part);
  const uint32_t* k_in = nullptr;
  const uint32_t* t_in = nullptr;
  {
    TraceScope trace(s, TTL_K_EMBED, 0.0, 16.0 * T);
    int out = 0;
    for (int shift = 0; shift < 32 && (shift == 0 || (V >> shift) > 0); shift += 8) {   // V itself is a key
      sort_count_kernel<<<static_cast<unsigned>(p.nb), kSortThreads, 0, s>>>(ids, k_in, T, V, shift, counts,
                                                                             static_cast<int>(p.nb), status);
      sort_scan_kernel<<<1, 1024, 0, s>>>(counts, kRadix * p.nb);
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
  embed_sum_kernel<<<grid, kSumThreads, 0, s>>>(G, k_in, t_in, reinterpret_cast<const __nv_bfloat16*>(dY), lddy, T, h,
                                                Vs, V, p.C, scale, accumulate, head, tail);
  embed_join_kernel<<<grid, kSumThreads, 0, s>>>(G, k_in, T, h, Vs, V, p.C, scale, accumulate, head, tail);
  return cuda_check(cudaGetLastError(), "embedding gradient launch");
}
