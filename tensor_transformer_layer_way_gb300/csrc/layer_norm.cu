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

#include "ttl_device.cuh"
#include "ttl_internal.h"

namespace ttl {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormParts = 304;   // partial sums of the weight gradients: two per SM of a 152-SM part

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
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

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

// One row per CTA at a time, any width, stride and alignment; the row is read again for each step
// (from L1 / L2).
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_any_kernel(const __grid_constant__ NormFwd P) {
  __shared__ float red[kNormThreads / 32];
  for (int64_t row = blockIdx.x; row < P.total; row += gridDim.x) {
    const int i = static_cast<int>(row / P.rows);
    const int64_t k = row - i * P.rows;
    const T* x = static_cast<const T*>(P.x[i]) + k * P.ldx;
    const T* r = P.r[i] ? static_cast<const T*>(P.r[i]) + k * P.ldr : nullptr;
    T* s = r ? static_cast<T*>(P.s[i]) + k * P.h : nullptr;
    T* y = static_cast<T*>(P.y[i]) + k * P.h;
    auto at = [&](int64_t c) {
      return r ? to_f(from_f<T>(to_f(x[c]) + to_f(r[c]))) : to_f(x[c]);
    };
    float sum = 0.0f;
    for (int64_t c = threadIdx.x; c < P.h; c += kNormThreads) {
      const float v = at(c);
      if (s) s[c] = from_f<T>(v);
      sum += v;
    }
    const float mean = block_sum(sum, red) / static_cast<float>(P.h);
    float sq = 0.0f;
    for (int64_t c = threadIdx.x; c < P.h; c += kNormThreads) {
      const float v = at(c) - mean;
      sq = fmaf(v, v, sq);
    }
    const float rstd = 1.0f / sqrtf(block_sum(sq, red) / static_cast<float>(P.h) + P.eps);
    for (int64_t c = threadIdx.x; c < P.h; c += kNormThreads) {
      const float b = P.beta ? load_w(P.beta, P.wtype, c) : 0.0f;
      y[c] = from_f<T>(fmaf((at(c) - mean) * rstd, load_w(P.gamma, P.wtype, c), b));
    }
    if (threadIdx.x == 0) {
      P.mean[i][k] = mean;
      P.rstd[i][k] = rstd;
    }
  }
}

// The same for the backward pass.  CTA b takes rows b, b + grid, ...; each thread owns its columns'
// partial sums of dgamma and dbeta, in the CTA's slice of the workspace.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_any_kernel(const __grid_constant__ NormBwd P) {
  __shared__ float red[kNormThreads / 32];
  float* pg = P.part + static_cast<int64_t>(blockIdx.x) * 2 * P.h;
  float* pb = pg + P.h;
  for (int64_t c = threadIdx.x; c < P.h; c += kNormThreads) pg[c] = pb[c] = 0.0f;
  for (int64_t row = blockIdx.x; row < P.total; row += gridDim.x) {
    const int i = static_cast<int>(row / P.rows);
    const int64_t k = row - i * P.rows;
    const T* x = static_cast<const T*>(P.x[i]) + k * P.ldx;
    const T* dy = static_cast<const T*>(P.dy[i]) + k * P.lddy;
    const T* ds = P.ds[i] ? static_cast<const T*>(P.ds[i]) + k * P.ldds : nullptr;
    T* dx = static_cast<T*>(P.dx[i]) + k * P.h;
    const float mean = P.mean[i][k], rstd = P.rstd[i][k];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < P.h; c += kNormThreads) {
      const float d = to_f(dy[c]), xh = (to_f(x[c]) - mean) * rstd;
      const float g = d * load_w(P.gamma, P.wtype, c);
      s1 += g;
      s2 = fmaf(g, xh, s2);
      pg[c] = fmaf(d, xh, pg[c]);
      pb[c] += d;
    }
    const float c1 = block_sum(s1, red) / static_cast<float>(P.h);
    const float c2 = block_sum(s2, red) / static_cast<float>(P.h);
    for (int64_t c = threadIdx.x; c < P.h; c += kNormThreads) {
      const float xh = (to_f(x[c]) - mean) * rstd;
      const float g = to_f(dy[c]) * load_w(P.gamma, P.wtype, c);
      float v = rstd * (g - c1 - xh * c2);
      if (ds) v += to_f(ds[c]);
      dx[c] = from_f<T>(v);
    }
  }
}

// dgamma and dbeta: the partial sums joined in the order of the CTAs.  One warp per 32 columns of
// one of the two, eight warps of a CTA each taking every eighth part.
__global__ void __launch_bounds__(256) norm_join_kernel(const float* part, int nparts, int64_t h, float* dgamma,
                                                        float* dbeta, int accumulate) {
  __shared__ float red[8][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  float s = 0.0f;
  if (c < h)
    for (int p = w; p < nparts; p += 8) s += part[(static_cast<int64_t>(p) * 2 + blockIdx.y) * h + c];
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < h) {
    float v = red[0][lane];
#pragma unroll
    for (int j = 1; j < 8; ++j) v += red[j][lane];
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

// Rows [rows, h] with stride ld at a and at b share memory.
bool overlap(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t rows, int64_t h, int bytes) {
  const char* p = static_cast<const char*>(a);
  const char* q = static_cast<const char*>(b);
  return p < q + ((rows - 1) * ldb + h) * bytes && q < p + ((rows - 1) * lda + h) * bytes;
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
  for (int i = 0; i < t; ++i)
    for (int o = 0; o < t; ++o)
      if (overlap(X[i], ldx, Y[o], h, rows, h, xb) || (R && overlap(R[i], ldr, Y[o], h, rows, h, xb)) ||
          (S && (overlap(X[i], ldx, S[o], h, rows, h, xb) || overlap(R[i], ldr, S[o], h, rows, h, xb) ||
                 overlap(S[i], h, Y[o], h, rows, h, xb))))
        return set_error(TTL_ERR_ARG, "%s: an output aliases an input or another output", name);
  if ((rc = require_sm103())) return rc;
  NormFwd P = {};
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
  const int64_t cap = static_cast<int64_t>(num_sms()) * 8;
  const unsigned grid = static_cast<unsigned>(P.total < cap ? P.total : cap);
  if (x_type == TTL_T_F32)
    norm_fwd_any_kernel<float><<<grid, kNormThreads, 0, s>>>(P);
  else
    norm_fwd_any_kernel<__nv_bfloat16><<<grid, kNormThreads, 0, s>>>(P);
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
    for (int i = 0; i < t; ++i)
      for (int o = 0; o < t; ++o)
        if (overlap(X[i], ldx, dX[o], h, rows, h, xb) || overlap(dY[i], lddy, dX[o], h, rows, h, xb) ||
            (dS && overlap(dS[i], ldds, dX[o], h, rows, h, xb)))
          return set_error(TTL_ERR_ARG, "%s: dX aliases an input", name);
    const size_t need = ttl_layer_norm_bwd_workspace_size(t, rows, h);
    if (!ws || ws_bytes < need)
      return set_error(TTL_ERR_ARG, "%s: workspace of %zu bytes needed, %zu given", name, need, ws_bytes);
    if (!aligned16(ws)) return set_error(TTL_ERR_ALIGN, "%s: workspace not 16-byte aligned", name);
  }
  if (rows == 0 && accumulate) return TTL_OK;
  if ((rc = require_sm103())) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int parts = 0;
  if (rows > 0) {
    NormBwd P = {};
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
    if (x_type == TTL_T_F32)
      norm_bwd_any_kernel<float><<<parts, kNormThreads, 0, s>>>(P);
    else
      norm_bwd_any_kernel<__nv_bfloat16><<<parts, kNormThreads, 0, s>>>(P);
    if ((rc = cuda_check(cudaGetLastError(), "layer norm backward launch"))) return rc;
  }
  TraceScope trace(s, TTL_K_NORM, 0.0, 8.0 * h * parts);
  norm_join_kernel<<<dim3(static_cast<unsigned>((h + 31) / 32), 2), 256, 0, s>>>(static_cast<const float*>(ws), parts,
                                                                                 h, dgamma, dbeta, accumulate);
  return cuda_check(cudaGetLastError(), "norm_join_kernel launch");
}
