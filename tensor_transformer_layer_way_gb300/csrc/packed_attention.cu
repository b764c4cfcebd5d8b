// Causal attention with grouped heads over a pack of documents, heads split across t shards.
//
// Source: "v4:Tensor Parallel 与 Sequence Parallel", section "Attention:按 head 切": each shard
// finishes its own heads alone.  ttl_tp_attn_fwd computes one sequence and keeps the probabilities
// (T^2 per head); here T tokens hold any number of documents, nothing of size T^2 reaches memory,
// and the backward pass recomputes the probabilities from each row's log-sum-exp.
//
// For the query at token i of a document that starts at lo, head c reading KV head g = c / grp:
//   s_j = scale q_i . k_j,  lse_i = log sum_{lo <= j <= i} exp(s_j),  p_j = exp(s_j - lse_i)
//   o_i = sum_j p_j v_j
//   D_i = do_i . o_i,  ds_j = p_j (do_i . v_j - D_i)
//   dq_i = scale sum_j ds_j k_j,  dk_j = scale sum_{c, i} ds_j q_i,  dv_j = sum_{c, i} p_j do_i
// A token of no document has o = 0, lse = -inf and zero gradients.

#include "operands.h"
#include "packed_attn.cuh"

namespace ttl {
namespace {

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

int check_shape(int t, int64_t T, int n_q, int n_kv, int d, int batch, const char* name) {
  if (t < 1 || t > kMaxShards) return set_error(TTL_ERR_ARG, "%s: t=%d outside [1,%d]", name, t, kMaxShards);
  if (T < 0 || n_q < 1 || n_kv < 1 || d < 1 || batch < 0) return set_error(TTL_ERR_ARG, "%s: bad shape", name);
  if (n_q % t || n_kv % t)
    return set_error(TTL_ERR_SHAPE, "%s: t=%d must divide the head counts %d and %d", name, t, n_q, n_kv);
  if (n_q % n_kv) return set_error(TTL_ERR_SHAPE, "%s: n_kv=%d must divide n_q=%d", name, n_kv, n_q);
  if (d != 64 && d != 128) return set_error(TTL_ERR_SHAPE, "%s: head dimension %d is not 64 or 128", name, d);
  if (T >= (int64_t(1) << 28) || n_q > 32768) return set_error(TTL_ERR_SHAPE, "%s: extent too large", name);
  return TTL_OK;
}

// t matrices [T, cols] with row stride ld, 16-byte rows.
int check_mats(const void* const* a, int t, int64_t cols, int64_t ld, const char* what, const char* name) {
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

int check_lse(const float* const* lse, int t, const char* name) {
  if (!lse) return set_error(TTL_ERR_ARG, "%s: lse: null shard array", name);
  for (int i = 0; i < t; ++i) {
    if (!lse[i]) return set_error(TTL_ERR_ARG, "%s: lse[%d] is null", name, i);
    if (reinterpret_cast<uintptr_t>(lse[i]) & 3) return set_error(TTL_ERR_ALIGN, "%s: lse[%d] not 4-byte aligned", name, i);
  }
  return TTL_OK;
}

int check_cu(const int32_t* cu, float scale, const char* name) {
  if (!cu) return set_error(TTL_ERR_ARG, "%s: cu_seqlens is null", name);
  if (reinterpret_cast<uintptr_t>(cu) & 3) return set_error(TTL_ERR_ALIGN, "%s: cu_seqlens not 4-byte aligned", name);
  if (!(scale > 0.0f && scale < INFINITY)) return set_error(TTL_ERR_ARG, "%s: scale must be positive and finite", name);
  return TTL_OK;
}

int64_t tiles_of(int64_t T) { return (T + kTile - 1) / kTile; }

// Room to list the rows that are computed again: of every query head, or of dK and dV of every KV head.
size_t redo_bytes(int64_t T, int heads) { return static_cast<size_t>(heads) * tiles_of(T) * 4 * sizeof(RedoEntry); }

// Forward workspace: the query tiles by work and how many were taken, and the rows that are computed again.
size_t fwd_list_bytes(int64_t T) { return round256(static_cast<size_t>(tiles_of(T) + 1) * 16); }

// Backward workspace: D, the query tiles by work, the key items by work with their counts, the key tiles that
// several items share, those items' partial sums, and the rows that are computed again.
struct BwdWs {
  size_t q_list, kv_list, head, join, part, redo, total;   // offsets after D
};
BwdWs bwd_ws(int64_t T, int n_q, int n_kv, int d) {
  const int64_t tiles = tiles_of(T);
  const int grp = n_q / n_kv;
  // A cut leaves at most 2 steps / most parts of a tile and most >= all steps / kSplitItems: at most
  // 2 kSplitItems parts in all; and no part is shorter than kSplitSteps / 2.
  int64_t slots = 0;
  if (pack_split(tiles, n_kv, grp)) {
    slots = 2 * kSplitItems / n_kv + 1;
    const int64_t most = tiles * (tiles * grp / kSplitSteps + 1);
    if (slots > most) slots = most;
  }
  BwdWs w;
  w.q_list = round256(static_cast<size_t>(n_q) * T * 4);
  w.kv_list = w.q_list + round256(static_cast<size_t>(tiles) * 16);
  w.head = w.kv_list + round256(static_cast<size_t>(tiles + slots) * 32);
  w.join = w.head + 256;
  w.part = w.join + round256(static_cast<size_t>(tiles) * 16);
  w.redo = w.part + static_cast<size_t>(slots) * n_kv * 2 * kTile * d * 4;
  w.total = w.redo + redo_bytes(T, n_q > 2 * n_kv ? n_q : 2 * n_kv) + 256;   // (it starts on 256 bytes)
  return w;
}

Operand mats(const char* name, const ttl_bf16* const* at, int t, int64_t T, int64_t ld, int64_t cols) {
  return operand(name, reinterpret_cast<const void* const*>(at), t, T, ld * 2, cols * 2);
}

const __nv_bfloat16* bf(const ttl_bf16* p) { return reinterpret_cast<const __nv_bfloat16*>(p); }
__nv_bfloat16* bf(ttl_bf16* p) { return reinterpret_cast<__nv_bfloat16*>(p); }

}  // namespace
}  // namespace ttl

using namespace ttl;

extern "C" size_t ttl_packed_attn_fwd_workspace_size(int t, int64_t T, int n_q, int n_kv, int d, int batch) {
  if (check_shape(t, T, n_q, n_kv, d, batch, "ttl_packed_attn_fwd_workspace_size")) return 0;
  return fwd_list_bytes(T) + redo_bytes(T, n_q);
}

extern "C" size_t ttl_packed_attn_bwd_workspace_size(int t, int64_t T, int n_q, int n_kv, int d, int batch) {
  if (check_shape(t, T, n_q, n_kv, d, batch, "ttl_packed_attn_bwd_workspace_size")) return 0;
  return bwd_ws(T, n_q, n_kv, d).total;
}

extern "C" int ttl_packed_attn_fwd(int t, int64_t T, int n_q, int n_kv, int d, int batch, const int32_t* cu_seqlens,
                                   float scale, const ttl_bf16* const* Q, int64_t ldq, const ttl_bf16* const* K,
                                   int64_t ldk, const ttl_bf16* const* V, int64_t ldv, ttl_bf16* const* O, int64_t ldo,
                                   float* const* lse, void* ws, size_t ws_bytes, void* stream) {
  const char* name = "ttl_packed_attn_fwd";
  int rc = check_shape(t, T, n_q, n_kv, d, batch, name);
  if (rc) return rc;
  if ((rc = check_cu(cu_seqlens, scale, name))) return rc;
  const int64_t qc = static_cast<int64_t>(n_q / t) * d, kc = static_cast<int64_t>(n_kv / t) * d;
  using CP = const void* const*;
  if (T == 0) return TTL_OK;
  if ((rc = check_mats(reinterpret_cast<CP>(Q), t, qc, ldq, "Q", name)) ||
      (rc = check_mats(reinterpret_cast<CP>(K), t, kc, ldk, "K", name)) ||
      (rc = check_mats(reinterpret_cast<CP>(V), t, kc, ldv, "V", name)) ||
      (rc = check_mats(reinterpret_cast<CP>(O), t, qc, ldo, "O", name)) || (rc = check_lse(lse, t, name)))
    return rc;
  const size_t need = ttl_packed_attn_fwd_workspace_size(t, T, n_q, n_kv, d, batch);
  if (!ws || ws_bytes < need)
    return set_error(TTL_ERR_ARG, "%s: workspace of %zu bytes needed, %zu given", name, need, ws_bytes);
  if (!aligned16(ws)) return set_error(TTL_ERR_ALIGN, "%s: workspace not 16-byte aligned", name);
  {
    const void *bounds = cu_seqlens, *space = ws;
    const Operand outs[3] = {mats("O", O, t, T, ldo, qc), operand("lse", reinterpret_cast<CP>(lse), t, n_q / t * T * 4),
                             operand("the workspace", &space, 1, static_cast<int64_t>(need))};
    const Operand ins[4] = {mats("Q", Q, t, T, ldq, qc), mats("K", K, t, T, ldk, kc), mats("V", V, t, T, ldv, kc),
                            operand("cu_seqlens", &bounds, 1, (int64_t(batch) + 1) * 4)};
    if ((rc = check_alias(outs, 3, ins, 4, name))) return rc;
  }
  if ((rc = require_sm103())) return rc;
  PackArgs A = {};
  A.status = device_status_ptr();
  if (!A.status) return TTL_ERR_CUDA;
  for (int i = 0; i < t; ++i) {
    A.s[i].q = bf(Q[i]);
    A.s[i].k = bf(K[i]);
    A.s[i].v = bf(V[i]);
    A.s[i].o = bf(O[i]);
    A.s[i].lse = lse[i];
  }
  A.t = t; A.nql = n_q / t; A.nkvl = n_kv / t; A.grp = n_q / n_kv; A.T = T;
  A.ldq = ldq; A.ldk = ldk; A.ldv = ldv; A.ldo = ldo;
  A.cu = cu_seqlens; A.batch = batch; A.scale = scale;
  A.redo = reinterpret_cast<RedoEntry*>(static_cast<char*>(ws) + fwd_list_bytes(T));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return pack_attn_fwd_launch(A, d, ws, s);
}

extern "C" int ttl_packed_attn_bwd(int t, int64_t T, int n_q, int n_kv, int d, int batch, const int32_t* cu_seqlens,
                                   float scale, const ttl_bf16* const* dO, int64_t lddo, const ttl_bf16* const* Q,
                                   int64_t ldq, const ttl_bf16* const* K, int64_t ldk, const ttl_bf16* const* V,
                                   int64_t ldv, const ttl_bf16* const* O, int64_t ldo, const float* const* lse,
                                   ttl_bf16* const* dQ, int64_t lddq, ttl_bf16* const* dK, int64_t lddk,
                                   ttl_bf16* const* dV, int64_t lddv, void* ws, size_t ws_bytes, void* stream) {
  const char* name = "ttl_packed_attn_bwd";
  int rc = check_shape(t, T, n_q, n_kv, d, batch, name);
  if (rc) return rc;
  if ((rc = check_cu(cu_seqlens, scale, name))) return rc;
  const int64_t qc = static_cast<int64_t>(n_q / t) * d, kc = static_cast<int64_t>(n_kv / t) * d;
  using CP = const void* const*;
  if (T == 0) return TTL_OK;
  if ((rc = check_mats(reinterpret_cast<CP>(dO), t, qc, lddo, "dO", name)) ||
      (rc = check_mats(reinterpret_cast<CP>(Q), t, qc, ldq, "Q", name)) ||
      (rc = check_mats(reinterpret_cast<CP>(K), t, kc, ldk, "K", name)) ||
      (rc = check_mats(reinterpret_cast<CP>(V), t, kc, ldv, "V", name)) ||
      (rc = check_mats(reinterpret_cast<CP>(O), t, qc, ldo, "O", name)) || (rc = check_lse(lse, t, name)) ||
      (rc = check_mats(reinterpret_cast<CP>(dQ), t, qc, lddq, "dQ", name)) ||
      (rc = check_mats(reinterpret_cast<CP>(dK), t, kc, lddk, "dK", name)) ||
      (rc = check_mats(reinterpret_cast<CP>(dV), t, kc, lddv, "dV", name)))
    return rc;
  const size_t need = ttl_packed_attn_bwd_workspace_size(t, T, n_q, n_kv, d, batch);
  if (!ws || ws_bytes < need)
    return set_error(TTL_ERR_ARG, "%s: workspace of %zu bytes needed, %zu given", name, need, ws_bytes);
  if (!aligned16(ws)) return set_error(TTL_ERR_ALIGN, "%s: workspace not 16-byte aligned", name);
  {
    const void *bounds = cu_seqlens, *space = ws;
    const Operand outs[4] = {mats("dQ", dQ, t, T, lddq, qc), mats("dK", dK, t, T, lddk, kc), mats("dV", dV, t, T, lddv, kc),
                             operand("the workspace", &space, 1, static_cast<int64_t>(need))};
    const Operand ins[7] = {mats("dO", dO, t, T, lddo, qc), mats("Q", Q, t, T, ldq, qc), mats("K", K, t, T, ldk, kc),
                            mats("V", V, t, T, ldv, kc), mats("O", O, t, T, ldo, qc),
                            operand("lse", reinterpret_cast<CP>(lse), t, n_q / t * T * 4),
                            operand("cu_seqlens", &bounds, 1, (int64_t(batch) + 1) * 4)};
    if ((rc = check_alias(outs, 4, ins, 7, name))) return rc;
  }
  if ((rc = require_sm103())) return rc;
  PackArgs A = {};
  A.status = device_status_ptr();
  if (!A.status) return TTL_ERR_CUDA;
  for (int i = 0; i < t; ++i) {
    A.s[i].q = bf(Q[i]);
    A.s[i].k = bf(K[i]);
    A.s[i].v = bf(V[i]);
    A.s[i].o = const_cast<__nv_bfloat16*>(bf(O[i]));
    A.s[i].lse = const_cast<float*>(lse[i]);
    A.s[i].dO = bf(dO[i]);
    A.s[i].dq = bf(dQ[i]);
    A.s[i].dk = bf(dK[i]);
    A.s[i].dv = bf(dV[i]);
  }
  A.t = t; A.nql = n_q / t; A.nkvl = n_kv / t; A.grp = n_q / n_kv; A.T = T;
  A.ldq = ldq; A.ldk = ldk; A.ldv = ldv; A.ldo = ldo;
  A.lddo = lddo; A.lddq = lddq; A.lddk = lddk; A.lddv = lddv;
  A.cu = cu_seqlens; A.batch = batch; A.scale = scale;
  A.D = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(ws) + 255) & ~uintptr_t(255));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Work lists where there are more items than SMs, or key tiles long enough to be cut; a batch below that
  // starts every item at once.
  const int64_t tiles = tiles_of(T);
  const bool split = pack_split(tiles, n_kv, A.grp);
  const bool listed = split || tiles * n_q > num_sms();
  PackPlan plan = {};
  const BwdWs w = bwd_ws(T, n_q, n_kv, d);
  char* base = reinterpret_cast<char*>(A.D);
  A.redo = reinterpret_cast<RedoEntry*>(base + w.redo);
  if (listed) {
    plan.q_list = reinterpret_cast<int4*>(base + w.q_list);
    plan.q_units = plan.tiles = static_cast<int>(tiles);
    plan.q_per = 1;
    plan.kv_list = reinterpret_cast<int4*>(base + w.kv_list);
    plan.kv_head = reinterpret_cast<int*>(base + w.head);
    plan.kv_taken = plan.kv_head + 2;
    plan.q_taken = plan.kv_head + 3;
    plan.join_list = reinterpret_cast<int4*>(base + w.join);
    plan.lanes = n_kv;
    plan.split = split;
    A.q_list = plan.q_list;
    A.kv_list = plan.kv_list;
    A.kv_head = plan.kv_head;
    A.q_taken = plan.q_taken;
    A.kv_taken = plan.kv_taken;
    A.join_list = plan.join_list;
    A.part = reinterpret_cast<float*>(base + w.part);
  }
  PackMaps maps = {};
  for (int i = 0; i < t; ++i)
    if ((rc = encode_map_bf16(&maps.q[i], A.s[i].q, T, qc, ldq, 64, kTile)) ||
        (rc = encode_map_bf16(&maps.k[i], A.s[i].k, T, kc, ldk, 64, kTile)) ||
        (rc = encode_map_bf16(&maps.v[i], A.s[i].v, T, kc, ldv, 64, kTile)) ||
        (rc = encode_map_bf16(&maps.dO[i], A.s[i].dO, T, qc, lddo, 64, kTile)))
      return rc;
  if ((rc = pack_attn_plan_launch(A, plan, d, s)) || (rc = pack_attn_dq_launch(A, maps, d, s)) ||
      (rc = pack_attn_dkv_launch(A, maps, d, s)))
    return rc;
  return split ? pack_attn_join_launch(A, d, s) : TTL_OK;
}
