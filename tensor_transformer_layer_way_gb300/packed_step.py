"""One training step on a pack of documents: scaled embedding, a sequence-parallel block with packed
attention, LM head and loss, and every gradient.

Source: "v4:Tensor Parallel 与 Sequence Parallel" -- "Embedding 和 LM head:按 vocab 切", "Attention:按
head 切" and "SP": between the tensor-parallel regions shard i holds token slab i of the residual
stream, where layer norm and the residual sum run; the regions themselves see all tokens.  The t
shards are buffers of one GPU, so a region's gathered input is one [T, h] buffer whose slabs the
norm writes in place, and the reduce-scatter behind W_O is ``shard_reduce_scatter``.

    x0 = scale E[ids]                      n1 = norm(x0)
    q, k, v = n1 Wqkv_i                    a = sum_i attention(q, k, v) Wo_i
    x1 = x0 + a, n2 = norm(x1)             z = sequence-parallel MLP(n2)
    x2 = x1 + z, n3 = norm(x2)             loss = cross-entropy(n3 W^T, target)

Where asked for, the heads of q and k are normalised and rotated by position before the attention, and the
attention sees a window of each document and its first tokens.

Only the order of the calls lives here: every step is a call into the C library, on the current
stream, into buffers that are allocated once per shape; a step can be captured into a CUDA graph.
Run as a module it trains a small model on synthetic packs and prints the loss.
"""
from __future__ import annotations

import math

import torch

from . import _binding as ttl


def init_weights(t, h, f, n_q, n_kv, d, V, *, head_norm=False, seed=0, device="cuda"):
    """Random weights of one block in the shards' layout: E and W [V/t, h], Wqkv [h, (n_q + 2 n_kv)/t d],
    Wo [n_q/t d, h], A and A_up [h, f/t], B [f/t, h], and the three norms' gamma and beta [h]; with head_norm
    the heads' gamma_q and gamma_k [d] too."""
    g = torch.Generator().manual_seed(seed)

    def mats(rows, cols, std):
        return [(torch.randn(rows, cols, generator=g) * std).to(torch.bfloat16).to(device) for _ in range(t)]

    w = {"E": mats(V // t, h, h ** -0.5), "W": mats(V // t, h, h ** -0.5),
         "Wqkv": mats(h, (n_q + 2 * n_kv) // t * d, h ** -0.5), "Wo": mats(n_q // t * d, h, (n_q * d) ** -0.5),
         "A": mats(h, f // t, h ** -0.5), "A_up": mats(h, f // t, h ** -0.5), "B": mats(f // t, h, f ** -0.5)}
    for n in ("1", "2", "3"):
        w["gamma" + n] = torch.ones(h, dtype=torch.bfloat16, device=device)
        w["beta" + n] = torch.zeros(h, dtype=torch.bfloat16, device=device)
    if head_norm:
        w["gamma_q"] = torch.ones(d, dtype=torch.bfloat16, device=device)
        w["gamma_k"] = torch.ones(d, dtype=torch.bfloat16, device=device)
    return w


class PackedStep:
    """Buffers and call order of the step for T tokens (a multiple of 128 t) in `batch` documents.  Weights gamma_q and
    gamma_k normalise the heads, a `Rotary` rotates them, `window` (with `sinks`) limits what they see."""

    def __init__(self, weights, T, batch, *, n_q, n_kv, d, rotary=None, window=None, sinks=0, device="cuda"):
        if window is None and sinks:
            raise ValueError("sinks are the first tokens that stay visible behind a window: they need one")
        self.w = weights
        self.t = t = len(weights["E"])
        self.heads = dict(n_q=n_q, n_kv=n_kv, d=d)
        Vs, h = weights["E"][0].shape
        V = Vs * t
        self.scale = math.sqrt(h)
        slab = T // t
        qc, kc = n_q // t * d, n_kv // t * d
        e = dict(device=device, dtype=torch.bfloat16)

        def slabs(m):
            return [m[i * slab:(i + 1) * slab] for i in range(t)]

        def each(*shape, dtype=torch.bfloat16):
            return [torch.empty(*shape, device=device, dtype=dtype) for _ in range(t)]

        def qkv(mats):
            return ([m[:, :qc] for m in mats], [m[:, qc:qc + kc] for m in mats], [m[:, qc + kc:] for m in mats])

        self.x0 = each(T, h)
        self.x0_slabs = [x[i * slab:(i + 1) * slab] for i, x in enumerate(self.x0)]
        # the norms in front of a region write its gathered input
        self.n1, self.n3 = torch.empty(T, h, **e), torch.empty(T, h, **e)
        self.norm1 = dict(ttl.layer_norm_fwd_buffers(t, slab, h, device=device), Y=slabs(self.n1))
        self.norm2 = ttl.layer_norm_fwd_buffers(t, slab, h, residual=True, device=device)
        self.norm3 = dict(ttl.layer_norm_fwd_buffers(t, slab, h, residual=True, device=device), Y=slabs(self.n3))
        self.qkv = each(T, qc + 2 * kc)
        self.q, self.k, self.v = qkv(self.qkv)
        # what the attention reads of q and k: the projection's columns, or normalised and rotated copies
        self.head_norm = dict(gamma_q=weights.get("gamma_q"), gamma_k=weights.get("gamma_k"))
        self.rotary = ttl.Rotary(()) if rotary is None and "gamma_q" in weights else rotary
        self.seen = {"Q": self.q, "K": self.k}
        if self.rotary is not None:
            self.seen = ttl.head_norm_rotary_fwd_buffers(t, T, n_q, n_kv, d, device)
        if window is None:
            self.view = {}
            self.attn_fwd, self.attn_bwd_of = ttl.packed_attn_fwd, ttl.packed_attn_bwd
            self.attn = ttl.packed_attn_fwd_buffers(t, T, n_q, n_kv, d, batch, device)
            attn_bwd = ttl.packed_attn_bwd_buffers(t, T, n_q, n_kv, d, batch, device)
        else:
            self.view = dict(window=window, sinks=sinks)
            self.attn_fwd, self.attn_bwd_of = ttl.packed_window_attn_fwd, ttl.packed_window_attn_bwd
            self.attn = ttl.packed_window_attn_fwd_buffers(t, T, n_q, n_kv, d, batch, window, sinks, device)
            attn_bwd = ttl.packed_window_attn_bwd_buffers(t, T, n_q, n_kv, d, batch, window, sinks, device)
        self.partial = each(T, h)              # per-shard sums over its heads, forward and backward
        self.partial_slabs = [p[i * slab:(i + 1) * slab] for i, p in enumerate(self.partial)]
        self.mlp = None                        # allocated by the first call
        self.ce = ttl.ce_buffers(t, T, h, V, device)
        self.dH_slabs = slabs(self.ce["dH"])

        self.g1, self.dx0 = torch.empty(T, h, **e), torch.empty(T, h, **e)
        self.bwd3 = ttl.layer_norm_bwd_buffers(t, slab, h, device=device)
        self.bwd2 = dict(ttl.layer_norm_bwd_buffers(t, slab, h, device=device), dX=slabs(self.g1))
        self.bwd1 = dict(ttl.layer_norm_bwd_buffers(t, slab, h, device=device), dX=slabs(self.dx0))
        self.mlp_bwd = None
        self.dO = each(T, qc)
        self.dqkv = each(T, qc + 2 * kc)
        dq, dk, dv = qkv(self.dqkv)
        self.attn_bwd = dict(attn_bwd, dQ=dq, dK=dk, dV=dv)
        self.rotary_bwd = None
        if self.rotary is not None:            # in place: the columns of dqkv that the attention's gradients are in
            self.rotary_bwd = dict(ttl.head_norm_rotary_bwd_buffers(t, 0, n_q, n_kv, d, "gamma_q" in weights, device),
                                   dQ=dq, dK=dk)
            if "gamma_q" in weights:
                ws = int(ttl.lib().ttl_head_norm_rotary_bwd_workspace_size(t, T, n_q, n_kv, d))
                self.rotary_bwd["ws"] = torch.empty(ws, dtype=torch.uint8, device=device)
        self.dW = each(Vs, h, dtype=torch.float32)
        self.dWo = each(qc, h, dtype=torch.float32)
        self.dWqkv = each(h, qc + 2 * kc, dtype=torch.float32)
        self.dE = each(Vs, h, dtype=torch.float32)
        self.embed_ws = ttl.embedding_sorted_bwd_workspace(t, T, h, V, device)

    def _check_positions(self, positions):
        if positions is not None and (self.rotary is None or self.rotary.rot == 0):
            raise ValueError("positions are the rotation's: this step has none")

    def forward(self, ids, target, cu_seqlens, positions=None):
        """The mean loss over all tokens (a tensor of one fp32 value).  `positions` (int32, [axes, T]) are the rotation's;
        by default a token's place in its document."""
        self._check_positions(positions)
        w = self.w
        ttl.vocab_parallel_embedding_scaled_fwd(ids, w["E"], self.scale, out=self.x0)
        ttl.layer_norm_fwd(self.x0_slabs, w["gamma1"], w["beta1"], out=self.norm1)
        for i in range(self.t):
            ttl.gemm(self.n1, w["Wqkv"][i], self.qkv[i], b_kmajor=False)
        if self.rotary is not None:
            ttl.head_norm_rotary_fwd(self.q, self.k, self.rotary, positions=positions, cu_seqlens=cu_seqlens,
                                     out=self.seen, **self.heads, **self.head_norm)
        self.attn_fwd(self.seen["Q"], self.seen["K"], self.v, cu_seqlens, out=self.attn, **self.heads, **self.view)
        for i in range(self.t):
            ttl.gemm(self.attn["O"][i], w["Wo"][i], self.partial[i], b_kmajor=False)
        ttl.shard_reduce_scatter(self.partial)
        ttl.layer_norm_fwd(self.x0_slabs, w["gamma2"], w["beta2"], residual=self.partial_slabs, out=self.norm2)
        self.mlp = ttl.sp_mlp_fwd(self.norm2["Y"], w["A"], w["B"], act="swiglu", A_up=w["A_up"], out=self.mlp)
        ttl.layer_norm_fwd(self.norm2["S"], w["gamma3"], w["beta3"], residual=self.mlp["Z_slabs"], out=self.norm3)
        ttl.vocab_parallel_ce(self.n3, w["W"], target, out=self.ce)
        return self.ce["loss"]

    def backward(self, ids, cu_seqlens, positions=None):
        """Every weight's gradient, under the weight's name; after forward() on the same pack (and positions)."""
        self._check_positions(positions)
        w, out = self.w, {}
        tn = dict(a_kmajor=False, b_kmajor=False)
        for i in range(self.t):
            ttl.gemm(self.ce["dlogits"][i], self.n3, self.dW[i], **tn)
        ttl.layer_norm_bwd(self.norm3["S"], self.dH_slabs, w["gamma3"], self.norm3, out=self.bwd3)
        self.mlp_bwd = ttl.sp_mlp_bwd(self.norm2["Y"], self.bwd3["dX"], w["A"], w["B"], self.mlp, act="swiglu",
                                      A_up=w["A_up"], out=self.mlp_bwd)
        ttl.layer_norm_bwd(self.norm2["S"], self.mlp_bwd["dX_slabs"], w["gamma2"], self.norm2, dS=self.bwd3["dX"],
                           out=self.bwd2)
        for i in range(self.t):
            ttl.gemm(self.g1, w["Wo"][i], self.dO[i])
            ttl.gemm(self.attn["O"][i], self.g1, self.dWo[i], **tn)
        self.attn_bwd_of(self.dO, self.seen["Q"], self.seen["K"], self.v, self.attn, cu_seqlens, out=self.attn_bwd,
                         **self.heads, **self.view)
        if self.rotary is not None:
            ttl.head_norm_rotary_bwd(self.attn_bwd["dQ"], self.attn_bwd["dK"], self.rotary, Q=self.q, K=self.k,
                                     positions=positions, cu_seqlens=cu_seqlens, out=self.rotary_bwd, **self.heads,
                                     **self.head_norm)
        for i in range(self.t):
            ttl.gemm(self.dqkv[i], w["Wqkv"][i], self.partial[i])
            ttl.gemm(self.n1, self.dqkv[i], self.dWqkv[i], **tn)
        ttl.shard_reduce_scatter(self.partial)
        ttl.layer_norm_bwd(self.x0_slabs, self.partial_slabs, w["gamma1"], self.norm1, dS=self.bwd2["dX"], out=self.bwd1)
        ttl.vocab_parallel_embedding_sorted_bwd(ids, self.dx0, self.scale, self.dE, ws=self.embed_ws)
        out.update(E=self.dE, W=self.dW, Wqkv=self.dWqkv, Wo=self.dWo, A=self.mlp_bwd["dA"],
                   A_up=self.mlp_bwd["dA_up"], B=self.mlp_bwd["dB"])
        for n, b in (("1", self.bwd1), ("2", self.bwd2), ("3", self.bwd3)):
            out["gamma" + n], out["beta" + n] = b["dgamma"], b["dbeta"]
        if "gamma_q" in w:
            out["gamma_q"], out["gamma_k"] = self.rotary_bwd["dgamma_q"], self.rotary_bwd["dgamma_k"]
        return out


def synthetic_pack(T, batch, V, *, seed, device="cuda"):
    """Documents of uneven lengths that count upwards from a random id: ids, targets (the next id) and bounds."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, T + 1, (batch - 1,), generator=g).sort()[0]
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([T])])
    start = torch.randint(0, V, (batch,), generator=g)
    doc = torch.repeat_interleave(torch.arange(batch), cu[1:] - cu[:-1])
    ids = (start[doc] + torch.arange(T) - cu[:-1][doc]) % V
    return ids.to(device), ((ids + 1) % V).to(device), cu.to(torch.int32).to(device)


def main(steps=20, lr=0.2, rotated=False, window=None, sinks=0):
    """Trains; `rotated` with normalised and rotated heads, `window` and `sinks` as PackedStep takes them."""
    t, T, h, f, n_q, n_kv, d, V, batch = 2, 1024, 256, 512, 4, 2, 64, 512, 6
    w = init_weights(t, h, f, n_q, n_kv, d, V, head_norm=rotated)
    master = {n: [p.float() for p in (m if isinstance(m, list) else [m])] for n, m in w.items()}
    rotary = ttl.Rotary(ttl.rotary_freqs(d)) if rotated else None
    step = PackedStep(w, T, batch, n_q=n_q, n_kv=n_kv, d=d, rotary=rotary, window=window, sinks=sinks)
    losses = []
    for s in range(steps):
        ids, target, cu = synthetic_pack(T, batch, V, seed=s)
        losses.append(step.forward(ids, target, cu).item())
        grads = step.backward(ids, cu)
        for n, m in w.items():
            lists = (m, grads[n]) if isinstance(m, list) else ([m], [grads[n]])
            for p, full, g in zip(lists[0], master[n], lists[1]):
                full.sub_(g.float(), alpha=lr)
                p.copy_(full)
        print(f"step {s:3d}  loss {losses[-1]:.4f}")
    if ttl.device_status() != 0:
        raise RuntimeError("the library reported a device error: " + ttl.last_error())
    return losses


if __name__ == "__main__":
    import argparse
    parser = argparse.ArgumentParser(description="Trains a small model on synthetic packs.")
    parser.add_argument("--rotated", action="store_true", help="normalised and rotated heads")
    parser.add_argument("--window", type=int, help="keys that a query sees up to itself")
    parser.add_argument("--sinks", type=int, default=0, help="first tokens of a document that stay visible behind the window")
    main(**vars(parser.parse_args()))
