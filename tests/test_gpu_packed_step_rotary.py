"""The packed training step with normalised and rotated heads and a window vs a plain 64-bit step (GPU).

Bounds.  The kernels round every tensor that passes from one step to the next to bf16: from ids to the last gradient
x0, n1, qkv, the rotated q and k, P, O, the partial sums and a, x1, n2, U and V, H, Z, x2, n3 (16), and going back dlogits,
dH, dx2, dH of the MLP, dU and dV, dn2, dx1, dO, dS, the gradients of the rotated q and k, dqkv, the partial sums and
dn1, dx0 (15).  Each moves its tensor by at most half a step (2^-8) of the elements, independently of the others, so
they add in quadrature: sqrt(31) 2^-8 = 2.2e-2 of a gradient's Frobenius norm.  Twice that is allowed: the norms' and the softmax's
backward passes subtract means, which leaves less of a gradient than of its rounding.  The loss is a mean of T logit
differences, each off by at most the logits' size times the forward part of that.
"""
import pytest
import torch

import tensor_transformer_layer_way_gb300 as ttl
from tensor_transformer_layer_way_gb300 import packed_step as ps

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8
GRAD_TOL = 2 * 31 ** 0.5 * HALF
F8 = torch.float64


def _norm(x, g, b):
    m = x.mean(1, keepdim=True)
    v = (x - m).square().mean(1, keepdim=True)
    return (x - m) / (v + 1e-5).sqrt() * g + b


def _rotated(x, gamma, angle):
    """x [T, heads, d], angle [T, rot/2]; columns i and rot/2 + i are a pair."""
    if gamma is not None:
        x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * gamma
    n = angle.shape[1]
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    a, b = x[..., :n], x[..., n:2 * n]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * n:]], -1)


def _reference(w, ids, target, cu, n_q, n_kv, d, freqs, axes, positions, window, sinks):
    """Loss, logits and every gradient in 64 bits by automatic differentiation of the plain formulas."""
    p = {n: ([m.detach().to(F8).requires_grad_() for m in v] if isinstance(v, list) else
             v.detach().to(F8).requires_grad_()) for n, v in w.items()}
    t, h, T = len(p["E"]), p["E"][0].shape[1], ids.shape[0]
    qc, kc, grp = n_q // t * d, n_kv // t * d, n_q // n_kv
    x0 = torch.cat(p["E"])[ids] * h ** 0.5
    n1 = _norm(x0, p["gamma1"], p["beta1"])
    tok = torch.arange(T, device=ids.device)
    cu = cu.to(torch.int64)
    doc = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    place = tok - cu[doc]
    back = tok[:, None] - tok[None, :]
    hide = (back < 0) | (doc[:, None] != doc[None, :])
    if window is not None:
        hide |= (back >= window) & (place >= sinks)[None, :]
    pos = place[None] if positions is None else positions.to(torch.int64)
    angle = pos[axes].T.to(F8) * torch.tensor(freqs, dtype=F8, device=ids.device)
    a = 0
    for i in range(t):
        m = n1 @ p["Wqkv"][i]
        q, k, v = (c.view(T, -1, d) for c in (m[:, :qc], m[:, qc:qc + kc], m[:, qc + kc:]))
        q, k = _rotated(q, p.get("gamma_q"), angle), _rotated(k, p.get("gamma_k"), angle)
        heads = []
        for c in range(n_q // t):
            s = (q[:, c] @ k[:, c // grp].T * d ** -0.5).masked_fill(hide, -float("inf"))
            heads.append(torch.softmax(s, 1) @ v[:, c // grp])
        a = a + torch.cat(heads, 1) @ p["Wo"][i]
    x1 = x0 + a
    n2 = _norm(x1, p["gamma2"], p["beta2"])
    z = 0
    for A, U, B in zip(p["A"], p["A_up"], p["B"]):
        u = n2 @ A
        z = z + (u * torch.sigmoid(u) * (n2 @ U)) @ B
    n3 = _norm(x1 + z, p["gamma3"], p["beta3"])
    logits = n3 @ torch.cat(p["W"]).T
    loss = (torch.logsumexp(logits, 1) - logits.gather(1, target[:, None])[:, 0]).mean()
    loss.backward()
    return loss.item(), logits.detach(), {n: ([m.grad for m in v] if isinstance(v, list) else v.grad) for n, v in p.items()}


# t, T, h, f, query heads, KV heads, d, V, documents; head norm, rotated columns, axes, window, sinks
CASES = [
    ((2, 1024, 256, 512, 4, 2, 64, 512, 7), True, 64, 1, 48, 2), ((1, 256, 128, 192, 2, 1, 64, 256, 3), False, 32, 1, None, 0),
    ((4, 512, 264, 544, 8, 4, 128, 800, 2), True, 0, 1, 128, 0), ((2, 768, 256, 256, 6, 2, 64, 304, 40), True, 64, 3, 5, 1),
    ((1, 512, 128, 256, 3, 1, 128, 256, 4), True, 128, 2, None, 0),
]


def _setup(shape, norm, rot, axes, window, sinks):
    t, T, h, f, n_q, n_kv, d, V, batch = shape
    w = ps.init_weights(t, h, f, n_q, n_kv, d, V, head_norm=norm, seed=T)
    g = torch.Generator().manual_seed(d)
    for n in ("gamma_q", "gamma_k"):
        if norm:
            w[n].copy_(1 + 0.2 * torch.randn(d, generator=g))
    freqs, pair_axes = ttl.rotary_freqs(rot), [i * axes // (rot // 2) for i in range(rot // 2)]
    step = ps.PackedStep(w, T, batch, n_q=n_q, n_kv=n_kv, d=d, rotary=ttl.Rotary(freqs, axes=pair_axes), window=window,
                         sinks=sinks)
    positions = None if axes == 1 else torch.randint(0, 40, (axes, T), generator=g, dtype=torch.int32).cuda()
    return w, step, ps.synthetic_pack(T, batch, V, seed=t), freqs, pair_axes, positions


@pytest.mark.parametrize("shape,norm,rot,axes,window,sinks", CASES)
def test_step_matches_the_plain_formulas(shape, norm, rot, axes, window, sinks):
    w, step, (ids, target, cu), freqs, pair_axes, positions = _setup(shape, norm, rot, axes, window, sinks)
    loss = step.forward(ids, target, cu, positions).item()
    grads = step.backward(ids, cu, positions)
    assert ttl.device_status() == 0
    want, logits, ref = _reference(w, ids, target, cu, *shape[4:7], freqs, pair_axes, positions, window, sinks)
    assert abs(loss - want) <= 16 ** 0.5 * HALF * logits.square().mean().sqrt().item()
    assert set(grads) == set(ref)
    for n, r in ref.items():
        got = torch.cat([x.to(F8).flatten() for x in grads[n]]) if isinstance(r, list) else grads[n].to(F8)
        r = torch.cat([x.flatten() for x in r]) if isinstance(r, list) else r
        err = ((got - r).norm() / r.norm()).item()
        assert err <= GRAD_TOL, f"{n}: {err:.3e}"


def test_step_replayed_from_a_graph_gives_the_same_bits():
    shape = CASES[0][0]
    w, step, pack, freqs, pair_axes, _ = _setup(*CASES[0])
    V, T, batch = shape[7], shape[1], shape[8]
    ids, target, cu = (x.clone() for x in pack)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step.forward(ids, target, cu)
        step.backward(ids, cu)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        loss = step.forward(ids, target, cu)
        grads = step.backward(ids, cu)
    for seed in (11, 12):                       # other packs in the same buffers
        for into, new in zip((ids, target, cu), ps.synthetic_pack(T, batch, V, seed=seed)):
            into.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        flat = [loss.clone()] + [x.clone() for v in grads.values() for x in (v if isinstance(v, list) else [v])]
        fresh = ps.PackedStep(w, T, batch, n_q=shape[4], n_kv=shape[5], d=shape[6], rotary=step.rotary, window=CASES[0][4],
                              sinks=CASES[0][5])
        again = [fresh.forward(ids, target, cu)]
        again += [x for v in fresh.backward(ids, cu).values() for x in (v if isinstance(v, list) else [v])]
        assert ttl.device_status() == 0
        assert all(torch.equal(a, b) for a, b in zip(flat, again))


def test_the_example_runs(capsys):
    losses = ps.main(steps=3, rotated=True, window=64, sinks=4)
    assert len(losses) == 3 and all(x == x for x in losses)
