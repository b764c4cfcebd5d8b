"""Workspaces and streams of the layer norm, embedding and packed attention calls (GPU)."""
import pytest
import torch

import tensor_transformer_layer_way_gb300 as ttl

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
T, H, V, N_Q, N_KV, D = 300, 256, 512, 4, 2, 64
HEADS = dict(n_q=N_Q, n_kv=N_KV, d=D)


def _inputs():
    g = torch.Generator("cuda").manual_seed(3)

    def mat(rows, cols):
        return torch.randn(rows, cols, generator=g, device="cuda").to(BF16)

    return {"X": [mat(T, H)], "dY": [mat(T, H)], "gamma": mat(1, H)[0], "E": [mat(V, H)],
            "ids": torch.randint(0, V, (T,), generator=g, device="cuda"), "Q": [mat(T, N_Q * D)], "K": [mat(T, N_KV * D)],
            "V": [mat(T, N_KV * D)], "dO": [mat(T, N_Q * D)], "cu": torch.tensor([0, 100, T], dtype=torch.int32, device="cuda")}


def _norm_bwd(x, fwd, **kw):
    return ttl.layer_norm_bwd(x["X"], x["dY"], x["gamma"], fwd, **kw)


def _attn_bwd(x, fwd, **kw):
    return ttl.packed_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], fwd, x["cu"], **HEADS, **kw)


def _spaces():
    """What is no workspace: host memory, a view that repeats its bytes, and one that is too small."""
    return [torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 20),
            torch.empty(1 << 21, dtype=torch.uint8, device="cuda")[::2], torch.empty(16, dtype=torch.uint8, device="cuda"), None]


def test_workspaces_that_are_none_are_refused():
    x = _inputs()
    norm = ttl.layer_norm_fwd(x["X"], x["gamma"])
    attn = ttl.packed_attn_fwd(x["Q"], x["K"], x["V"], x["cu"], **HEADS)
    dE = [torch.zeros(V, H, device="cuda")]
    for ws in _spaces():
        errors = (ValueError, TypeError, ttl.TTLError)
        with pytest.raises(errors):
            _norm_bwd(x, norm, out=dict(ttl.layer_norm_bwd_buffers(1, T, H), ws=ws))
        with pytest.raises(errors):
            ttl.packed_attn_fwd(x["Q"], x["K"], x["V"], x["cu"], out=dict(ttl.packed_attn_fwd_buffers(1, T, N_Q, N_KV, D, 2), ws=ws), **HEADS)
        with pytest.raises(errors):
            _attn_bwd(x, attn, out=dict(ttl.packed_attn_bwd_buffers(1, T, N_Q, N_KV, D, 2), ws=ws))
        if ws is not None:          # (None: the call makes its own)
            with pytest.raises(errors):
                ttl.vocab_parallel_embedding_sorted_bwd(x["ids"], x["dY"][0], 1.0, dE, ws=ws)
    assert ttl.device_status() == 0 and torch.count_nonzero(dE[0]) == 0


def test_a_workspace_of_another_type_counts_its_bytes():
    x = _inputs()
    norm = ttl.layer_norm_fwd(x["X"], x["gamma"])
    out = ttl.layer_norm_bwd_buffers(1, T, H)
    want = _norm_bwd(x, norm)
    out["ws"] = torch.empty(out["ws"].numel() // 4, device="cuda")
    got = _norm_bwd(x, norm, out=out)
    assert torch.equal(got["dX"][0], want["dX"][0]) and torch.equal(got["dgamma"], want["dgamma"])
