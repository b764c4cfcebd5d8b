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


CALLS = {
    "layer_norm_fwd": lambda x, r, **kw: ttl.layer_norm_fwd(x["X"], x["gamma"], **kw),
    "layer_norm_bwd": lambda x, r, **kw: _norm_bwd(x, r["norm"], **kw),
    "scaled_fwd": lambda x, r, **kw: ttl.vocab_parallel_embedding_scaled_fwd(x["ids"], x["E"], 2.0, **kw),
    "sorted_bwd": lambda x, r, **kw: ttl.vocab_parallel_embedding_sorted_bwd(x["ids"], x["dY"][0], 2.0, r["dE"], **kw),
    "packed_attn_fwd": lambda x, r, **kw: ttl.packed_attn_fwd(x["Q"], x["K"], x["V"], x["cu"], **HEADS, **kw),
    "packed_attn_bwd": lambda x, r, **kw: _attn_bwd(x, r["attn"], **kw),
}


def _before(x):
    return {"norm": ttl.layer_norm_fwd(x["X"], x["gamma"]), "dE": [torch.zeros(V, H, device="cuda")],
            "attn": ttl.packed_attn_fwd(x["Q"], x["K"], x["V"], x["cu"], **HEADS)}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_that_a_call_makes_belong_to_its_stream(name, monkeypatch):
    x = _inputs()
    r = _before(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    made, empty = [], torch.empty

    def watched(*a, **kw):
        made.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", watched)
    CALLS[name](x, r, stream=side)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert made and set(made) == {side.cuda_stream}
    assert torch.cuda.current_stream().cuda_stream != side.cuda_stream


def _flat(out):
    out = [out[n] for n in sorted(out) if n != "ws" and out[n] is not None] if isinstance(out, dict) else [out]
    return [m for v in out for m in (v if isinstance(v, list) else [v])]


@pytest.mark.parametrize("name", CALLS)
def test_work_of_another_stream_does_not_meet_a_calls_buffers(name):
    """A call on a stream that is busy for a while, then allocations and writes on the current one."""
    x = _inputs()
    r = _before(x)
    want = [m.clone() for m in _flat(CALLS[name](x, r))]
    for m in r["dE"]:
        m.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    out = CALLS[name](x, r, stream=side)
    junk = []
    for size in (1 << 9, 1 << 12, 1 << 16, 1 << 19, 1 << 20, 3 << 20):
        for _ in range(8):
            junk.append(torch.full((size,), 255, dtype=torch.uint8, device="cuda"))
    side.synchronize()
    assert ttl.device_status() == 0
    for a, b in zip(want, _flat(out)):
        assert torch.equal(a, b)
