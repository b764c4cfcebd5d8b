"""Refusals of the windowed packed attention entry points: status codes before anything touches a GPU (CPU only)."""
import ctypes

import pytest
import torch

import __graft_entry__ as entry


@pytest.fixture(scope="module")
def lib():
    entry.build()
    import tensor_transformer_layer_way_gb300 as ttl
    return ttl.lib()


def _arr(*vals):
    return (ctypes.c_void_p * len(vals))(*vals)


def _mat(base):
    return _arr(base, base + 0x100000)


# 16 tokens, two shards of 2 query heads and 1 KV head of 64
A2, B2, C2, D2, F2, L2, H2, I2, J2 = (_mat(0x1000000 * k) for k in range(1, 10))
BASE = dict(t=2, T=16, n_q=4, n_kv=2, d=64, batch=2, window=8, sinks=2, cu=0xb000000, scale=0.125, dO=A2, lddo=128, Q=B2,
            ldq=128, K=C2, ldk=64, V=D2, ldv=64, O=F2, ldo=128, lse=L2, dQ=H2, lddq=128, dK=I2, lddk=64, dV=J2, lddv=64,
            ws=0xa000000, ws_bytes=1 << 20)
HEAD = ("t", "T", "n_q", "n_kv", "d", "batch", "window", "sinks", "cu", "scale")


def _fwd(lib, **change):
    a = dict(BASE, **change)
    return lib.ttl_packed_window_attn_fwd(*[a[n] for n in HEAD + ("Q", "ldq", "K", "ldk", "V", "ldv", "O", "ldo", "lse", "ws",
                                                                  "ws_bytes")], None)


def _bwd(lib, **change):
    a = dict(BASE, **change)
    return lib.ttl_packed_window_attn_bwd(*[a[n] for n in HEAD + ("dO", "lddo", "Q", "ldq", "K", "ldk", "V", "ldv", "O", "ldo",
                                                                  "lse", "dQ", "lddq", "dK", "lddk", "dV", "lddv", "ws",
                                                                  "ws_bytes")], None)


@pytest.mark.parametrize("code,change", [
    (1, dict(window=0)), (1, dict(window=-3)), (1, dict(window=-2 ** 63)), (1, dict(sinks=-1)), (1, dict(sinks=-2 ** 63)),
    (1, dict(t=0)), (1, dict(T=-1)), (2, dict(t=3)), (2, dict(d=96)), (2, dict(T=1 << 28)), (1, dict(cu=None)),
    (3, dict(cu=0xb000002)), (1, dict(scale=0.0)), (1, dict(Q=None)), (3, dict(ldk=68)), (2, dict(ldv=56)), (1, dict(O=None)),
    (1, dict(lse=None)), (1, dict(ws=None)), (1, dict(ws_bytes=8)), (3, dict(ws=0xa000004)),
])
def test_refusals(lib, code, change):
    assert _fwd(lib, **change) == code
    assert len(lib.ttl_last_error()) > 10
    assert _bwd(lib, **change) == code


@pytest.mark.parametrize("change", [dict(dQ=A2), dict(dK=C2), dict(dV=I2), dict(ws=0x8000000), dict(dQ=_arr(0x8000000, 0x6100000))])
def test_backward_refuses_outputs_that_share_memory(lib, change):
    assert _bwd(lib, **change) == 1
    assert b"shares memory" in lib.ttl_last_error()


@pytest.mark.parametrize("change", [dict(O=B2), dict(lse=F2), dict(ws=0x2100000)])
def test_forward_refuses_outputs_that_share_memory(lib, change):
    assert _fwd(lib, **change) == 1
    assert b"shares memory" in lib.ttl_last_error()


def test_workspace_sizes(lib):
    fwd, bwd = lib.ttl_packed_window_attn_fwd_workspace_size, lib.ttl_packed_window_attn_bwd_workspace_size
    for f in (fwd, bwd):
        assert f(3, 16, 4, 2, 64, 1, 8, 0) == 0 and f(2, 16, 4, 2, 64, 1, 0, 0) == 0 and f(2, 16, 4, 2, 64, 1, 8, -1) == 0
    shape = (1, 40000, 32, 32, 64, 1)
    assert fwd(*shape, 100, 4) == lib.ttl_packed_attn_fwd_workspace_size(*shape)
    # where nothing is hidden, what packed attention needs; with a window, room for two parts of a key tile a block
    plain = lib.ttl_packed_attn_bwd_workspace_size(*shape)
    assert bwd(*shape, 40000, 4) == plain and bwd(*shape, 39996, 4) == plain
    for sinks in (0, 4):
        assert bwd(*shape, 100, sinks) >= 4 * 32 * 40000 + 2 * 152 * 2 * 128 * 64 * 4


def test_nothing_to_do(lib):
    assert _fwd(lib, T=0) == 0 and _bwd(lib, T=0) == 0
    assert _fwd(lib, T=0, window=0) == 1


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not memory: only where no kernel can be launched")
def test_what_is_taken(lib):
    """Windows and sinks of any size: as far as the device."""
    taken = lambda rc: rc not in (0, 1, 2, 3)     # noqa: E731
    for w, s in ((1, 0), (1, 2 ** 62), (2 ** 62, 2 ** 62), (15, 1), (3, 0)):
        assert taken(_fwd(lib, window=w, sinks=s)) and taken(_bwd(lib, window=w, sinks=s))
    cols = lambda base, at: _arr(base + 2 * at, base + 0x100000 + 2 * at)   # noqa: E731
    fused = dict(Q=cols(0x2000000, 0), K=cols(0x2000000, 128), V=cols(0x2000000, 192), ldq=256, ldk=256, ldv=256,
                 dQ=cols(0x7000000, 0), dK=cols(0x7000000, 128), dV=cols(0x7000000, 192), lddq=256, lddk=256, lddv=256)
    assert taken(_bwd(lib, **fused)) and taken(_fwd(lib, **fused))


def test_binding_refusals(lib):
    import tensor_transformer_layer_way_gb300 as ttl
    for w, s in ((0, 0), (4, -1)):
        with pytest.raises(ttl.TTLError):
            ttl.packed_window_attn_fwd_buffers(1, 16, 2, 1, 64, 1, w, s, device="cpu")
        with pytest.raises(ttl.TTLError):
            ttl.packed_window_attn_bwd_buffers(1, 16, 2, 1, 64, 1, w, s, device="cpu")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ttl.packed_window_attn_fwd([x], [x], [x], torch.zeros(2, dtype=torch.int32), window=2, n_q=1, n_kv=1, d=64)
    out = ttl.packed_window_attn_fwd_buffers(1, 16, 2, 1, 64, 1, 4, 1, device="cpu")
    assert out["O"][0].shape == (16, 128) and out["lse"][0].shape == (2, 16) and out["ws"].numel() > 0


@pytest.mark.parametrize("shape,code", [((1, 16, 2, 1, 96, 1, 4, 0), 2), ((3, 16, 4, 2, 64, 1, 4, 0), 2), ((1, 1 << 28, 2, 1, 64, 1, 4, 0), 2),
                                        ((1, 16, 3, 2, 64, 1, 4, 0), 2), ((17, 16, 17, 17, 64, 1, 4, 0), 1),
                                        ((1, 16, 2, 1, 64, -1, 4, 0), 1), ((1, 16, 2, 1, 64, 1, 0, 0), 1), ((1, 16, 2, 1, 64, 1, 4, -1), 1)])
def test_buffers_raise_the_codes_of_the_entry_points(lib, shape, code):
    import tensor_transformer_layer_way_gb300 as ttl
    for buffers in (ttl.packed_window_attn_fwd_buffers, ttl.packed_window_attn_bwd_buffers):
        with pytest.raises(ttl.TTLError) as e:
            buffers(*shape, device="cpu")
        assert e.value.code == code and "ttl_packed_window_attn_" in str(e.value)


@pytest.mark.parametrize("window,sinks", [(2 ** 64 + 5, 0), (2 ** 63, 2 ** 64), (5, 2 ** 64), (10 ** 30, 10 ** 30)])
def test_windows_beyond_64_bits_hide_nothing(lib, window, sinks):
    """Any size is taken: what the C integer cannot hold is longer than every document."""
    import tensor_transformer_layer_way_gb300 as ttl
    from tensor_transformer_layer_way_gb300 import _binding
    shape = (1, 40000, 32, 32, 64, 1)
    ws = ttl.lib().ttl_packed_attn_bwd_workspace_size(*shape)
    got = _binding._window_size(lib.ttl_packed_window_attn_bwd_workspace_size, lib.ttl_packed_window_attn_bwd, *shape,
                                *_binding._view(window, sinks))
    assert got == ws
    assert _binding._view(7, 3) == (7, 3) and _binding._view(-2 ** 70, -2 ** 70) == (-1, -1)
