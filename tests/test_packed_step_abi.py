"""Refusals of the layer norm, sorted embedding and packed attention entry points: status codes
before anything touches a GPU (CPU only)."""
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


X2, R2, S2, Y2 = (_arr(a, a + 0x8000) for a in (0x100000, 0x200000, 0x300000, 0x400000))
M2, I2 = _arr(0x500000, 0x510000), _arr(0x520000, 0x530000)


def _norm_fwd(lib, t=2, rows=4, h=64, xt=0, wt=0, X=X2, ldx=64, R=None, ldr=64, gamma=0x600000, beta=0x610000,
              eps=1e-5, S=None, Y=Y2, mean=M2, rstd=I2):
    return lib.ttl_layer_norm_fwd(t, rows, h, xt, wt, X, ldx, R, ldr, gamma, beta, eps, S, Y, mean, rstd, None)


def _norm_bwd(lib, t=2, rows=4, h=64, xt=0, wt=0, X=X2, ldx=64, dY=R2, lddy=64, dS=None, ldds=64, gamma=0x600000,
              mean=M2, rstd=I2, dX=Y2, dgamma=0x700000, dbeta=0x710000, accumulate=0, ws=0x800000, ws_bytes=1 << 20):
    return lib.ttl_layer_norm_bwd(t, rows, h, xt, wt, X, ldx, dY, lddy, dS, ldds, gamma, mean, rstd, dX, dgamma,
                                  dbeta, accumulate, ws, ws_bytes, None)


@pytest.mark.parametrize("code,change", [
    (1, dict(t=0)), (1, dict(t=17)), (1, dict(rows=-1)), (1, dict(h=0)), (1, dict(xt=2)), (1, dict(wt=-1)),
    (1, dict(X=None)), (1, dict(X=_arr(0x100000, None))), (1, dict(gamma=None)), (1, dict(eps=-1.0)),
    (1, dict(eps=float("nan"))), (1, dict(R=R2)), (1, dict(S=S2)), (2, dict(ldx=63)),
    (2, dict(R=R2, S=S2, ldr=32)), (3, dict(X=_arr(0x100001, 0x108000))), (3, dict(gamma=0x600001)),
    (3, dict(xt=1, X=_arr(0x100002, 0x108000))), (1, dict(Y=X2)), (1, dict(R=R2, S=R2)), (1, dict(mean=None)),
    (1, dict(Y=_arr(0x100000 + 4 * 64 * 2 - 2, 0x400000))),    # Y[0] begins in X[0]'s last element
])
def test_layer_norm_fwd_refusals(lib, code, change):
    assert _norm_fwd(lib, **change) == code
    assert len(lib.ttl_last_error()) > 10


@pytest.mark.parametrize("code,change", [
    (1, dict(t=0)), (1, dict(accumulate=2)), (1, dict(dgamma=None)), (3, dict(dgamma=0x700002)), (1, dict(dY=None)),
    (2, dict(lddy=8)), (2, dict(dS=S2, ldds=8)), (1, dict(ws=None)), (1, dict(ws_bytes=16)), (3, dict(ws=0x800008)),
    (1, dict(dX=X2)), (1, dict(dX=R2)), (1, dict(dS=S2, dX=S2)), (1, dict(rstd=None)),
])
def test_layer_norm_bwd_refusals(lib, code, change):
    assert _norm_bwd(lib, **change) == code


def test_layer_norm_nothing_to_do(lib):
    assert _norm_fwd(lib, rows=0) == 0
    assert _norm_bwd(lib, rows=0, accumulate=1) == 0
    assert lib.ttl_layer_norm_bwd_workspace_size(0, 4, 64) == 0
    assert lib.ttl_layer_norm_bwd_workspace_size(2, 4, 64) >= 2 * 64 * 4


E2, G2, O2 = _arr(0x100000, 0x200000), _arr(0x300000, 0x400000), _arr(0x500000, 0x600000)


def _emb_bwd(lib, t=2, T=8, h=64, V=32, ids=0x10000, dY=0x20000, lddy=64, scale=2.0, dE=G2, accumulate=0,
             ws=0x800000, ws_bytes=1 << 24):
    return lib.ttl_vocab_parallel_embedding_sorted_bwd(t, T, h, V, ids, dY, lddy, scale, dE, accumulate, ws,
                                                       ws_bytes, None)


@pytest.mark.parametrize("code,change", [
    (1, dict(t=0)), (1, dict(T=-1)), (2, dict(V=33)), (2, dict(h=12)), (2, dict(T=1 << 31)), (1, dict(ids=None)),
    (3, dict(ids=0x10004)), (1, dict(dY=None)), (3, dict(dY=0x20008)), (3, dict(lddy=68)), (2, dict(lddy=56)),
    (1, dict(dE=None)), (1, dict(dE=_arr(0x300000, None))), (3, dict(dE=_arr(0x300000, 0x400008))),
    (1, dict(accumulate=2)), (1, dict(ws=None)), (1, dict(ws_bytes=64)), (3, dict(ws=0x800008)), (2, dict(V=0)),
])
def test_sorted_embedding_refusals(lib, code, change):
    assert _emb_bwd(lib, **change) == code


def test_scaled_embedding_refusals(lib):
    f = lib.ttl_vocab_parallel_embedding_scaled_fwd
    assert f(2, 8, 64, 33, 0x10000, E2, 2.0, O2, None) == 2
    assert f(2, 8, 60, 32, 0x10000, E2, 2.0, O2, None) == 2
    assert f(2, 8, 64, 32, 0x10004, E2, 2.0, O2, None) == 3
    assert f(2, 8, 64, 32, 0x10000, E2, 2.0, None, None) == 1
    assert f(2, 8, 64, 32, None, E2, 2.0, O2, None) == 1
    assert f(2, 0, 64, 32, None, E2, 2.0, O2, None) == 0
    assert _emb_bwd(lib, T=0, accumulate=1) == 0


def _attn_args(**change):
    a = dict(t=2, T=16, n_q=4, n_kv=2, d=64, batch=2, cu=0x10000, scale=0.125, dO=E2, lddo=128, Q=E2, ldq=128, K=G2,
             ldk=64, V=O2, ldv=64, O=Y2, ldo=128, lse=M2, dQ=X2, lddq=128, dK=R2, lddk=64, dV=S2, lddv=64,
             ws=0x900000, ws_bytes=1 << 20)
    a.update(change)
    return a


def _attn_fwd(lib, **change):
    a = _attn_args(**change)
    return lib.ttl_packed_attn_fwd(a["t"], a["T"], a["n_q"], a["n_kv"], a["d"], a["batch"], a["cu"], a["scale"],
                                   a["Q"], a["ldq"], a["K"], a["ldk"], a["V"], a["ldv"], a["O"], a["ldo"], a["lse"],
                                   a["ws"], a["ws_bytes"], None)


def _attn_bwd(lib, **change):
    a = _attn_args(**change)
    return lib.ttl_packed_attn_bwd(a["t"], a["T"], a["n_q"], a["n_kv"], a["d"], a["batch"], a["cu"], a["scale"],
                                   a["dO"], a["lddo"], a["Q"], a["ldq"], a["K"], a["ldk"], a["V"], a["ldv"], a["O"],
                                   a["ldo"], a["lse"], a["dQ"], a["lddq"], a["dK"], a["lddk"], a["dV"], a["lddv"],
                                   a["ws"], a["ws_bytes"], None)


SHARED = [
    (1, dict(t=0)), (1, dict(T=-1)), (1, dict(batch=-1)), (2, dict(t=3)), (2, dict(n_q=6, n_kv=4)), (2, dict(d=96)),
    (2, dict(T=1 << 28)), (1, dict(cu=None)), (3, dict(cu=0x10002)), (1, dict(scale=0.0)),
    (1, dict(scale=float("inf"))), (1, dict(scale=float("nan"))), (1, dict(Q=None)), (1, dict(K=_arr(0x300000, None))),
    (3, dict(V=_arr(0x500000, 0x600008))), (2, dict(ldq=120)), (3, dict(ldk=68)), (2, dict(ldv=56)), (1, dict(O=None)),
    (1, dict(lse=None)), (3, dict(lse=_arr(0x500002, 0x510000))),
]


@pytest.mark.parametrize("code,change", SHARED)
def test_packed_attn_fwd_refusals(lib, code, change):
    assert _attn_fwd(lib, **change) == code


@pytest.mark.parametrize("code,change", SHARED + [
    (1, dict(dO=None)), (3, dict(lddo=132)), (1, dict(dQ=None)), (2, dict(lddk=32)), (3, dict(dV=_arr(0x1, 0x2))),
    (1, dict(ws=None)), (1, dict(ws_bytes=8)), (3, dict(ws=0x900004)),
])
def test_packed_attn_bwd_refusals(lib, code, change):
    assert _attn_bwd(lib, **change) == code


def test_packed_attn_nothing_to_do(lib):
    assert _attn_fwd(lib, T=0) == 0 and _attn_bwd(lib, T=0) == 0
    assert lib.ttl_packed_attn_bwd_workspace_size(3, 16, 4, 2, 64, 1) == 0
    assert lib.ttl_packed_attn_bwd_workspace_size(2, 16, 4, 2, 64, 1) >= 4 * 16 * 4


def test_binding_refuses_host_tensors_and_wrong_types(lib):
    import tensor_transformer_layer_way_gb300 as ttl
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ttl.layer_norm_fwd([x], w)
    with pytest.raises(TypeError):
        ttl.layer_norm_fwd([x.half()], w)
    with pytest.raises(ValueError):
        ttl.layer_norm_fwd(x, w)
    with pytest.raises(ValueError):
        ttl.packed_attn_fwd([x], [x], [x], torch.zeros(2, dtype=torch.int32), n_q=1, n_kv=1, d=64)
    with pytest.raises(ValueError):
        ttl.vocab_parallel_embedding_scaled_fwd(torch.zeros(4, dtype=torch.int64), [x], 1.0)


# ---- outputs that share memory (4 rows of 64 bf16: 512 bytes a slab, 16 a slab of mean or rstd)
@pytest.mark.parametrize("change", [
    dict(Y=_arr(0x400000, 0x400000)), dict(Y=_arr(0x400000, 0x400100)), dict(R=R2, S=_arr(0x300000, 0x300000)),
    dict(R=R2, S=_arr(0x300000, 0x400000)), dict(R=R2, S=_arr(0x408000, 0x308000)), dict(R=R2, S=_arr(0x208000, 0x308000)),
    dict(mean=I2), dict(mean=_arr(0x500000, 0x50000c)), dict(rstd=_arr(0x100000, 0x530000)), dict(mean=_arr(0x4000f0, 0x510000)),
    dict(Y=_arr(0x600000, 0x408000)), dict(rstd=_arr(0x520000, 0x610040)),
])
def test_layer_norm_fwd_refuses_outputs_that_share_memory(lib, change):
    assert _norm_fwd(lib, **change) == 1
    assert b"shares memory" in lib.ttl_last_error()


@pytest.mark.parametrize("change", [
    dict(dX=_arr(0x400000, 0x400000)), dict(dX=_arr(0x100100, 0x408000)), dict(dgamma=0x710000), dict(dgamma=0x710080),
    dict(dbeta=0x100010), dict(dgamma=0x600000), dict(dX=_arr(0x500000, 0x408000)), dict(dX=_arr(0x400000, 0x530000)),
    dict(ws=0x400000), dict(ws=0x200000), dict(dS=S2, dX=_arr(0x400000, 0x308010)),
])
def test_layer_norm_bwd_refuses_outputs_that_share_memory(lib, change):
    assert _norm_bwd(lib, **change) == 1
    assert b"shares memory" in lib.ttl_last_error()


@pytest.mark.parametrize("change", [
    dict(dE=_arr(0x300000, 0x300000)), dict(dE=_arr(0x300000, 0x300ff0)), dict(dE=_arr(0x20010, 0x400000)),
    dict(dE=_arr(0x10030, 0x400000)), dict(ws=0x300000), dict(ws=0x20000), dict(ws=0x10000),
])
def test_sorted_embedding_refuses_outputs_that_share_memory(lib, change):
    assert _emb_bwd(lib, **change) == 1
    assert b"shares memory" in lib.ttl_last_error()


def test_scaled_embedding_refuses_outputs_that_share_memory(lib):
    f = lib.ttl_vocab_parallel_embedding_scaled_fwd
    for out in (E2, _arr(0x500000, 0x500010), _arr(0x1007f0, 0x600000), _arr(0x500000, 0x10030)):
        assert f(2, 8, 64, 32, 0x10000, E2, 2.0, out, None) == 1
        assert b"shares memory" in lib.ttl_last_error()


# 16 tokens, rows of 128 and 64 bf16, two shards each
A2, B2, C2, D2, F2, L2 = (_arr(a, a + 0x100000) for a in (0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x5000000, 0x6000000))
H2, I3, J2 = (_arr(a, a + 0x100000) for a in (0x7000000, 0x8000000, 0x9000000))


def _apart(**change):
    return dict(dict(dO=A2, Q=B2, K=C2, V=D2, O=F2, lse=L2, dQ=H2, dK=I3, dV=J2, ws=0xa000000, cu=0xb000000), **change)


@pytest.mark.parametrize("change", [
    dict(O=B2), dict(O=C2), dict(O=_arr(0x5000000, 0x5000000)), dict(lse=F2), dict(lse=_arr(0x6000000, 0x600007c)),
    dict(O=_arr(0x5000000, 0x4100010)), dict(lse=_arr(0xb000000, 0x6100000)), dict(ws=0x2100000), dict(ws=0x5000000),
    dict(ldo=192, ldq=192, O=_arr(0x5000000, 0x2100000 + 112)),         # 8 columns into Q's
])
def test_packed_attn_fwd_refuses_outputs_that_share_memory(lib, change):
    assert _attn_fwd(lib, **_apart(**change)) == 1
    assert b"shares memory" in lib.ttl_last_error()


@pytest.mark.parametrize("change", [
    dict(dQ=A2), dict(dQ=B2), dict(dQ=F2), dict(dK=C2), dict(dV=D2), dict(dV=I3), dict(dK=_arr(0x8000000, 0x8000000)),
    dict(dQ=_arr(0x7000000, 0x6100000)), dict(dV=_arr(0xb000000, 0x9100000)), dict(ws=0x7000000), dict(ws=0x6000000),
    dict(lddq=256, lddk=256, dK=_arr(0x7000000 + 240, 0x8100000)),      # dK 8 columns into dQ's
    dict(lddq=256, lddk=192, dK=_arr(0x7000000 + 256, 0x8100000)),      # two row strides in one place
])
def test_packed_attn_bwd_refuses_outputs_that_share_memory(lib, change):
    assert _attn_bwd(lib, **_apart(**change)) == 1
    assert b"shares memory" in lib.ttl_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not memory: only where no kernel can be launched")
def test_outputs_beside_each_other_are_taken(lib):
    """Column ranges of one matrix, neighbours in memory, inputs that are the same: the calls get as far as the device."""
    taken = lambda rc: rc not in (0, 1, 2, 3)     # noqa: E731
    cols = lambda base, at: _arr(base + 2 * at, base + 0x100000 + 2 * at)   # noqa: E731
    fused = dict(Q=cols(0x2000000, 0), K=cols(0x2000000, 128), V=cols(0x2000000, 192), ldq=256, ldk=256, ldv=256,
                 dQ=cols(0x7000000, 0), dK=cols(0x7000000, 128), dV=cols(0x7000000, 192), lddq=256, lddk=256, lddv=256)
    assert taken(_attn_bwd(lib, **_apart(**fused))) and taken(_attn_fwd(lib, **_apart(**fused)))
    assert taken(_attn_fwd(lib, **_apart(K=D2))) and taken(_attn_bwd(lib, **_apart(dO=F2, K=D2)))
    assert taken(_attn_fwd(lib, **_apart(O=_arr(0x5000000, 0x5000000 + 16 * 128 * 2))))
    assert taken(_attn_fwd(lib, T=1, **_apart(O=_arr(0x5000000, 0x5000000 + 256))))
    assert taken(_norm_fwd(lib, Y=_arr(0x400000, 0x400000 + 512), mean=_arr(0x500000, 0x500010), rstd=_arr(0x500020, 0x500030)))
    assert taken(_norm_fwd(lib, X=_arr(0x100000, 0x100000)))
    assert taken(_norm_bwd(lib, dY=X2, dS=X2)) and taken(_norm_bwd(lib, dbeta=0x700100))
    assert taken(_emb_bwd(lib, dE=_arr(0x300000, 0x300000 + 16 * 64 * 4)))
    f = lib.ttl_vocab_parallel_embedding_scaled_fwd
    assert taken(f(2, 8, 64, 32, 0x10000, E2, 2.0, _arr(0x500000, 0x500000), None))
    assert taken(f(2, 8, 64, 32, 0x10000, _arr(0x100000, 0x100000), 2.0, O2, None))


def test_binding_refuses_workspaces_that_are_no_device_memory(lib):
    from tensor_transformer_layer_way_gb300 import _binding
    for bad, error in ((torch.empty(64, dtype=torch.uint8), ValueError), (torch.empty(1 << 20, dtype=torch.uint8, device="meta"), ValueError),
                       (None, TypeError), (1 << 20, TypeError)):
        with pytest.raises(error):
            _binding._space(bad)
