"""Refusals of the head norm and rotation: status codes before anything touches a GPU (CPU only)."""
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


def _doubles(*v):
    return (ctypes.c_double * len(v))(*v)


F8 = _doubles(*[10000.0 ** (-i / 8) for i in range(8)])
AX = lambda *v: (ctypes.c_int32 * len(v))(*v)   # noqa: E731
Q2, K2, QO, KO, DY, DK = (_mat(a) for a in (0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x5000000, 0x6000000))
# two shards of 2 and 1 heads of 64, 16 tokens, 16 columns rotated
BASE = dict(t=2, T=16, n_q=4, n_kv=2, d=64, rot=16, inter=0, freqs=F8, pair_axis=None, axes=1, pos=None, batch=2,
            cu=0x8000000, wt=0, gq=0x8100000, gk=0x8200000, eps=1e-6, Q=Q2, ldq=128, K=K2, ldk=64, Qo=QO, ldqo=128,
            Ko=KO, ldko=64, dYq=DY, lddyq=128, dYk=DK, lddyk=64, dgq=0x8300000, dgk=0x8400000, accumulate=0,
            ws=0x9000000, ws_bytes=1 << 22)


def _head(a):
    return [a[n] for n in ("t", "T", "n_q", "n_kv", "d", "rot", "inter", "freqs", "pair_axis", "axes", "pos", "batch", "cu",
                           "wt", "gq", "gk", "eps")]


def _fwd(lib, **change):
    a = dict(BASE, **change)
    return lib.ttl_head_norm_rotary_fwd(*_head(a), a["Q"], a["ldq"], a["K"], a["ldk"], a["Qo"], a["ldqo"], a["Ko"],
                                        a["ldko"], None)


def _bwd(lib, **change):
    a = dict(BASE, **change)
    return lib.ttl_head_norm_rotary_bwd(*_head(a), a["dYq"], a["lddyq"], a["dYk"], a["lddyk"], a["Q"], a["ldq"], a["K"],
                                        a["ldk"], a["Qo"], a["ldqo"], a["Ko"], a["ldko"], a["dgq"], a["dgk"],
                                        a["accumulate"], a["ws"], a["ws_bytes"], None)


BOTH = [
    (1, dict(t=0)), (1, dict(t=17)), (1, dict(T=-1)), (1, dict(n_kv=0)), (2, dict(t=3)), (2, dict(n_q=3)), (2, dict(d=72)),
    (2, dict(d=272)), (2, dict(T=1 << 31)), (2, dict(rot=8)), (2, dict(rot=80)), (2, dict(rot=-16)), (1, dict(inter=2)),
    (1, dict(freqs=None)), (1, dict(freqs=_doubles(*[1.0] * 7, float("nan")))), (1, dict(freqs=_doubles(*[1.0] * 7, 2e6))),
    (1, dict(axes=0)), (1, dict(axes=9, pos=0x7000000)), (1, dict(axes=2)),
    (1, dict(axes=2, pos=0x7000000, pair_axis=AX(0, 0, 0, 0, 1, 1, 1, 2))), (1, dict(pair_axis=AX(*[-1] * 8))),
    (3, dict(pos=0x7000002)), (1, dict(batch=-1)), (3, dict(cu=0x8000001)), (1, dict(gq=None)), (1, dict(gk=None)),
    (1, dict(wt=2)), (3, dict(gq=0x8100001)), (3, dict(wt=1, gk=0x8200002)), (1, dict(eps=-1.0)), (1, dict(eps=float("nan"))),
    (1, dict(eps=float("inf"))), (1, dict(Q=None)), (1, dict(K=_arr(0x2000000, None))), (3, dict(Q=_arr(0x1000008, 0x1100000))),
    (2, dict(ldq=120)), (3, dict(ldk=68)), (2, dict(ldqo=64)), (3, dict(ldko=65)), (1, dict(Ko=None)), (2, dict(ldq=1 << 31)),
]


@pytest.mark.parametrize("code,change", BOTH)
def test_refusals(lib, code, change):
    assert _fwd(lib, **change) == code
    assert len(lib.ttl_last_error()) > 10
    assert _bwd(lib, **change) == code


@pytest.mark.parametrize("code,change", [
    (1, dict(dYq=None)), (2, dict(lddyk=32)), (3, dict(lddyq=132)), (1, dict(dgq=None)), (3, dict(dgk=0x8400002)),
    (1, dict(gq=None, gk=None)), (1, dict(accumulate=2)), (1, dict(ws=None)), (1, dict(ws_bytes=64)), (3, dict(ws=0x9000008)),
])
def test_backward_refusals(lib, code, change):
    assert _bwd(lib, **change) == code
    assert len(lib.ttl_last_error()) > 10


@pytest.mark.parametrize("change", [
    dict(Qo=K2), dict(Ko=K2, ldko=72), dict(Qo=_arr(0x1000000, 0x3100000)), dict(Qo=_arr(0x1100000, 0x1000000)),
    dict(Ko=QO), dict(Qo=_arr(0x3000000, 0x3000000)), dict(Qo=_arr(0x1000010, 0x1100010)), dict(Qo=_arr(0x8000000, 0x3100000)),
    dict(Qo=_arr(0x8100000 - 16, 0x3100000)), dict(pos=0x3000040), dict(ldqo=192, ldko=192, Ko=_arr(0x3000000 + 240, 0x4100000)),
])
def test_forward_refuses_outputs_that_share_memory(lib, change):
    assert _fwd(lib, **change) == 1
    assert b"shares memory" in lib.ttl_last_error()


@pytest.mark.parametrize("change", [
    dict(Qo=Q2), dict(Ko=K2), dict(Qo=DK), dict(Ko=DY), dict(dgq=0x8400000), dict(dgq=0x8100000), dict(dgk=0x3000000),
    dict(ws=0x1000000), dict(ws=0x4000000), dict(ws=0x8300000 - 256), dict(Qo=_arr(0x5000000, 0x3100000)),
])
def test_backward_refuses_outputs_that_share_memory(lib, change):
    assert _bwd(lib, **change) == 1
    assert b"shares memory" in lib.ttl_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not memory: only where no kernel can be launched")
def test_what_is_taken(lib):
    """Outputs in place of the inputs, column ranges of one matrix, no norm, no rotation: as far as the device."""
    taken = lambda rc: rc not in (0, 1, 2, 3)     # noqa: E731
    cols = lambda base, at: _arr(base + 2 * at, base + 0x100000 + 2 * at)   # noqa: E731
    bare = dict(gq=None, gk=None, dgq=None, dgk=None)
    assert taken(_fwd(lib)) and taken(_bwd(lib)) and taken(_fwd(lib, **bare))
    assert taken(_bwd(lib, Q=None, K=None, ws=None, ws_bytes=0, **bare))
    assert taken(_fwd(lib, Qo=Q2, Ko=K2)) and taken(_bwd(lib, Qo=DY, Ko=DK))
    fused = dict(Q=cols(0x1000000, 0), K=cols(0x1000000, 128), ldq=256, ldk=256, Qo=cols(0x1000000, 0),
                 Ko=cols(0x1000000, 128), ldqo=256, ldko=256)
    assert taken(_fwd(lib, **fused))
    assert taken(_fwd(lib, rot=0, freqs=None)) and taken(_fwd(lib, cu=None, pos=0x7000000))
    assert taken(_fwd(lib, axes=3, pos=0x7000000, pair_axis=AX(0, 0, 0, 1, 1, 1, 2, 2)))


def test_nothing_to_do(lib):
    assert _fwd(lib, T=0) == 0 and _bwd(lib, T=0, accumulate=1) == 0
    assert lib.ttl_head_norm_rotary_bwd_workspace_size(2, 16, 4, 2, 72) == 0
    assert lib.ttl_head_norm_rotary_bwd_workspace_size(2, 16, 4, 2, 64) >= 2 * 64 * 4


def test_binding_refusals(lib):
    import tensor_transformer_layer_way_gb300 as ttl
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    kw = dict(n_q=1, n_kv=1, d=64)
    with pytest.raises(ValueError):
        ttl.Rotary([1.0, 0.5], axes=[0])
    with pytest.raises(ValueError):
        ttl.Rotary([1.0], axes=[-1])
    with pytest.raises(ValueError):
        ttl.head_norm_rotary_fwd([x], [x], ttl.Rotary(ttl.rotary_freqs(64)), **kw)
    with pytest.raises(TypeError):
        ttl.head_norm_rotary_fwd([x.half()], [x], ttl.Rotary(ttl.rotary_freqs(64)), **kw)
    meta = torch.zeros(4, 64, dtype=torch.bfloat16, device="meta")
    from tensor_transformer_layer_way_gb300._binding import _rotary_args
    with pytest.raises(TypeError):
        _rotary_args(None, 4, 64, 1, 1, 1, None, None, 1e-6, None, None)
    with pytest.raises(ValueError):
        _rotary_args(ttl.Rotary([1.0] * 8, axes=[0, 1] * 4), 4, 64, 1, 1, 1, None, None, 1e-6, meta[:1], None)
    with pytest.raises(ValueError):
        _rotary_args(ttl.Rotary([1.0] * 8), 4, 64, 1, 1, 1, meta[0], None, 1e-6, None, None)
    r = ttl.Rotary(ttl.rotary_freqs(32), axes=[0] * 8 + [1] * 4 + [2] * 4)
    assert (r.rot, r.axes) == (32, 3) and ttl.Rotary([]).rot == 0
    assert ttl.rotary_freqs(4, 100.0) == [1.0, 0.1]


@pytest.mark.parametrize("how", ["copy", "deepcopy", "pickle"])
def test_a_copy_of_a_rotary_reads_its_own_arrays(how):
    import copy
    import pickle
    import tensor_transformer_layer_way_gb300 as ttl
    r = ttl.Rotary([1.0, 0.5, -0.25], axes=[0, 1, 1], interleaved=True)
    c = pickle.loads(pickle.dumps(r)) if how == "pickle" else getattr(copy, how)(r)
    assert (c.rot, c.axes, c.interleaved) == (6, 2, True)
    assert list(c._kept[0]) == [1.0, 0.5, -0.25] and list(c._kept[1]) == [0, 1, 1]
    assert (c._freqs, c._pair_axis) == tuple(ctypes.addressof(a) for a in c._kept)
