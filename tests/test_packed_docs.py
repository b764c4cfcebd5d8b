"""The look-up of a token's document, compiled for the host: what it answers for bounds of every kind (CPU).

The kernels ask for the documents of every row of a 128-token tile, rows behind the pack's last token among them, and
use the answer as a range of rows to read and write: it has to stay inside [0, T) whatever the bounds hold.
"""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_transformer_layer_way_gb300", "csrc")


@pytest.fixture(scope="module")
def look_up(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("docs")
    src = d / "docs.cpp"
    src.write_text('#include "pack_docs.h"\n'
                   'extern "C" void docs(const int32_t* cu, int batch, int T, int tok, int* out) {\n'
                   "  const ttl::DocRange r = ttl::doc_of(cu, batch, T, tok);\n  out[0] = r.lo;\n  out[1] = r.hi;\n}\n"
                   'extern "C" uint64_t wait_ns(int64_t steps) { return ttl::pack_wait_ns(steps); }\n')
    lib = d / "docs.so"
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    host = ctypes.CDLL(str(lib))
    f = host.docs
    host.wait_ns.restype, host.wait_ns.argtypes = ctypes.c_uint64, [ctypes.c_int64]

    def call(cu, T, tok):
        out = (ctypes.c_int * 2)()
        f((ctypes.c_int32 * len(cu))(*cu), len(cu) - 1, T, tok, out)
        return out[0], out[1]

    call.wait_ns = host.wait_ns
    return call


def _tile_rows(T):
    return range((T + 127) // 128 * 128)


@pytest.mark.parametrize("T,cu", [(200, [40, 5000]), (200, [0, 100, 5000]), (129, [0, 300]), (1, [0, 2]), (127, [-5, 127, 128]),
                                  (3000, [0, 1000, 50000]), (200, [300, 400]), (200, [150, 250, 260]), (256, [0, 1 << 30])])
def test_rows_behind_the_pack_are_in_no_document(look_up, T, cu):
    for tok in _tile_rows(T):
        lo, hi = look_up(cu, T, tok)
        if tok >= T:
            assert hi <= lo
        elif hi > lo:
            assert 0 <= lo <= tok < hi <= T


def test_any_bounds_stay_inside_the_pack(look_up):
    rng = random.Random(5)
    for _ in range(300):
        T = rng.randint(1, 400)
        cu = [rng.randint(-20, T + 300) for _ in range(rng.randint(1, 12))]
        for tok in _tile_rows(T):
            lo, hi = look_up(cu, T, tok)
            assert hi <= lo or 0 <= lo <= tok < hi <= T, (T, cu, tok)


def test_valid_bounds(look_up):
    rng = random.Random(6)
    for _ in range(100):
        T = rng.randint(1, 400)
        cu = sorted(rng.randint(0, T) for _ in range(rng.randint(2, 12)))
        for tok in _tile_rows(T):
            want = next(((a, b) for a, b in zip(cu, cu[1:]) if a <= tok < b), None)
            lo, hi = look_up(cu, T, tok)
            assert (lo, hi) == want if want else hi <= lo


@pytest.mark.parametrize("tokens,grp", [(1, 1), (8192, 4), (65536, 16), (4 << 20, 64)])
def test_a_wait_may_take_as_long_as_an_item(look_up, tokens, grp):
    """Some warps wait for a whole item: one step of 1.6 us per query tile and head of the group for the longest."""
    steps = (tokens + 127) // 128 * grp
    ns = look_up.wait_ns(steps)
    assert ns >= 2_000_000_000 and ns >= 5 * 1600 * steps
    assert ns <= 2_000_000_000 + 100_000 * steps          # and what nothing ends does end
