"""How the head norm and rotation deals out its work, compiled for the host (CPU)."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_transformer_layer_way_gb300", "csrc")


@pytest.fixture(scope="module")
def deal(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("deal")
    src = d / "deal.cpp"
    src.write_text('#include "head_deal.h"\n'
                   'extern "C" void deal(int64_t T, int64_t heads, int d, int resident, int sms, int64_t* out) {\n'
                   "  const ttl::HeadDeal r = ttl::head_deal(T, heads, d, resident, sms);\n"
                   "  out[0] = r.groups;\n  out[1] = r.warps;\n  out[2] = r.blocks;\n  out[3] = ttl::head_lanes(d);\n}\n")
    lib = d / "deal.so"
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).deal
    f.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int64)]

    def call(*a):
        out = (ctypes.c_int64 * 4)()
        f(*a, out)
        return list(out)

    return call


@pytest.mark.parametrize("sms", [1, 19, 76, 148, 152, 160])
@pytest.mark.parametrize("resident", [1, 2])
def test_no_more_blocks_than_the_device_holds(deal, sms, resident):
    rng = random.Random(sms)
    for _ in range(300):
        T, heads, d = int(2 ** rng.uniform(0, 22)), int(2 ** rng.uniform(1, 8)), 16 * rng.randint(1, 16)
        groups, warps, blocks, lanes = deal(T, heads, d, resident, sms)
        assert lanes * 16 >= d and 32 % lanes == 0
        assert groups * (32 // lanes) >= T > (groups - 1) * (32 // lanes)
        assert 1 <= blocks <= resident * min(sms, 152)             # and rows of the workspace for as many
        assert warps <= groups * heads and 0 <= blocks * 8 - warps < 8
        if groups * heads >= resident * min(sms, 152) * 8:
            assert blocks == resident * min(sms, 152)              # all of it, where there is work
