"""How an attention call is cut (csrc/kv4_cut.h, built here as host code): the copy that other tests use, and that
each kernel's instances are reached (CPU)."""
import ctypes
import os
import random
import re
import shutil
import subprocess

import pytest

import attention_rows
from w4a4_group_quantized_amd import build

NAMES = ("rows", "share", "sorted", "rt", "tiles", "deep")
WRAPPER = """
#include "kv4_cut.h"
extern "C" void cut(int64_t T, int B, int Hkv, int share, int D, int max_q, int max_kv, int window, int cus, int64_t* out)
{
    const apex4::Cut c = apex4::kv4_cut(T, B, Hkv, share, D, max_q, max_kv, window, cus);
    const int64_t all[] = {c.rows, c.share, c.sorted, c.rt, c.tiles, c.deep, c.blocks};
    for (int i = 0; i < 7; ++i) out[i] = all[i];
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("cut")
    (at / "cut.cpp").write_text(WRAPPER)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, str(at / "cut.cpp"), "-o",
                           str(at / "cut.so")])
    f = ctypes.CDLL(str(at / "cut.so")).cut
    f.argtypes = [ctypes.c_int64] + 8 * [ctypes.c_int] + [ctypes.POINTER(ctypes.c_int64)]

    def call(*args):
        out = (ctypes.c_int64 * 7)()
        f(*args, out)
        return dict(zip(NAMES + ("blocks",), out))
    return call


def draw(rng):
    spread = lambda most: int(2 ** rng.uniform(0, most))  # noqa: E731
    B, Hkv, share = spread(10), rng.choice([1, 2, 4, 8, 32]), rng.choice([1, 2, 4, 7, 8, 16])
    T = min(B + spread(13) - 1, 2 ** 24 - 1)
    max_q = max(-(-T // B), min(T, spread(13)))             # (kept within these by the call)
    return T, B, Hkv, share, rng.choice([64, 128, 256]), max_q, spread(17), rng.choice([0, 0, 1, 300, spread(14)]), 256


def test_copy_and_instances(rule):
    rng, reached = random.Random(5), set()
    for _ in range(20000):
        T, B, Hkv, share, D, max_q, max_kv, window, cus = args = draw(rng)
        c = rule(*args)
        copy = attention_rows.cut(T, B, Hkv * share, Hkv, D, max_q, max_kv, window, cus)
        assert copy == dict(kernel="rows" if c["rows"] else "few", rt=c["rt"], uneven=c["tiles"] == 0,
                            share=bool(c["share"]), deep=bool(c["deep"]), sorted=bool(c["sorted"])), args
        assert 1 <= c["blocks"] <= 2 ** 24 - 1 and (not c["share"] or c["blocks"] <= 2 * cus)
        reached.add(("rows", D, c["rt"], c["tiles"] == 0) if c["rows"] else ("few", D, c["rt"]))
        if c["share"]:
            reached.add(("join", D, c["rt"], c["deep"]))
    few = [(64, 1), (64, 2), (128, 1), (128, 2), (256, 1)]
    # the instances that launch() has, each of them reached
    assert reached == {("few", *x) for x in few} | {("join", *x, d) for x in few for d in (0, 1)} | \
        {("rows", D, 1 if D == 256 else 2, u) for D in (64, 128, 256) for u in (False, True)}


def test_the_library_holds_no_other_instances():
    """Kernels of the attention file by their mangled names, as the host's launch stubs have them."""
    obj = os.path.join(os.path.dirname(build.LIB), "_build", "kv4_attention.hip.o")
    if not os.path.exists(obj):
        pytest.skip("libapex4.so not built here")
    names = subprocess.run(["nm", obj], capture_output=True, text=True, check=True).stdout
    have = set(re.findall(r"__device_stub__rows_kernelILb([01])ELi(\d+)ELi(\d)ELb([01])E", names))
    assert have == {(b, str(D), "1" if D == 256 else "2", u) for b in "01" for D in (64, 128, 256) for u in "01"}
