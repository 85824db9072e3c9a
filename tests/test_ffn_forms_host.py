"""Which kernel instances the dense feed-forward block's sizes take (no GPU):
the plan is host code, compiled here on its own.  Which form runs follows from
a cost estimate, so a change of its table moves sizes between forms; these
tests fail where that leaves an instance without a parity test."""

import ctypes
import math
import os
import random
import shutil
import subprocess

import pytest

import test_gpu_ffn as G
from ffn_form_sizes import SIZES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# the gradients asked for: 0 the forward, 1 dx, 2 dw_gu, 4 dw2
STEP = (0, 7)
ALL = (0, 7, 1, 2, 3, 4, 5, 6)
STEP_AND_ALONE = (0, 7, 1, 2, 4)


@pytest.fixture(scope="module")
def forms(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    lib = str(tmp_path_factory.mktemp("forms") / "ffn_forms.so")
    subprocess.run(
        [cxx, "-std=c++17", "-O2", "-shared", "-fPIC", "-I", os.path.join(
            ROOT, "mixture_experts_expert_top_amd", "csrc"),
         os.path.join(ROOT, "tests", "native", "ffn_forms.cpp"), "-o", lib],
        check=True)
    fn = ctypes.CDLL(lib).ffn_forms
    fn.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.c_char_p,
                                          ctypes.c_int]
    fn.restype = None
    buf = ctypes.create_string_buffer(1024)

    def get(size, wants):
        names = set()
        for w in wants:
            fn(*size, w, buf, len(buf))
            names |= {n for n in buf.value.decode().split(";") if n}
        return names
    return get


def _params(test, names):
    return next(m.args[1] for m in test.pytestmark
                if m.name == "parametrize" and m.args[0] == names)


def test_forms_of_known_sizes(forms):
    """The instances two operator-sized steps are known to run."""
    assert forms((1, 4096, 14336), (0,)) == {
        "fc1 thin 1 blocks 16 rows", "y thin 1 blocks 16 rows"}
    assert forms((8192, 4096, 14336), STEP) == {
        "fc1 256x256x1", "y 256x256x1", "dw 256x256x1", "dact 256x256x1",
        "dx 256x256x1"}


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes_take_the_forms_they_are_there_for(forms, size):
    assert SIZES[size] <= forms(size, STEP_AND_ALONE)


def test_every_form_has_a_parity_test(forms):
    covered = set()
    for s in G.SIZES + G.TALL:
        covered |= forms(s, STEP)
    for s in _params(G.test_ffn_large_products, "T,d,f") + list(SIZES):
        covered |= forms(s, STEP_AND_ALONE)
    rng = random.Random(3)

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    drawn = {}
    for _ in range(40000):
        s = (log(1, 8192), max(8, log(8, 4096) // 8 * 8),
             max(8, log(8, 14336) // 8 * 8))
        for n in forms(s, ALL):
            drawn.setdefault(n, s)
    missing = {n: s for n, s in drawn.items() if n not in covered}
    assert not missing
