"""The sizes of dense_dispatch against the rule that chooses a product's kernel, compiled for the host: a kernel that a
changed rule takes out of the tests' reach is missed here."""
import ctypes
import os
import shutil
import subprocess

import pytest

import dense_dispatch
from conftest import ROOT

SHIM = """
#include "dense_rule.h"
extern "C" int rule_tile(int I, int J, int K, int format, int *parts) { return moe::choose_tile(I, J, K, format, parts); }
extern "C" int rule_few(int I, int J, int format, int h8) { return moe::few_rows(I, J, format, h8 != 0); }
extern "C" size_t rule_part_bytes(size_t I, size_t J) { return moe::part_bytes(I, J); }
"""


class Rule:
    def __init__(self, lib):
        self.lib = lib
        lib.rule_part_bytes.restype = ctypes.c_size_t
        lib.rule_part_bytes.argtypes = [ctypes.c_size_t, ctypes.c_size_t]

    def parts(self, I, J, K, f):
        n = ctypes.c_int()
        return self.lib.rule_tile(I, J, K, f, ctypes.byref(n)), n.value

    def tile(self, I, J, K, f):
        t, n = self.parts(I, J, K, f)
        return t, n > 1

    def few(self, I, J, f, h8):
        return bool(self.lib.rule_few(I, J, f, h8))


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    compiler = shutil.which("g++") or shutil.which("c++") or "/opt/rocm/llvm/bin/clang++"
    d = tmp_path_factory.mktemp("rule")
    (d / "rule.cpp").write_text(SHIM)
    subprocess.run([compiler, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "routed_expert_ffn_router_amd", "csrc"),
                    str(d / "rule.cpp"), "-o", str(d / "rule.so")], check=True)
    return Rule(ctypes.CDLL(str(d / "rule.so")))


@pytest.mark.parametrize("op,operands", dense_dispatch.CASES)
def test_every_kernel_has_a_size(rule, op, operands):
    want = {(t, parts) for t in range(dense_dispatch.TILES) for parts in (False, True)}
    assert {dense_dispatch.place(rule, op, operands, *size) for size in dense_dispatch.CASES[op, operands]} == want


def test_every_operator_is_there():
    forward = {(op, f) for op in ("matmul", "gated", "gated8") for f in dense_dispatch.FORMATS}
    assert set(dense_dispatch.CASES) == forward | {(op, f) for op in ("dx", "dw") for f in ("bf16", "f32")}


def test_parts_fit_their_room(rule):
    """The sums of the parts lie within what the workspace keeps for them, at every size."""
    for f in range(3):
        for I in (1, 33, 64, 1000, 4096, 65536):
            for J in (8, 136, 4096, 1 << 20):
                for K in (8, 520, 8192, 65536, 1 << 20):
                    t, n = rule.parts(I, J, K, f)
                    assert 0 <= t < dense_dispatch.TILES and 1 <= n <= 16
                    assert n == 1 or n * I * J * 4 <= rule.lib.rule_part_bytes(I, J)
                    assert n == 1 or 4 * n <= -(-K // {0: 64, 1: 32, 2: 128}[f])     # no part without steps
