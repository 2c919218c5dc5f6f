"""The cases of layer_sizes.py get the tiles, slots and steps that they are
there for (csrc/kda_layer.h, built with g++), on a device of 256 compute units."""
import ctypes
import os
import shutil
import subprocess

import pytest

import layer_sizes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "kda_layer.h"
extern "C" {
int forward_tile(int bf16, long tokens, int D) { return kda::conv_forward_tile(bf16, tokens, D); }
int backward_tile(long tokens, int D) { return kda::conv_backward_tile(tokens, D); }
int forward_slots(long tokens, int rows, long T, int packed, int D, int N, int G) {
  const kda::ScanPlan p = kda::plan_scan(tokens, rows, T, packed, D, N, G, 256);
  return p.carry ? (int)p.n_slots : -(int)p.n_slots;
}
int backward_slots(long tokens, int rows, int D, int N, int G) {
  return (int)kda::plan_scan_backward(tokens, rows, D, N, G).n_slots;
}
int step_seqs(long tokens, int D, int N) { return kda::scan_step_seqs(tokens, D, N); }
int norm_steps_of(int tokens, int Hq, int Hk, int d, int rot, int* waves) {
  const int groups = kda::norm_groups(Hq, Hk, kda::norm_head_lanes(d, rot));
  const int steps = kda::norm_steps(tokens, groups, kda::kNormMinWaves);
  *waves = (int)kda::ceil_div(groups, steps);
  return steps;
}
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("plans")
    (d / "plans.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wall", "-I",
                    os.path.join(ROOT, "gated_delta_rule_105_amd", "csrc"), "-o", str(d / "plans.so"),
                    str(d / "plans.cpp")], check=True, timeout=300)
    lib = ctypes.CDLL(str(d / "plans.so"))
    n, i = ctypes.c_long, ctypes.c_int
    lib.forward_tile.argtypes = [i, n, i]
    lib.backward_tile.argtypes = [n, i]
    lib.forward_slots.argtypes = [n, i, n, i, i, i, i]
    lib.backward_slots.argtypes = [n, i, i, i, i]
    lib.step_seqs.argtypes = [n, i, i]
    lib.norm_steps_of.argtypes = [i] * 5 + [ctypes.POINTER(i)]
    return lib


@pytest.mark.parametrize("case", layer_sizes.CONV)
def test_convolution_tiles(lib, case):
    c = layer_sizes.CONV[case]
    tokens = sum(c["lengths"]) if "lengths" in c else c["B"] * c["T"]
    assert (lib.forward_tile(c["dtype"] == "bf16", tokens, c["D"]), lib.backward_tile(tokens, c["D"])) == c["tiles"]


@pytest.mark.parametrize("case", layer_sizes.SCAN)
def test_scan_slots(lib, case):
    c = layer_sizes.SCAN[case]
    packed = "lengths" in c
    tokens, rows = (sum(c["lengths"]), len(c["lengths"])) if packed else (c["B"] * c["T"], c["B"])
    T, G = tokens if packed else c["T"], c.get("G", 1)
    forward = lib.forward_slots(tokens, rows, T, packed, c["D"], c["N"], G)
    assert (abs(forward), lib.backward_slots(tokens, rows, c["D"], c["N"], G)) == c["slots"]
    assert (forward > 0) == c["carry"]


@pytest.mark.parametrize("case", layer_sizes.STEP)
def test_step_sequences(lib, case):
    c = layer_sizes.STEP[case]
    assert lib.step_seqs(c["S"], c["D"], c["N"]) == c["seqs"] and c["S"] % c["seqs"] != 0


@pytest.mark.parametrize("case", layer_sizes.NORM)
def test_norm_steps(lib, case):
    c = layer_sizes.NORM[case]
    tokens = 1
    for n in c["rows"]:
        tokens *= n
    waves = ctypes.c_int(0)
    assert lib.norm_steps_of(tokens, c["Hq"], c["Hk"], c["d"], c["rot"], waves) == c["steps"]
    assert waves.value == c["waves"]
