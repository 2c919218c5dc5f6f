"""The cases of block_sizes.py get the slots that they are there for
(csrc/kda_linear.h, built with g++), on a device of 256 compute units, and
what a plan puts into the workspace does not overlap."""
import ctypes
import os
import shutil
import subprocess

import pytest

import block_sizes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "kda_block.h"
#include "kda_linear.h"
extern "C" {
// slot, slots, carry, then the areas' offsets in order and the workspace
void plan(long tokens, int rows, long T, int packed, int H, int Hq, int dk, int dv, int backward, long* out) {
  kda::LinearPlan p = kda::plan_linear(tokens, rows, T, packed, H, 256, dk, dv, backward);
  if (backward) kda::plan_linear_shared(&p, tokens, H, Hq, dk);
  const long v[] = {p.slot, p.n_slots, p.carry, (long)p.end_off, (long)p.adj_off, (long)p.sum_off, (long)p.kind_off,
                    (long)p.dot_q_off, (long)p.dot_k_off, (long)p.slot_dot_off, (long)p.seq_dot_off, (long)p.dq_off,
                    (long)p.dk_off, (long)p.ws_bytes};
  for (int i = 0; i < 14; ++i) out[i] = v[i];
}
void shape(int D, int elem, int* out) {
  const kda::RowShape s = kda::block_norm_shape(D, elem);
  out[0] = s.vec, out[1] = s.lanes, out[2] = s.loads;
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
    lib.plan.argtypes = [n, i, n, i, i, i, i, i, i, ctypes.POINTER(n)]
    lib.shape.argtypes = [i, i, ctypes.POINTER(i)]
    return lib


def plan(lib, tokens, rows, T, packed, H, Hq, dk, dv, backward):
    out = (ctypes.c_long * 14)()
    lib.plan(tokens, rows, T, packed, H, Hq, dk, dv, backward, out)
    return list(out)


@pytest.mark.parametrize("name", block_sizes.LINEAR)
@pytest.mark.parametrize("backward", [0, 1])
def test_slots(lib, name, backward):
    c = block_sizes.LINEAR[name]
    packed = "lengths" in c
    rows = len(c["lengths"]) if packed else c["B"]
    got = plan(lib, block_sizes.tokens(c), rows, c["T"], packed, c["H"], c["Hq"], c["dk"], c["dv"], backward)
    assert tuple(got[:2]) == c["slots"] and got[2] == 1


@pytest.mark.parametrize("tokens,rows,T,packed", [(4096, 1, 4096, 0), (4096, 2, 2048, 0), (5003, 37, 0, 1), (0, 3, 0, 0),
                                                  (64, 64, 1, 0), (10 ** 6, 1, 10 ** 6, 0)])
@pytest.mark.parametrize("H,Hq,dk,dv", [(16, 16, 128, 128), (6, 2, 64, 100), (1, 1, 1, 1), (40, 1, 128, 64)])
def test_slots_cover_the_tokens_and_areas_do_not_overlap(lib, tokens, rows, T, packed, H, Hq, dk, dv):
    for backward in (0, 1):
        slot, n, carry, end, adj, sums, kinds, dot_q, dot_k, slot_dot, seq_dot, dq, dkk, size = plan(
            lib, tokens, rows, T, packed, H, Hq, dk, dv, backward)
        assert slot * n >= tokens and slot * (n - 1) < max(tokens, 1)
        if not carry and n > 1:  # slots are whole rows
            assert not packed and slot % T == 0
        record = (64 if dk <= 64 else 128) * (64 if dv <= 64 else 128) * 4
        used = n if carry else 0
        areas = [(end, used * H * record), (sums, used * H * 8), (kinds, used * 4)]
        if backward:
            areas += [(adj, used * H * record), (dot_q, tokens * H * 4), (dot_k, tokens * H * 4), (slot_dot, n * H * 4),
                      (seq_dot, rows * H * 4)]
            if H != Hq:
                areas += [(dq, tokens * H * dk * 4), (dkk, tokens * H * dk * 4)]
        areas = sorted(a for a in areas if a[1])
        for (at, length), (then, _) in zip(areas, areas[1:] + [(size, 0)]):
            assert at % 256 == 0 and at + length <= then


@pytest.mark.parametrize("elem", [2, 4])
def test_row_shapes_cover_the_channels(lib, elem):
    for D in range(1, 8193):
        s = (ctypes.c_int * 3)()
        lib.shape(D, elem, s)
        vec, lanes, loads = s
        assert D % vec == 0 and vec * lanes * loads >= D and (vec == 1 or vec * elem == 16)
