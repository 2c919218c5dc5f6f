"""The sequences that the kernels make of packed offsets (csrc/kda_seqs.h,
built with g++): valid ones as they are, and of offsets that nobody checked
ranges inside the batch, none of negative length, that a walk over a slot's
sequences leaves after its own tokens."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "kda_seqs.h"
extern "C" {
long seq_start(const int* cu, int n, long T, long tokens, int s) { return kda::Seqs{cu, n, T, tokens}.start(s); }
long seq_end(const int* cu, int n, long T, long tokens, int s) { return kda::Seqs{cu, n, T, tokens}.end(s); }
int seq_from(const int* cu, int n, long T, long tokens, long t) { return kda::Seqs{cu, n, T, tokens}.from(t); }
// tokens that a walk from sequence s on and token `at` on takes before token `hi`, and whether it stays in range
long seq_walk(const int* cu, int n, long T, long tokens, int s, int at, int hi) {
  const kda::Seqs seqs{cu, n, T, tokens};
  long taken = 0;
  const int lo = at;
  for (; s < n; ++s) {
    const kda::Span r = seqs.next(s, &at);
    if (r.start < lo || r.end < r.start || r.end > tokens) return -1;
    if (r.start >= hi) break;
    taken += (r.end < hi ? r.end : hi) - r.start;
  }
  return taken;
}
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("seqs")
    (d / "seqs.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wall", "-I",
                    os.path.join(ROOT, "gated_delta_rule_105_amd", "csrc"), "-o", str(d / "seqs.so"),
                    str(d / "seqs.cpp")], check=True, timeout=300)
    lib = ctypes.CDLL(str(d / "seqs.so"))
    head = [ctypes.c_void_p, ctypes.c_int, ctypes.c_long, ctypes.c_long]
    for name, res, tail in (("seq_start", ctypes.c_long, [ctypes.c_int]), ("seq_end", ctypes.c_long, [ctypes.c_int]),
                            ("seq_from", ctypes.c_int, [ctypes.c_long]),
                            ("seq_walk", ctypes.c_long, [ctypes.c_int] * 3)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = head + tail, res
    return lib


def batch(cu, tokens):
    return (ctypes.c_int32 * len(cu))(*cu), len(cu) - 1, tokens, tokens


def offsets(rng, kind, n, tokens):
    if kind == "valid":
        return [0] + sorted(rng.randint(0, tokens) for _ in range(n - 1)) + [tokens]
    if kind == "saw":
        return [tokens * (i % 2) for i in range(n + 1)]
    if kind == "falling":
        return sorted((rng.randint(0, tokens) for _ in range(n + 1)), reverse=True)
    return [rng.choice([rng.randint(0, tokens), rng.randint(-2 ** 31, 2 ** 31 - 1)]) for _ in range(n + 1)]


@pytest.mark.parametrize("kind", ["valid", "saw", "falling", "anything"])
def test_ranges_stay_in_the_batch(lib, kind):
    rng = random.Random(kind)
    for _ in range(300):
        n, tokens = rng.randint(1, 12), rng.choice([0, 1, 5, 64, 300])
        cu = offsets(rng, kind, n, tokens)
        b = batch(cu, tokens)
        for s in range(n):
            lo, hi = lib.seq_start(*b, s), lib.seq_end(*b, s)
            assert 0 <= lo <= hi <= tokens, (cu, s)
            if kind == "valid":
                assert (lo, hi) == (cu[s], cu[s + 1])
        for t in range(0, tokens + 1, max(1, tokens // 7)):
            first = lib.seq_from(*b, t)
            assert 0 <= first <= n
            if kind == "valid":
                assert all(cu[s] < t for s in range(first)) and (first == n or cu[first] >= t)


@pytest.mark.parametrize("kind", ["valid", "saw", "falling", "anything"])
def test_a_walk_takes_its_slot_at_most(lib, kind):
    rng = random.Random(kind + "walk")
    for _ in range(300):
        n, tokens, slot = rng.randint(1, 40), rng.choice([1, 64, 300]), 64
        cu = offsets(rng, kind, n, tokens)
        b = batch(cu, tokens)
        total = 0
        for lo in range(0, tokens, slot):
            hi = min(lo + slot, tokens)
            s = lib.seq_from(*b, lo)
            at = min(max(lib.seq_end(*b, s - 1), lo), hi) if s > 0 else lo
            taken = lib.seq_walk(*b, s, at, hi)
            assert 0 <= taken <= hi - at, (cu, lo)
            total += taken + at - lo
        if kind == "valid":
            assert total == tokens
