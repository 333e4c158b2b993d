"""The choice among the FP8 projection's kernels: what each listed size runs, and that the list has them all."""
import ctypes
import math
import os
import random
import subprocess

import pytest

from tests.linear_choices import CHOICES

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "precision_moe_expert_amd", "csrc")
SHIM = """
#include "linear_choice.h"
using namespace moe;
// out: kind (0 few, 1 batch, 2 tile) and its three numbers
extern "C" void one(int64_t m, int64_t n, int kt, int cols, int* out) {
  const LinChoice c = lin_choose(m, n, kt, cols != 0);
  if (!cols && lin_is_few(m, kt)) { out[0] = 0; out[1] = lin_few_waves(kt); out[2] = out[3] = 0; return; }
  if (!cols && lin_is_batch(m, kt)) { out[0] = 1; out[1] = m <= 16 ? 1 : 2; out[2] = lin_batch_cols(n); out[3] = 0; return; }
  out[0] = 2; out[1] = c.shape; out[2] = c.splits > 1; out[3] = c.halved > 0;
}
// d_x and d_w in one launch: 0 no, 1 d_x's product first, 2 d_w's; whether the second's last round is in halves
extern "C" void both(int64_t M, int64_t K, int64_t N, int* out) {
  const int kx = (int)((N + 127) / 128), kw = (int)((M + 127) / 128);
  out[0] = out[1] = 0;
  if (lin_is_few(M, kx)) return;
  const LinChoice cx = lin_is_batch(M, kx) ? LinChoice{LIN_BATCH, 1, 0} : lin_choose(M, K, kx, false);
  if (!lin_joined(cx, lin_choose(N, K, kw, true))) return;
  const int nx = lin_tiles(M, K, kLinShapes[0]), nw = lin_tiles(N, K, kLinShapes[0]);
  out[0] = kw > kx ? 2 : 1;
  out[1] = (kw > kx ? lin_joined_halves(nw, kw, nx, kx) : lin_joined_halves(nx, kx, nw, kw)) > 0;
}
"""


@pytest.fixture(scope="module")
def chosen(tmp_path_factory):
    """chosen(M, K, N) -> the kernels of (forward, d_x, d_w, both gradients) as in CHOICES."""
    d = tmp_path_factory.mktemp("choice")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC,
                           str(d / "shim.cpp"), "-o", str(d / "shim.so")])
    L = ctypes.CDLL(str(d / "shim.so"))
    L.one.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    L.both.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_void_p]

    def one(m, n, c, cols):
        o = (ctypes.c_int * 4)()
        L.one(m, n, -(-c // 128), cols, o)
        return ("few", o[1]) if o[0] == 0 else ("batch", o[1], o[2]) if o[0] == 1 else ("tile", o[1], bool(o[2]), bool(o[3]))

    def all_of(M, K, N):
        o = (ctypes.c_int * 2)()
        L.both(M, K, N, o)
        return (one(M, N, K, 0), one(M, K, N, 0), one(N, K, M, 1),
                (None, ("dx", bool(o[1])), ("dw", bool(o[1])))[o[0]])

    return all_of


def _outcomes(c):
    """What a size's calls run, told apart by the operands' scales; a joined launch in place of its two products."""
    return {("rows", c[0])} | ({("both", c[3])} if c[3] else {("rows", c[1]), ("cols", c[2])})


def test_listed_sizes(chosen):
    for size, want in CHOICES:
        assert chosen(*size) == want, size


def test_the_list_has_every_choice(chosen):
    have = set().union(*(_outcomes(c) for _, c in CHOICES))
    rng = random.Random(0)
    for _ in range(30000):
        M, K, N = (int(round(math.exp(rng.uniform(math.log(a), math.log(b))))) for a, b in ((1, 8192), (1, 1152), (1, 1152)))
        size = (M, 16 * K, 16 * N)
        assert _outcomes(chosen(*size)) <= have, size
