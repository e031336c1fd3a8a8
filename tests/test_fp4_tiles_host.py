"""Which tiles a product of 4-bit matrices takes, compiled for the host: what the
kernels need of them, and that the GPU's tests have a shape for every kind."""

import ctypes
import os
import subprocess

import pytest

from quantized_expert_ffn_router_gb300.build import CSRC
from test_gpu_fp4_tiles import SHAPES

SMS = 152
SOURCE = r"""
#include <set>
#include "ft_fp4_tiles.h"

static int64_t kind(int64_t T, int64_t N, int64_t K, int sms, bool* fits) {
  const int steps = static_cast<int>((K + ft::kStep - 1) / ft::kStep);
  const ft::Tiles t = ft::choose_tiles(T, N, steps, sms);
  const int64_t tiles = ft::tiles_of(T, N, t.width, t.pair), places = sms / (t.pair * t.slices);
  const int64_t waves = std::min<int64_t>(3, (tiles + places - 1) / places);
  *fits = (t.pair == 1 || t.pair == 2) && t.width >= 16 && t.width <= ft::kMaxWidth &&
          (T <= 64 ? t.width % 16 == 0 && t.width >= T : t.width % 64 == 0) && t.slices >= 1 && t.slices <= 8 &&
          t.slices <= steps && (t.slices == 1 || (t.pair == 1 && tiles <= places)) && (t.pair == 1 || T > 64);
  return ((t.pair * 1000 + t.width) * 10 + t.slices) * 10 + waves;
}

extern "C" int64_t kind_of(int64_t T, int64_t N, int64_t K, int sms) {
  bool fits;
  const int64_t k = kind(T, N, K, sms, &fits);
  return fits ? k : -1;
}

// The kinds of all sizes on a grid of steps of `by`; -1 where one does not fit.
extern "C" int kinds(int sms, double by, int64_t* out, int most) {
  std::set<int64_t> seen;
  bool fits;
  for (double T = 1; T < 20000; T = std::max(T + 1, T * by))
    for (double N = 1; N < 140000; N = std::max(N + 1, N * by))
      for (double K = 16; K < 20000; K = std::max(K + 16, K * by)) {
        const int64_t k = kind(static_cast<int64_t>(T), static_cast<int64_t>(N), static_cast<int64_t>(K), sms, &fits);
        seen.insert(fits ? k : -1);
      }
  int n = 0;
  for (const int64_t k : seen)
    if (n < most) out[n++] = k;
  return n;
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    at = tmp_path_factory.mktemp("tiles")
    src, so = at / "tiles.cpp", at / "tiles.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(os.fspath(so))
    lib.kind_of.restype = ctypes.c_int64
    lib.kind_of.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int]
    lib.kinds.argtypes = [ctypes.c_int, ctypes.c_double, ctypes.c_void_p, ctypes.c_int]
    return lib


def kinds(rule, sms, by):
    out = (ctypes.c_int64 * 512)()
    return set(out[:rule.kinds(sms, by, out, 512)])


def test_the_gpu_tests_have_a_shape_of_every_kind(rule):
    missing = kinds(rule, SMS, 1.13) - {rule.kind_of(*s, SMS) for s in SHAPES}
    assert not missing, sorted(missing)


@pytest.mark.parametrize("sms", [1, 2, 7, 64, 148, 160])
def test_tiles_fit_the_kernels_whatever_the_number_of_sms(rule, sms):
    assert -1 not in kinds(rule, sms, 1.3)


def test_sizes_at_the_ends(rule):
    for T in (1, 64, 65, (1 << 31) - 1024):
        for N in (1, 129, (1 << 31) - 1024):
            for K in (16, 272, (1 << 31) - 16):
                assert rule.kind_of(T, N, K, SMS) > 0


def test_kinds_that_were_measured(rule):
    for shape, kind in (((2048, 4096, 4096), (2, 256, 1, 2)), ((777, 2560, 2560), (1, 128, 1, 1)), ((300, 300, 8192), (1, 64, 8, 1)),
                        ((64, 2560, 2048), (1, 64, 1, 1))):
        p, w, s, n = kind
        assert rule.kind_of(*shape, SMS) == ((p * 1000 + w) * 10 + s) * 10 + n
