"""Where the kernels for operands of any alignment read: every piece of a row of
activations, codes, scales and zero points lies inside the row, whatever its
length, and has what it is read for.  grouped_bounds.h, the arithmetic that the
kernels run, compiled for the host.  CPU only."""
import ctypes
import shutil
import subprocess

import pytest

from dense_gemm_row_amd import build

SOURCE = r"""
#include "grouped_bounds.h"
using namespace gemm::grouped;
static int bad;
static void check(bool ok) { bad += !ok; }

// The general kernels' pieces of `per` values across a row of `total` (tiles of
// `side`) and along one.
extern "C" int across(int total, int per, int side) {
  bad = 0;
  for (int n0 = 0; n0 < total; n0 += side)
    for (int n = 0; n < side; n += per) {
      const int rows = total - n0, cut = piece_early(rows - n, per), start = n0 + n - cut;
      check(cut >= 0 && start >= 0 && start + per <= total);
      for (int u = 0; u < per && n + u < rows; ++u) check(u + cut < per);
    }
  return bad;
}
extern "C" int along(int K, int per) {
  bad = 0;
  for (int64_t k = 0; k < K; k += per) {
    const int gone = piece_early(K - k, per);
    check(gone >= 0 && k - gone >= 0 && k - gone + per <= K);
    for (int u = 0; u < per && k + u < K; ++u) check(u + gone < per);
  }
  return bad;
}

// The few-row 4-bit products' reads of a row: spans of SPAN k dealt to KW wave
// rows, DEPTH ahead, GB k a scale.
template <int KW, int SPAN>
static int spans_of(int K, int GB, int depth) {
  const int ng = (K + GB - 1) / GB, padded = (K + 31) / 32 * 32, groups = SPAN / GB;
  const int spans = ((K + SPAN - 1) / SPAN + KW - 1) / KW;
#ifdef PLANTED
  const int past = K;
#else
  const int past = past_spans<SPAN>(K);
#endif
  const bool pieces = K >= 8 && ng >= groups;
  bad = 0;
  for (int turn = 0; turn < spans; ++turn) {
    int seen = 0;
    for (int part = 0; part < KW; ++part)
      for (int i = 0; i < spans + depth; ++i) {
        const int k0 = span_start<KW, SPAN>(i, spans, turn, part, past);
        check(k0 >= 0);
        if (i >= spans) check(k0 >= K);
        if (k0 < K) seen += K - k0 < SPAN ? K - k0 : SPAN;
        for (int k = k0; k < k0 + SPAN; k += 32) {  // (a lane's codes, aligned)
          const int at = code_byte(k, padded);
          check(at >= 0 && at % 16 == 0 && at + 16 <= padded / 2);
          if (k < K) check(at == k / 2);
        }
        for (int h = 0; h < groups; ++h) {  // (scales and zero points one by one)
          const int at = piece_start(k0 / GB + h, ng, 1);
          check(at >= 0 && at < ng);
          if (k0 / GB + h < ng) check(at == k0 / GB + h);
        }
        if (!pieces) continue;
        const int s = piece_start(k0 / GB, ng, groups);
        check(s >= 0 && s + groups <= ng);
        for (int h = 0; h < groups && k0 / GB + h < ng; ++h) check(k0 / GB + h - s < groups);
        for (int k = k0; k < k0 + SPAN; k += 8) {
          const int x = piece_start(k, K, 8);
          check(x >= 0 && x + 8 <= K);
          for (int u = 0; u < 8 && k + u < K; ++u) check(k + u - x < 8);
        }
      }
    check(seen == K);
  }
  return bad;
}
extern "C" int spans(int K, int GB, int span, int kw, int depth) {
  if (span == 256) return kw == 1 ? spans_of<1, 256>(K, GB, depth) : kw == 2 ? spans_of<2, 256>(K, GB, depth)
                          : kw == 4 ? spans_of<4, 256>(K, GB, depth) : spans_of<8, 256>(K, GB, depth);
  return kw == 1 ? spans_of<1, 128>(K, GB, depth) : kw == 2 ? spans_of<2, 128>(K, GB, depth) : spans_of<4, 128>(K, GB, depth);
}
"""
LENGTHS = [*range(1, 700), 1000, 1001, 2040, 2047, 2048, 2049, 4095, 4097]


def compiled(folder, *flags):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    src, out = folder / "reads.cc", folder / "reads.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", *flags, "-I", build.CSRC, str(src), "-o", str(out)], check=True)
    return ctypes.CDLL(str(out))


@pytest.fixture(scope="module")
def reads(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("reads"))


@pytest.mark.parametrize("per", [4, 8])
def test_pieces_of_the_general_kernels(reads, per):
    for n in LENGTHS:
        if n >= per:  # (shorter rows are read by element)
            assert reads.along(n, per) == 0, n
            for side in (64, 128):
                assert reads.across(n, per, side) == 0, (n, side)


@pytest.mark.parametrize("depth", [2, 4])
@pytest.mark.parametrize("span, kw", [(256, 1), (256, 2), (256, 4), (256, 8), (128, 1), (128, 2), (128, 4)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_spans_of_the_4_bit_products(reads, group, span, kw, depth):
    for K in LENGTHS:
        assert reads.spans(K, group, span, kw, depth) == 0, K


def test_the_check_sees_a_span_that_begins_at_the_end(tmp_path):
    """(A lane's codes there are not a whole aligned 32 k, and may lie past the row.)"""
    planted = compiled(tmp_path, "-DPLANTED")
    assert planted.spans(2047, 32, 256, 8, 4) > 0
