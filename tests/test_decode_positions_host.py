"""Rows of the RoPE table that a decode split's lanes start from (no GPU needed): the library's own index function,
compiled for the host."""
import subprocess

import pytest

from sub_bit_kv_b200 import _build, lvq, synth
from tests._helpers import make_cfg

PROGRAM = r"""
#include <cstdio>
#include "lvq_common.cuh"
int main() {
  int S, max_ctx, n0;
  while (std::scanf("%d %d %d", &S, &max_ctx, &n0) == 3) {
    lvq::Geo g = {};
    g.S = S;
    g.max_ctx = max_ctx;
    for (int w = 0; w < lvq::kDecodeWarps; ++w)
      for (int t = 0; t < 8; ++t) std::printf("%d ", lvq::decode_first_position(g, n0, w, t));
    std::printf("\n");
  }
}
"""


@pytest.fixture(scope="module")
def positions(tmp_path_factory):
    _build.build()
    d = tmp_path_factory.mktemp("positions")
    (d / "p.cu").write_text(PROGRAM)
    r = subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-I", _build.INCLUDE, "-I", _build.CSRC, str(d / "p.cu"), "-o", str(d / "p")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(rows):
        out = subprocess.run([str(d / "p")], input="".join("%d %d %d\n" % r for r in rows), capture_output=True, text=True)
        return [[int(x) for x in line.split()] for line in out.stdout.splitlines()]

    return run


def test_first_positions_lie_in_the_table(positions):
    """Every split start of layouts short and long: no lane starts past the table's coarse rows, a lane whose
    token can exist starts at its position.  (Without the bound the lanes of a split from token 384 on, in a layout of
    521 positions, started at row 105 of 82.)"""
    cases, rows = [], []
    for S in (0, 4, 5):
        for max_ctx in (9, 17, 100, 464, 521, 600, 1000, 1025, 4109, 32768):
            cfg = make_cfg(synth.WORKLOADS["tiny"], max_ctx=max_ctx)
            cfg.n_sink = S
            coarse = lvq.lvq_cache_layout(cfg).rope_coarse
            last = max_ctx - S - 1                                         # the last coded token a request can have
            for n0 in sorted({0, *range(0, last + 1, 32 if max_ctx < 5000 else 4096), max(0, last // 32 * 32)}):
                cases.append((S, max_ctx, n0, coarse))
                rows.append((S, max_ctx, n0))
    beyond = 0
    for (S, max_ctx, n0, coarse), got in zip(cases, positions(rows)):
        assert len(got) == 15 * 8
        for i, p in enumerate(got):
            want = S + n0 + 32 * (i // 8) + i % 8
            assert 0 <= p and p // 8 < coarse
            assert p == want or want >= max_ctx
            beyond += want // 8 >= coarse
    assert beyond > 0
