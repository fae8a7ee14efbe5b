"""The line that attention's work is cut along (host arithmetic of csrc/idx_attn.cuh, compiled with
the compiler of the library): what a unit's end takes on it always fits, and does not depend on how
many units there are but through the CTAs that share them."""
import subprocess

import pytest

from sparse_attention_indexer_packed_gb300 import build

PROGRAM = r"""
#include <stdio.h>
#include "idx_attn.cuh"
using namespace idx::attn;
int main() {
  int rows, blocks, nvfp4, drafts, ctas;
  long long units;
  printf("%lld %lld\n", kMaxUnits, kMaxPositions);
  while (scanf("%d %d %d %d %lld %d", &rows, &blocks, &nvfp4, &drafts, &units, &ctas) == 6) {
    const int cost = unit_cost(rows, blocks, nvfp4, drafts, units, ctas);
    // one request of so many units, the most pieces that a call may have
    const int shift = position_shift(1, units, 2 * 65536 + 2, cost);
    printf("%d %lld\n", cost, units * (((2 * 65536 + 2 + (1ll << shift) - 1) >> shift) + cost));
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    at = tmp_path_factory.mktemp("line")
    (at / "line.cu").write_text(PROGRAM)
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I" + build.CSRC, "-o", str(at / "line"),
                    str(at / "line.cu")], check=True, capture_output=True, text=True)

    def run(cases):
        text = "".join(" ".join(str(int(x)) for x in c) + "\n" for c in cases)
        got = [tuple(map(int, line.split())) for line in
               subprocess.run([str(at / "line")], input=text, check=True, capture_output=True, text=True).stdout.splitlines()]
        assert len(got) == len(cases) + 1
        return got[0], got[1:]
    return run


def test_every_units_end_fits_the_line(ask):
    units = sorted({1, 2, 39, 40, 41, 1000, *(2 ** i + d for i in range(10, 19) for d in (-1, 0, 1)), 86255, 86256})
    cases = [(rows, blocks, nvfp4, drafts, u, ctas) for rows in (16, 128) for blocks in (0, 1) for nvfp4 in (0, 1)
             for drafts in (1, 2, 4, 16) for u in units if u <= 1 << 18 for ctas in (1, 76, 152, 192)]
    (most_units, most), got = ask(cases)
    assert most_units == 1 << 18
    for c, (cost, line) in zip(cases, got):
        assert 1 <= cost and (cost + 1) * c[4] <= most and line <= most, c
        assert line * 193 < 2 ** 31


def test_a_units_end_goes_by_units_for_each_cta(ask):
    """(NVFP4, up to 16 rows, the whole cache.)"""
    cases = [(16, 0, 1, 1, u, ctas) for ctas in (19, 38, 76, 152) for u in range(1, 2 * ctas + 1)]
    _, got = ask(cases)
    by_share = {}
    for (*_, u, ctas), (cost, _) in zip(cases, got):
        assert by_share.setdefault(u / ctas, cost) == cost, (u, ctas)
    assert len(set(by_share.values())) == 2


def test_many_lists_lose_no_more_than_the_line_asks(ask):
    """(NVFP4, block lists of four draft rows: 128 positions, or what is left of the line.)"""
    cases = [(16, 1, 1, 4, u, 152) for u in (1, 10000, 86000, 90112, 1 << 17, 1 << 18)]
    (_, most), got = ask(cases)
    for c, (cost, _) in zip(cases, got):
        assert cost == min(128, most // c[4] - 1)
