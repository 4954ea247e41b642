"""Unit slots of packed sequences, as the kernels compute them (the host side of ragged.cuh, no GPU needed)."""
import os
import subprocess

import pytest

from factorized_sparse_self_b200 import build

MAX_ROWS = 0x7FFF0000  # most query rows of a call

SOURCE = r"""
#include <cstdio>
#include "ragged.cuh"
using namespace st::rag;
// mult BM total S cu[0..S] -> a line "sequence tile" for every slot
int main() {
  int mult, BM, total, S;
  while (std::scanf("%d %d %d %d", &mult, &BM, &total, &S) == 4) {
    int cu[64];
    for (int i = 0; i <= S; ++i)
      if (std::scanf("%d", cu + i) != 1) return 1;
    Geo g = {};
    g.S = S;
    g.total = total;
    const long long n = slot_count(g, mult, BM);
    std::printf("%lld\n", n);
    for (long long x = 0; x < n; ++x) {
      int s = 0;  // the last one that starts at or before the slot, the first one otherwise
      for (int i = 0; i < S; ++i)
        if (slot_first(cu[i], i, mult, BM) <= x) s = i;
      std::printf("%d %d\n", s, slot_tile((int)x, slot_first(cu[s], s, mult, BM), BM));
    }
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def slots(tmp_path_factory):
    at = tmp_path_factory.mktemp("slots")
    (at / "slots.cu").write_text(SOURCE)
    subprocess.check_call([build.NVCC, "-std=c++17", "-I" + build.CSRC, "-I" + os.path.join(build.ROOT, "include"),
                           *build.ARCH, "-o", str(at / "slots"), str(at / "slots.cu")])

    def run(mult, BM, cu, total):
        text = " ".join(map(str, [mult, BM, total, len(cu) - 1, *cu]))
        out = subprocess.run([str(at / "slots")], input=text, capture_output=True, text=True, check=True).stdout.split()
        v = list(map(int, out[1:]))
        assert len(v) == 2 * int(out[0])
        return list(zip(v[::2], v[1::2]))

    return run


@pytest.mark.parametrize("BM", [16, 64, 128, 256])
@pytest.mark.parametrize("mult", [1, 3, 4, 5, 32])
@pytest.mark.parametrize("lead", [0, 1, 3, 63, 64, 200, 300, 1000, 4097])
def test_every_tile_of_every_sequence_has_one_slot(slots, lead, mult, BM):
    for lens, tail in (([100, 100], 0), ([1], 0), ([0, 700, 0, 0, 3, 257], 5), ([0], 9), ([64] * 20, 300)):
        cu = [lead]
        for n in lens:
            cu.append(cu[-1] + n)
        want = {(s, t) for s, n in enumerate(lens) for t in range(-(-n * mult // BM))}
        got = []
        for s, t in slots(mult, BM, cu, cu[-1] + tail):
            assert t >= 0, "a tile before its sequence's rows"
            if t * BM < lens[s] * mult:
                got.append((s, t))
            else:  # past the rows of any sequence that starts where this one does
                assert t * BM >= lens[s] * mult and t * BM < 2 ** 31
        assert sorted(got) == sorted(want)


def test_slots_of_no_sequence_lie_past_the_largest_one(slots):
    for BM in (16, 64, 128, 256):
        first = slots(1, BM, [4000, 4001], 4001)[0]
        assert first[0] == 0 and MAX_ROWS <= first[1] * BM < 2 ** 31


def test_lengths_that_decrease_name_no_tile_before_a_sequence(slots):
    """Such lengths are not allowed, but they must not lead outside the tensors."""
    for cu in ([500, 100, 600], [0, 900, 30, 20], [700, 0, 0]):
        for s, t in slots(4, 128, cu, 1000):
            assert t >= 0
