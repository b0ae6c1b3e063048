"""How a sweep cuts a head's weights into tiles, compiled as the host code that it is (no GPU needed)."""
import os
import random
import subprocess

import pytest

from speculative_decoding_verify_lm_gb300 import build as B

MAIN = """
#include <cstdio>
#include "wf_tiles.cuh"
int main() {
    int v, slots, mt, pair, kept;
    while (std::scanf("%d %d %d %d %d", &v, &slots, &mt, &pair, &kept) == 5) {
        const wf::Tiles t = wf::tiles_of(v, slots, mt, wf::tile_step(pair, kept));
        std::printf("%d %d %d %d\\n", t.num_n, t.bn, t.nbig, t.step);
    }
}
"""


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    d = tmp_path_factory.mktemp("tiles")
    (d / "main.cc").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", B.CSRC, "-x", "c++", str(d / "main.cc"), "-o", str(d / "tiles")],
                   check=True)

    def run(cases):
        out = subprocess.run([str(d / "tiles")], input="\n".join(" ".join(map(str, c)) for c in cases),
                             capture_output=True, text=True, check=True).stdout.split("\n")
        return [tuple(map(int, ln.split())) for ln in out if ln]

    return run


def test_tiles(tiles):
    """Every id in one tile, no tile empty, heights that the products' forms take, starts that tensor copies take."""
    rng = random.Random(5)
    cases = [(v, slots, mt, pair, kept) for v in list(range(1, 1400)) + [32000, 151936, 123478, 2 ** 31 - 300]
             for slots, mt, pair in ((152, 1, 0), (76, 1, 1), (76, 5, 1), (3, 64, 1)) for kept in (0, 1)]
    cases += [(int(2 ** rng.uniform(0, 31)) - 300 if i % 9 == 0 else rng.randint(1, 300000), rng.randint(1, 160),
               rng.randint(1, 64), rng.randint(0, 1), rng.randint(0, 1)) for i in range(20000)]
    cases = [c for c in cases if c[0] >= 1]
    got = tiles(cases)
    assert len(got) == len(cases)
    for (v, slots, mt, pair, kept), (num_n, bn, nbig, step) in zip(cases, got):
        small = bn - step
        assert 1 <= nbig <= num_n and 64 <= bn <= 256 and (nbig == num_n or small >= 64)
        of = 32 if pair or kept else 16
        assert bn % of == 0 and (nbig == num_n or small % of == 0)
        rows = nbig * bn + (num_n - nbig) * small
        last = bn if nbig == num_n else small
        assert rows - last < v <= rows


def test_a_pairs_products_have_n_in_steps_of_32(tiles):
    """Sizes that steps of 16 cut into tiles of 240 rows or 80."""
    for v, slots, mt in ((151936, 76, 5), (32000, 76, 8), (255, 76, 2), (123478, 76, 5), (4999, 76, 1)):
        (num_n, bn, nbig, step), = tiles([(v, slots, mt, 1, 0)])
        assert step == 32 and bn % 32 == 0
