"""How the products of an orthogonalisation are cut into tiles (CPU only): the sizes that the GPU
tests run reach every kind of tile and every way to split them, for each product."""
import os
import re
import shutil
import subprocess

import pytest

import muon_error_ref as E
import zero_partitioned_optimizer_amd as Z
from zero_partitioned_optimizer_amd import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KINDS = {"few", "mid", "two", "wide"}
# the tiles that a product splits, in one part or two ("two"), behind whole ones or alone
SPLITS = {"wide+split+two", "wide+split+whole", "wide+split+two+whole"}


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("plan") / "plans")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", B.CSRC,
                    os.path.join(ROOT, "tests", "c", "orth_plans.cpp"), "-o", exe], check=True)

    def run(sizes):
        out = subprocess.run([exe, *(str(v) for s in sizes for v in s)], check=True, capture_output=True, text=True).stdout
        return {tuple(int(v) for v in f[:3]): f[3:] for f in (line.split() for line in out.splitlines())}
    return run


def test_every_way_is_among_the_tested_sizes(plans):
    got = {k: set() for k in ("gram flat", "gram tall", "square", "update flat", "update tall")}
    for (_, r, c), ways in plans(E.PLAN_SIZES).items():
        side = " tall" if r > c else " flat"
        for op, way in zip(("gram" + side, "square", "update" + side), ways):
            got[op].add(way)
    for op, ways in got.items():
        assert KINDS <= ways, (op, KINDS - ways)
    # a single tile split alone is the Gram product's of a long narrow matrix only, and the
    # update has whole tiles before those that it splits
    assert {"wide+split"} | SPLITS <= got["gram flat"] and {"wide+split"} | SPLITS <= got["gram tall"]
    assert SPLITS <= got["square"]
    for op in ("update flat", "update tall"):
        assert SPLITS - {"wide+split+two"} <= got[op], op


def test_fastest_kinds_as_measured(plans):
    """Sizes whose kinds were all timed: the estimate takes the fastest (within 1%)."""
    want = {(1, 768, 768): "few few few", (12, 768, 2304): "mid mid two", (1, 4096, 4096): "split split wide",
            (1, 11008, 4096): "split split wide", (1, 1000, 4096): "few few mid", (4, 2304, 4096): "wide wide split",
            (1, 130, 5000): "few few few", (24, 64, 768): "few few mid", (1, 64, 11008): "few few few",
            (3, 1000, 1000): "few few mid", (40, 700, 500): "two two wide", (1, 2304, 4096): "mid mid wide",
            (6, 1500, 1500): "two two wide", (1, 5000, 2000): "split mid wide", (2, 4200, 5600): "split split wide"}
    for size, ways in plans(want).items():
        assert ["split" if "split" in w else w for w in ways] == want[size].split(), size


def test_workspace_holds_what_the_plan_needs(plans):
    """Two parts of 256 tiles of partial sums where any product splits, and none otherwise."""
    def up(n):
        return -(-n // 128) * 128
    for (b, r, c), ways in plans(E.PLAN_SIZES).items():
        R, C, m = up(r), up(c), min(up(r), up(c))
        each = 8 * R * C + 8 * m * m + 8 * m + 8 * 256
        part = 2 * 256 * 256 * 256 * 4 if any("split" in w for w in ways) else 0
        assert Z.zero_orthogonalize_workspace_bytes(b, r, c) == b * each + part


def test_lanes_that_exchange_rows_through_lds_meet():
    """Between a wave's writes to its part of LDS and other lanes' reads of them stands a fence, and
    one before the next run's writes."""
    text = open(os.path.join(B.CSRC, "orth_kernels.hip")).read()
    assert re.search(r'void meet_lanes\(\) \{\s*__builtin_amdgcn_fence\(__ATOMIC_ACQ_REL, "wavefront", "local"\);\s*'
                     r'__builtin_amdgcn_wave_barrier\(\);', text)
    finish = text[text.index("struct Finish {"):text.index("// products\n")]
    assert finish.count("meet_lanes();") == 3
