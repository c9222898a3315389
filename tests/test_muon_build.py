"""Build-level checks of the norms' and the matrix step's kernels (CPU only): no private
memory, loads to LDS that wait for their descriptors, headers that are plain C."""
import os
import re
import shutil
import subprocess

import pytest

from test_layer_build import HIPCC, ROOT, _sgprs


def _compile(tmp_path, source, *more):
    from zero_partitioned_optimizer_amd import build as B
    flags = [f for f in B.HIPCC_FLAGS if f not in ("-fPIC", "-shared")]
    cmd = [B.hipcc(), *flags, "-I", os.path.join(ROOT, "include"), "-I", B.CSRC, *more, os.path.join(B.CSRC, source)]
    return subprocess.run(cmd, capture_output=True, text=True, check=True).stderr


@pytest.mark.skipif(not HIPCC, reason="hipcc not available")
@pytest.mark.parametrize("source,kernel", [("norm_kernels.hip", "k_norm_grad"), ("muon_kernels.hip", "k_update"),
                                           ("orth_kernels.hip", "k_orth")])
def test_kernels_use_no_scratch(tmp_path, source, kernel):
    out = _compile(tmp_path, source, "-c", "-o", str(tmp_path / "k.o"), "-Rpass-analysis=kernel-resource-usage")
    names = re.findall(r"Function Name: (\S+)", out)
    scratch = [int(x) for x in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", out)]
    assert names and len(names) == len(scratch)
    assert any(kernel in n for n in names)
    assert not [(n, s) for n, s in zip(names, scratch) if s != 0]


@pytest.mark.skipif(not HIPCC, reason="hipcc not available")
def test_loads_to_lds_wait_for_their_descriptors(tmp_path):
    """Five wait states between a vector instruction that writes a scalar register and the load
    to LDS that reads it, which the compiler does not see to for inline assembly; and none
    between m0's write and the load that uses it is left out."""
    out = tmp_path / "k.s"
    _compile(tmp_path, "orth_kernels.hip", "--cuda-device-only", "-S", "-o", str(out))
    before, loads, bad = [], 0, []
    for line in out.read_text().splitlines():
        line = line.split(";")[0].strip()
        if line.endswith(":"):              # a block begins: what ran before it is not known
            before = ["block"]
            continue
        if not line or line.startswith("."):
            continue
        if line.startswith("buffer_load") and line.endswith(" lds"):
            loads += 1
            assert before[-1].startswith("s_nop") and " m0," in before[-2], before[-3:]
            reads, states = _sgprs(line), 0
            for prev in reversed(before):
                if states >= 5:
                    break
                if prev == "block" or prev.startswith("v_") and _sgprs(",".join(prev.split(",")[:2])) & reads:
                    bad.append((states, prev, line))
                    break
                states += int(prev.split()[1], 0) + 1 if prev.startswith("s_nop") else 1
        before = before[-16:] + [line]
    assert loads >= 40
    assert not bad, (len(bad), bad[:4])


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_headers_are_plain_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "zero_layer.h"\n#include "zero_muon.h"\n'
                   "_Static_assert(sizeof(zero_norm_args) == 128, \"\");\n"
                   "_Static_assert(sizeof(zero_norm_grad_args) == 152, \"\");\n"
                   "_Static_assert(sizeof(zero_muon_momentum_args) == 64, \"\");\n"
                   "_Static_assert(sizeof(zero_muon_update_args) == 56, \"\");\n"
                   "_Static_assert(sizeof(zero_orthogonalize_args) == 120, \"\");\n"
                   "int (*f)(const zero_norm_args*, void*) = zero_norm_forward;\n"
                   "int (*g)(const zero_orthogonalize_args*, void*) = zero_orthogonalize;\n")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), "-c", str(src),
                    "-o", str(tmp_path / "h.o")], check=True)
