"""Build-level checks of the layer operators (CPU only): their kernels use no private
memory, and the header is plain C."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") is not None or os.path.exists("/opt/rocm/bin/hipcc")


@pytest.mark.skipif(not HIPCC, reason="hipcc not available")
@pytest.mark.parametrize("source,kernel", [("linear_kernels.hip", "k_product_wide"), ("dropout_kernels.hip", "k_dropout")])
def test_kernels_use_no_scratch(tmp_path, source, kernel):
    from zero_partitioned_optimizer_amd import build as B
    flags = [f for f in B.HIPCC_FLAGS if f not in ("-fPIC", "-shared")]
    cmd = [B.hipcc(), *flags, "-I", os.path.join(ROOT, "include"), "-I", B.CSRC, "-c", os.path.join(B.CSRC, source),
           "-o", str(tmp_path / "k.o"), "-Rpass-analysis=kernel-resource-usage"]
    out = subprocess.run(cmd, capture_output=True, text=True, check=True).stderr
    names = re.findall(r"Function Name: (\S+)", out)
    scratch = [int(x) for x in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", out)]
    assert names and len(names) == len(scratch)
    assert any(kernel in n for n in names)
    assert not [(n, s) for n, s in zip(names, scratch) if s != 0]


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_header_is_plain_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "zero_layer.h"\n'
                   "_Static_assert(sizeof(zero_dropout) == 32, \"\");\n"
                   "_Static_assert(sizeof(zero_linear_args) == 176, \"\");\n"
                   "_Static_assert(sizeof(zero_linear_grad_input_args) == 152, \"\");\n"
                   "_Static_assert(sizeof(zero_linear_grad_weight_args) == 112, \"\");\n"
                   "_Static_assert(sizeof(zero_dropout_args) == 128, \"\");\n"
                   "int (*f)(const zero_linear_args*, void*) = zero_linear_forward;\n")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), "-c", str(src),
                    "-o", str(tmp_path / "h.o")], check=True)


def test_layer_mode_needs_a_layer():
    r = subprocess.run(["python3", os.path.join(ROOT, "bench.py"), "--layer", "--config", "tiny"], capture_output=True,
                       text=True, timeout=120, cwd=ROOT)
    assert r.returncode == 2 and "--layer" in r.stderr
