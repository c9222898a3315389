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


def _sgprs(text):
    out = set()
    for lo, hi in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        out |= set(range(int(lo), int(hi) + 1))
    return out | {int(n) for n in re.findall(r"\bs(\d+)\b", text)}


@pytest.mark.skipif(not HIPCC, reason="hipcc not available")
def test_loads_to_lds_wait_for_their_descriptors(tmp_path):
    """A scalar register that a vector instruction wrote (v_readfirstlane, v_readlane) may
    be read by a memory instruction five wait states later. The compiler sees to that for
    its own instructions but does not look into inline assembly, so each load to LDS there
    has to bring the distance with it, whatever the compiler puts before it."""
    from zero_partitioned_optimizer_amd import build as B
    flags = [f for f in B.HIPCC_FLAGS if f not in ("-fPIC", "-shared")]
    out = tmp_path / "k.s"
    subprocess.run([B.hipcc(), *flags, "-I", os.path.join(ROOT, "include"), "-I", B.CSRC, "--cuda-device-only", "-S",
                    os.path.join(B.CSRC, "linear_kernels.hip"), "-o", str(out)], check=True, capture_output=True)
    name, before, loads, bad = None, [], 0, []
    for line in out.read_text().splitlines():
        line = line.split(";")[0].strip()
        if line.endswith(":"):              # a block begins: what ran before it is not known
            name = line if line.startswith("_Z") else name
            before = ["block"]
            continue
        if not line or line.startswith("."):
            continue
        if line.startswith("buffer_load") and line.endswith(" lds"):
            loads += 1
            reads, states = _sgprs(line), 0
            for prev in reversed(before):
                if states >= 5:
                    break
                written = prev.startswith("v_") and _sgprs(",".join(prev.split(",")[:2])) & reads
                if prev == "block" or written:
                    bad.append((name, states, prev, line))
                    break
                states += int(prev.split()[1], 0) + 1 if prev.startswith("s_nop") else 1
        before = before[-16:] + [line]
    assert loads > 100
    assert not bad, (len(bad), bad[:4])


def test_assembly_names_what_it_writes():
    """A scalar register or flag that inline assembly writes by name is in its list of
    clobbers: the compiler may otherwise keep a value of its own there."""
    from zero_partitioned_optimizer_amd import build as B
    seen = 0
    for source in B.SOURCES:
        text = open(os.path.join(B.CSRC, source)).read()
        for block in re.findall(r"asm volatile\((.*?)\);", text, re.S):
            code = "".join(re.findall(r'"([^"]*)"', block.split("\n" + " " * 8 + ":")[0].split(" : ")[0]))
            clobbers = set(re.findall(r'"([^"]*)"', block.split(":")[-1]))
            written = set(re.findall(r"\b\w+ (m0|vcc|exec)\b,", code)) | (
                {"scc"} if re.search(r"\bs_(add|sub|and|or|cmp|lshl|lshr)", code) else set())
            seen += bool(written)
            assert written <= clobbers, (source, written - clobbers, block)
    assert seen


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
