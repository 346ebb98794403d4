"""Orders between waves and wait states that no run shows reliably, read from
the kernels' sources and from the built code (CPU)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_weight_quantization_amd", "csrc")


def _source(name):
    return open(os.path.join(CSRC, name), encoding="utf-8").read()


def test_top_logits_sums_do_not_overwrite_the_maxima():
    """Between the waves' maxima being read and their partial sums being
    written no barrier is certain (the threshold's search has none where all
    of a row's groups agree), so the two lie in arrays of their own."""
    src = _source("top.hip")
    maxima = re.search(r"s\.(\w+)\[w\] = m\b", src).group(1)
    assert len(re.findall(rf"s\.{maxima}\b", src)) == 3  # written once, read once by max3 of two operands
    sums = re.findall(r"block_reduce<TPB>\(sum, s\.(\w+),", src)
    assert sums and maxima not in sums


def test_a_wait_state_between_m0_and_the_load_into_lds():
    """A scalar write of m0 and a load into LDS that takes its address from
    there need a wait state between them. The compiler sees to it in its own
    code, not within inline asm."""
    seen = 0
    for name in sorted(os.listdir(CSRC)):
        for text in re.findall(r'asm volatile\(\s*"((?:[^"\\]|\\.)*)"', _source(name)):
            ops = [o.strip() for o in text.replace("\\t", "").split("\\n")]
            for at, op in enumerate(ops):
                if re.match(r"s_\w+ m0\b", op):
                    seen += 1
                    assert "lds" not in ops[at + 1], (name, text)
    assert seen >= 3


def test_wait_states_in_the_built_code():
    """The same in every load into LDS of the built library's device code."""
    import subprocess
    import tempfile

    import pytest

    bin_ = "/opt/rocm/lib/llvm/bin"
    lib = os.path.join(ROOT, "post_weight_quantization_amd", "libkq.so")
    if not (os.path.exists(lib) and os.path.exists(os.path.join(bin_, "llvm-objdump"))):
        pytest.skip("needs the built library and llvm-objdump")
    loads, bare = 0, []
    with tempfile.TemporaryDirectory() as tmp:
        link = os.path.join(tmp, "libkq.so")
        os.symlink(lib, link)
        subprocess.run([os.path.join(bin_, "llvm-objdump"), "--offloading", link], cwd=tmp, check=True,
                       capture_output=True)
        objects = [f for f in sorted(os.listdir(tmp)) if "gfx950" in f]
        assert objects
        for f in objects:
            text = subprocess.run([os.path.join(bin_, "llvm-objdump"), "-d", "--no-show-raw-insn",
                                   os.path.join(tmp, f)], check=True, capture_output=True, text=True).stdout
            before = ""
            for line in text.splitlines():
                op = line.split("//")[0].strip()
                if "load_lds" in op or (op.startswith("buffer_load") and op.endswith(" lds")):
                    loads += 1
                    if re.match(r"s_\w+ m0\b", before):
                        bare.append((before, op))
                before = op
    assert loads > 0 and not bare, (len(bare), bare[:3])
