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
