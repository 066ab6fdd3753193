"""The distance within which mk_tree_verify leaves an acceptance to 64-bit sums covers what its fp32
sums of exponentials can be off by (CPU only: the bound's arithmetic, from the kernel's constants)."""
import math
import pathlib
import re

import numpy as np

TEXT = (pathlib.Path(__file__).resolve().parents[1] / "persistent_megakernel_decode_04_b200" / "csrc" /
        "mk_tree_verify.cu").read_text()
MAX_VOCAB = 1 << 20


def constant(name):
    return float(re.search(rf"constexpr \w+ {name} = ([\d.e-]+)f?;", TEXT).group(1))


def relative_error_of_a_rows_sum():
    """Largest relative error of a row's fp32 sum of exponentials."""
    h = 2.0 ** -24                      # a rounding
    threads, chunk = constant("kStatThreads"), constant("kChunk")
    chunks = math.ceil((MAX_VOCAB + 8) / chunk)
    per_lane = math.ceil(chunks / 16)   # chunks that a lane joins one after another
    # a value and its way up: its exponential, to the warp's, the block's, the lane's, the row's maximum, and
    # up to per_lane - 1 times to a higher maximum of a later chunk; 2^-22 and a product's rounding each
    exponentials = 5 + per_lane - 1
    # two sums side by side per thread, joined; then a warp's, a block's, a lane's, half a warp's
    additions = chunk / threads / 2 + 1 + 5 + math.log2(threads / 32) + per_lane + 4
    # exponents: the difference, the product, and log2(e) / temperature, two roundings; an error of the
    # exponent y moves a value by y ln 2 times that.  All but one word at -t is the worst: the mean of
    # |y| over the sum's weights
    t = np.linspace(0.0, 40.0, 4001)
    w = MAX_VOCAB * 2.0 ** -t
    mean = float((w * t / (1 + w)).max())
    return exponentials * (2.0 ** -22 + h) + additions * h + 4 * h * math.log(2) * mean


def test_close_decisions_are_left_to_exact_sums():
    bound = relative_error_of_a_rows_sum()
    assert 4e-6 < bound < 1e-5
    # u q / ZQ < p / ZP is decided by both rows' sums; p and q are 64-bit
    assert 2 * bound + 2.0 ** -40 < constant("kClose")
