"""The rules by which MXFP4 calls choose their kernels, as the tests know them,
against the library: a rule that moves fails here instead of leaving a kernel
without a test."""
import os
import random
import re

import pytest

from conftest import ROOT

import mx_rules
from sparse_bf16_delta_amd import _abi


def source(name):
    text = open(os.path.join(ROOT, "sparse_bf16_delta_amd", "csrc", name)).read()
    return re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", text))


def test_rules_of_the_apply():
    text = source("mxfp4.hip")
    for words in ("kLargeDelta = int64_t(1) << 20, kLargeSpread = 20;",
                  "kDenseSpread = 10, kDenseExtra = int64_t(1) << 19;",
                  "max_nnz >= list.elems / kDenseSpread + kDenseExtra",
                  "max_nnz >= kLargeDelta && max_nnz >= elems / kLargeSpread"):
        assert words in text, words


def test_rules_of_the_product():
    text = source("mxfp4_matmul.hip")
    for words in ("m <= 32 && (m + 15) / 16 * n <= 16384;",
                  "{256, 256, 8.5, 0.0, 1}, {128, 128, 2.9, 1.2, 2}, {64, 64, 1.0, 0.9, 4}",
                  "constexpr int kCus = 256;",
                  "tiles > kCus && last > 0"):
        assert words in text, words


def test_shares_are_those_of_the_workspace():
    """The partial sums' bytes tell how k is shared out."""
    size = _abi.load().mxfp4_matmul_workspace_size
    rng = random.Random(3)
    seen = set()
    for _ in range(5000):
        m, n, k = (int(2 ** rng.uniform(0, e)) for e in (14, 16, 15))
        cut = mx_rules.cut_of(m, n, k)
        seen.add(cut)
        assert size(m, n, k) == (cut[1] * m * n * 4 if cut[1] > 1 else 0), (m, n, k)
    assert len(seen) >= 12


@pytest.mark.parametrize("shape,cut", list(mx_rules.CUTS.items()), ids=str)
def test_each_cut_has_a_shape(shape, cut):
    assert mx_rules.cut_of(*shape) == cut


def test_every_cut_is_listed():
    rng = random.Random(4)
    for _ in range(20000):
        shape = tuple(int(2 ** rng.uniform(0, e)) for e in (14, 16, 15))
        assert mx_rules.cut_of(*shape) in set(mx_rules.CUTS.values()), shape
