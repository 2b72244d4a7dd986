"""GPU: the example's decoding and training steps run, and the decoding step
is as far from 64 bits as its roundings allow: the projection quantises x and
its weights to E4M3 (2^-4 of each value at most), the experts' layer rounds h
to 9 bits and its output to BF16 (2^-9 and 2^-8, test_gpu_moe.py)."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import adapters_and_experts as ex
    finally:
        sys.path.pop(0)
    err, status = ex.main(["--requests", "5", "--width", "256", "--inner", "192",
                           "--experts", "4", "--adapters", "2", "--rank", "8",
                           "--train-tokens", "300"])
    assert status == 0
    assert err[0] <= 2 * 2.0 ** -4
    assert err[1] <= 2.0 ** -8 + 2.0 ** -9
