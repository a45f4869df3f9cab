"""The reciprocal, the scale and the quotient of the FP8 quantiser (the
reciprocal is the router's, too) against the IEEE operations, bit by bit."""
import ctypes
import os
import subprocess

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def counts(tmp_path_factory):
    from fp4_weight_moe_gb300 import build as b
    so = str(tmp_path_factory.mktemp("rounding") / "rounding.so")
    subprocess.run([b._nvcc(), *b.ARCH, *b.FLAGS, "-Xcompiler", "-fvisibility=default", "-I", b.CSRC, "-shared", "-o", so,
                    os.path.join(HERE, "rounding.cu")], check=True, capture_output=True)
    lib = ctypes.CDLL(so)
    for f in (lib.count_reciprocals, lib.count_scales, lib.count_quotients):
        f.restype = ctypes.c_ulonglong
    return lib


@pytest.mark.parametrize("exponent", [-100, -69, -1, 0, 1, 51, 125])
def test_reciprocal_of_every_significand(counts, exponent):
    assert counts.count_reciprocals(exponent) == 0


@pytest.mark.parametrize("exponent", [-60, -1, 0, 59])
def test_scale_of_every_significand(counts, exponent):
    assert counts.count_scales(exponent) == 0


@pytest.mark.parametrize("ev,es", [(0, 0), (8, 0), (-50, -50), (51, 50)])
def test_quotients(counts, ev, es):
    """Every divisor: 256 scrambled dividends and every BF16 one; the divisors
    next to the upper power of two, whose reciprocals are the farthest off,
    with the 2^16 dividends next to each."""
    assert counts.count_quotients(0, 0, 256, ev, es) == 0
    assert counts.count_quotients(1, 0, 128, ev, es) == 0
    assert counts.count_quotients(2, (1 << 23) - (1 << 13), 1 << 16, ev, es) == 0
