"""The references of capped scores and the fits of the tanh (csrc/packed_order.h, csrc/hashattn_api.cu), on the host:
that sums of weights stay within float32, and that the polynomials are as close as their comments say."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_sparse_score_gb300", "csrc")
SOURCE = """
#include "packed_order.h"
extern "C" void cap_range(double cap, int keys, double* low, double* high, int* fits) {
    const ha::CapRange r = ha::CapRange::of(cap, keys);
    *low = r.low, *high = r.high, *fits = r.fits();
}
"""


@pytest.fixture(scope="module")
def cap_range(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a host compiler")
    d = tmp_path_factory.mktemp("range")
    src, so = d / "range.cpp", d / "librange.so"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))

    def of(cap, keys):
        low, high, fits = ctypes.c_double(), ctypes.c_double(), ctypes.c_int()
        lib.cap_range(ctypes.c_double(cap), keys, ctypes.byref(low), ctypes.byref(high), ctypes.byref(fits))
        return low.value, high.value, bool(fits.value)

    return of


@pytest.mark.parametrize("keys", [1, 2, 1000, 1 << 14, 1 << 24, (1 << 24) + 1, (1 << 28) - 1, 1 << 28, (1 << 28) + 1, 1 << 30])
def test_sums_of_weights_stay_within_float32(cap_range, keys):
    """A row whose first keys give the lowest reference, and all others weigh 2^(cap - low), beside values of 2^20; and
    the smallest weight, 2^(-cap - high), beside values of 2^-40: 24 bits above 2^-149."""
    fitting = 0
    for cap in [2.0 ** -60, 1e-3, 1.0, *range(5, 130), 1e3, 2.0 ** 60]:
        low, high, fits = cap_range(cap, keys)
        assert fits == (low <= high)
        if fits:
            fitting += 1
            assert math.log2(keys) + (cap - low) + 20 <= 125
            assert -cap - high - 40 - 24 >= -149 - 1e-9
    assert fitting > 75  # caps of 50 e-folds (72 powers of 2) among them
    assert cap_range(50 / math.log(2), keys)[2]


def coefficients(name):
    text = open(os.path.join(CSRC, "hashattn_api.cu")).read()
    body = re.search(name + r"\[2\]\[7\] = \{(.*?)\n\};", text, re.S).group(1)
    rows = re.findall(r"\{([^}]*)\},  // degree (\d+) up to ([\d.]+): ([\d.e-]+)", body)
    assert len(rows) == 2
    return [([float(c) for c in row.split(",")], int(degree), float(to), float(err)) for row, degree, to, err in rows]


@pytest.mark.parametrize("name", ["kTanh16", "kTanh32"])
def test_fits_of_the_tanh(name):
    """In relative error, over 20,000 points, by the coefficients as they are used: in float32, with the sums in 64 bits."""
    for c, degree, to, err in coefficients(name):
        assert len(c) == degree + 1
        u = np.linspace(1e-6, to, 20001)
        for cs, more in ((c, 0.0), ([float(np.float32(x)) for x in c], 2.0 ** -24)):
            p = sum(x * u ** (2 * k) for k, x in enumerate(cs))
            off = np.abs(p * u / np.tanh(u) - 1).max()
            assert off <= err * 1.02 + more, (name, to, off)
