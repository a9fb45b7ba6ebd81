"""The work of a row of items under score options (csrc/packed_order.h, compiled for the host): key
tiles in closed form against counting them."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_sparse_score_gb300", "csrc")
SOURCE = """
#include "packed_order.h"
template <int K>
static uint32_t before(int base, int nq, int first, int prefix, int window, int t2, int qt) {
    const ha::TileSums<K> t((uint32_t)t2);
    uint16_t b[ha::TileSums<K>::kMost] = {};
    uint32_t at = 0;
    for (int x = 0; x < ha::TileSums<K>::kMost; ++x) {
        b[x] = (uint16_t)at;
        at += t.remainder((uint32_t)x);
    }
    return ha::MaskedItems<K>{base, nq, first, prefix, window, t2, ha::Quotient::of((uint32_t)t2)}.tiles_before(qt, t, b);
}
#define ARGS int base, int nq, int first, int prefix, int window, int t2, int qt
#define PASS base, nq, first, prefix, window, t2, ha::Quotient::of((uint32_t)t2)
#define PLAIN base, nq, first, prefix, window, t2
extern "C" {
uint32_t before6(ARGS) { return before<6>(PLAIN, qt); }
uint32_t before7(ARGS) { return before<7>(PLAIN, qt); }
int tiles6(ARGS) { return ha::MaskedItems<6>{PASS}.tiles(qt); }
int tiles7(ARGS) { return ha::MaskedItems<7>{PASS}.tiles(qt); }
int begin6(ARGS) { return ha::MaskedItems<6>{PASS}.begin_tile(qt); }
int begin7(ARGS) { return ha::MaskedItems<7>{PASS}.begin_tile(qt); }
int quotient(int n, int d) { return ha::Quotient::of((uint32_t)d)(n); }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a host compiler")
    d = tmp_path_factory.mktemp("items")
    src, so = d / "items.cpp", d / "libitems.so"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover=all", "-shared", "-fPIC", "-I", CSRC,
                    str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    for n in ("before6", "before7"):
        getattr(lib, n).restype = ctypes.c_uint32
    return lib


def seen(base, nq, first, prefix, window, t):
    """The keys that token t sees, as a half-open range (empty: None)."""
    pos = base + t
    lo, hi = max(first, pos - window + 1 if window else 0, 0), min(max(pos + 1, prefix), base + nq)
    return (lo, hi) if lo < hi else None


def item(base, nq, first, prefix, window, t2, qt, size):
    """First key tile and number of tiles of an item, from its tokens' keys."""
    spans = [s for t in range(qt * t2, min((qt + 1) * t2, nq)) if (s := seen(base, nq, first, prefix, window, t))]
    if not spans:
        return 0, 1
    lo, hi = min(s[0] for s in spans) // size, -(-max(s[1] for s in spans) // size)
    return lo, hi - lo


def cases(n, seed):
    r = random.Random(seed)
    for _ in range(n):
        t2 = 2 * (128 // r.choice([1, 2, 3, 4, 5, 7, 8, 16, 40, 128]))
        nq = r.choice([1, 2, t2, t2 + 1, r.randint(1, 40 * t2)])
        nk = max(0, nq + r.choice([0, 0, r.randint(-nq, 0), r.randint(0, 3000), r.randint(0, 300)]))
        base = nk - nq
        window = r.choice([0, 0, 1, 64, 128, r.randint(1, 400), r.randint(1, 5000)])
        first = r.choice([0, 0, r.randint(0, nk), nk])
        prefix = r.choice([0, 0, r.randint(0, nk), nk])
        yield base, nq, first, prefix, window, t2


@pytest.mark.parametrize("log2", [6, 7])
@pytest.mark.parametrize("seed", range(8))
def test_tiles_of_items(lib, log2, seed):
    for c in cases(60, seed):
        n_items = -(-c[1] // c[5])
        at = 0
        for qt in range(n_items):
            begin, tiles = item(*c, qt, 1 << log2)
            # a token that sees nothing between tokens that do may widen the span by what it would have seen
            got = getattr(lib, f"begin{log2}")(*c, qt), getattr(lib, f"tiles{log2}")(*c, qt)
            assert got[0] <= begin and got[0] + got[1] >= begin + tiles and got[1] <= tiles + 3, (c, qt, got, begin, tiles)
            assert getattr(lib, f"before{log2}")(*c, qt) == at, (c, qt)
            at += got[1]


@pytest.mark.parametrize("log2", [6, 7])
def test_tiles_of_items_of_long_caches(lib, log2):
    """Keys up to 2^30, no intermediate past 31 bits (the library is built to stop there)."""
    top, r = 1 << 30, random.Random(3)
    for _ in range(300):
        t2 = 2 * (128 // r.choice([1, 3, 4, 8]))
        nq = r.choice([1, 300, 1 << 24])
        nk = r.choice([top, top - r.randint(0, 1000), nq, r.randint(nq // 2, top)])
        first, prefix = (r.choice([0, nk, r.randint(0, nk)]) for _ in range(2))
        window = r.choice([0, 1, 4096, top - 1, r.randint(1, top - 1)])
        c = (nk - nq, nq, first, prefix, window, t2)
        n_items = -(-nq // t2)
        for qt in {0, n_items - 1, n_items // 2, max(0, n_items - 2)}:
            tiles = getattr(lib, f"tiles{log2}")(*c, qt)
            assert tiles >= 1
            if qt + 1 < n_items:
                a, b = getattr(lib, f"before{log2}")(*c, qt), getattr(lib, f"before{log2}")(*c, qt + 1)
                assert (b - a) % (1 << 32) == tiles, (c, qt)


def test_quotients(lib):
    r = random.Random(4)
    for d in [*range(1, 300), 1 << 20, (1 << 20) + 1, (1 << 31) - 1]:
        for n in [0, 1, d - 1, d, d + 1, (1 << 31) - 1, (1 << 31) - 2, (1 << 30) + 7] + [k * d + e for k in r.sample(range(1, max(2, (1 << 31) // d - 1)), min(6, max(1, (1 << 31) // d - 3))) for e in (-1, 0)]:
            if 0 <= n < 1 << 31:
                assert lib.quotient(n, d) == n // d, (n, d)
