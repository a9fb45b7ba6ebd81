"""The order of the products of packed attention at head dim 64, over all segments: the functions
that the kernel's warps use (csrc/packed_order.h), compiled for the host.

S and P have three places, product k uses place k % 3, and a barrier of the place completes a
phase with each product's P V. A warp that waits for product k by the parity of its phase must
have found it before product k + 3 completes the next one; so whoever waits has to hold
product k + 3 back."""
import ctypes
import itertools
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_sparse_score_gb300", "csrc")
SOURCE = """
#include "packed_order.h"
using P = ha::Products;
extern "C" {
int count(int e0, int nt, int one) { return P{e0, nt, one != 0}.count(); }
int tiles(int e0, int nt, int one, int t) { return P{e0, nt, one != 0}.tiles(t); }
int stream(int e0, int nt, int one, int k) { const P p{e0, nt, one != 0}; return p.stream(k, p.last_of_tile(k)); }
int last_of_tile(int e0, int nt, int one, int k) { return P{e0, nt, one != 0}.last_of_tile(k); }
int of(int e0, int nt, int one, int t, int i) { return P{e0, nt, one != 0}.of(t, i); }
int lapped(int e0, int nt, int one, int t) { return P{e0, nt, one != 0}.lapped(t); }
}
"""


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a host compiler")
    d = tmp_path_factory.mktemp("order")
    src, lib = d / "order.cpp", d / "liborder.so"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


# (e0, nt, one): row tile 1 sees up to two key tiles more (128 tokens of one head, tiles of 64 keys)
SEGMENTS = [(nt, nt, 1) for nt in range(1, 30)] + [(nt - x, nt, 0) for nt, x in itertools.product(range(1, 30), range(3)) if nt >= x] \
    + [(0, nt, 0) for nt in range(3, 6)]  # row tile 0 sees no key


def steps(order, seg):
    return {(t, i): order.of(*seg, t, i) for t in (0, 1) for i in range(order.tiles(*seg, t))}


@pytest.mark.parametrize("seg", SEGMENTS, ids=str)
def test_order_is_one_to_one(order, seg):
    of, n = steps(order, seg), order.count(*seg)
    assert sorted(of.values()) == list(range(n))
    for (t, i), k in of.items():
        assert order.stream(*seg, k) == t
        key = (2 * i + t) if seg[2] else i  # the key tile
        later = [x for (u, j), x in of.items() if ((2 * j + u) if seg[2] else j) == key and x > k]
        assert order.last_of_tile(*seg, k) == (not later)
    key_of = {k: (2 * i + t if seg[2] else i) for (t, i), k in of.items()}
    assert [key_of[k] for k in range(n)] == sorted(key_of.values())  # the ring's order


@pytest.mark.parametrize("seg", SEGMENTS, ids=str)
def test_a_stream_holds_back_what_laps_a_product_it_waits_for(order, seg):
    """While a stream works on tile i (its P is not full, so P V of product of(t, i) and of all behind
    it are not issued), it waits for S of that product and for P V of the tile before."""
    of = steps(order, seg)
    for (t, i), k in of.items():
        if i > 0:
            assert of[t, i - 1] + 3 > k  # the lapping product comes behind the one held back


@pytest.mark.parametrize("seg", SEGMENTS, ids=str)
def test_a_stream_that_can_be_lapped_at_its_end_is_known(order, seg):
    """Behind its last tile a stream holds nothing back in its segment. Where a later product uses the
    last one's place, it waits for the segment's end instead (the next segment waits for both
    streams, so no phase of it comes before they have found this one's)."""
    of, n = steps(order, seg), order.count(*seg)
    for t in (0, 1):
        tiles = order.tiles(*seg, t)
        assert order.lapped(*seg, t) == (tiles > 0 and of[t, tiles - 1] + 3 < n or (tiles == 0 and not seg[2] and seg[1] > 1))
    if seg == (10, 12, 0):  # stream 0 waits for product 18 while 21 is row tile 1's, on the same place
        assert of[0, 9] == 18 and order.stream(*seg, 21) == 1 and order.lapped(*seg, 0)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 128])
@pytest.mark.parametrize("keys", [64, 128])
def test_row_tiles_that_can_lap(G, keys):
    """Two key tiles more in row tile 1 take a row tile of 128 tokens and key tiles of 64: the bf16
    kernel (128 keys a tile) has no such segment, so it does not ask."""
    tq = 128 // G
    most = max(-(-(seen + x) // keys) - -(-seen // keys) for seen in range(1, 300) for x in range(tq + 1))
    assert (most > 1) == (keys == 64 and G == 1)


# ---------------------------------------------------------------- rows that leave through the ring

def second_phase_possible(stages, nt, full, all_wait):
    """Staged item A's rows lie in ring slots 0 and 1 (of the tiles counted from there), the next
    staged item has nt key tiles, and the warp that sends rows off has not looked at A's barrier yet,
    so neither slot is free again. Can all eight warps arrive for the next item? ``full``: its second row
    tile has a box to put; ``all_wait``: stream 1 waits for its slot without one too."""
    tiles = range(2, 2 + 2 * nt)
    if any(i >= stages and i - stages < 2 for i in tiles) or tiles[-1] >= stages + 2:
        return False  # the loader stands before A's slots
    waits = [tiles[-1] + 1] + ([tiles[-1] + 2] if full or all_wait else [])
    return not any(0 <= i - stages < 2 for i in waits)


def test_staged_rows_are_found_before_the_next_are_there():
    for nt in range(1, 40):
        for full in (False, True):
            assert not second_phase_possible(5, nt, full, True)
    # without the wait: a next item of one key tile whose second row tile is not full
    assert [(nt, full) for nt in range(1, 40) for full in (False, True) if second_phase_possible(5, nt, full, False)] == [(1, False)]
    # with a ring of more stages the wait would not hold it back
    assert second_phase_possible(6, 1, True, True)


# ---------------------------------------------------------------- the work of a row of items

TILE_SOURCE = """
#include "packed_order.h"
template <int K>
static uint32_t sum(uint32_t a, uint32_t n, uint32_t b) {
    const ha::TileSums<K> t(a);
    uint16_t before[ha::TileSums<K>::kMost] = {};
    uint32_t at = 0;
    for (int x = 0; x < ha::TileSums<K>::kMost; ++x) {
        before[x] = (uint16_t)at;
        at += t.remainder((uint32_t)x);
    }
    return t.sum(n, b, before);
}
extern "C" uint32_t sum6(uint32_t a, uint32_t n, uint32_t b) { return sum<6>(a, n, b); }
extern "C" uint32_t sum7(uint32_t a, uint32_t n, uint32_t b) { return sum<7>(a, n, b); }
"""


@pytest.fixture(scope="module")
def sums(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a host compiler")
    d = tmp_path_factory.mktemp("sums")
    src, lib = d / "sums.cpp", d / "libsums.so"
    src.write_text(TILE_SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    L = ctypes.CDLL(str(lib))
    for f in (L.sum6, L.sum7):
        f.restype, f.argtypes = ctypes.c_uint32, [ctypes.c_uint32] * 3
    return {64: L.sum6, 128: L.sum7}


@pytest.mark.parametrize("keys", [64, 128])
def test_key_tiles_of_a_row_of_items(sums, keys):
    """For every number of heads a KV head has: sum over i < n of floor((a i + b) / keys)."""
    f = sums[keys]
    for a in sorted({2 * (128 // G) for G in range(1, 129)}):
        for b in list(range(0, 3 * keys, 7)) + [keys - 1, keys, 12345, (1 << 20) + 77]:
            total = 0
            for n in range(1, 150):
                total += (a * (n - 1) + b) // keys
                assert f(a, n, b) == total % 2 ** 32, (a, n, b)
    import random
    r = random.Random(keys)
    for _ in range(300):
        a, n = 2 * (128 // r.randint(1, 128)), r.randint(1, 20000)
        b = r.randrange(1 << r.randint(1, 30))
        total = sum((a * i + b) // keys for i in range(n))
        assert f(a, n, b) == total % 2 ** 32, (a, n, b)
    # as many tokens as a call takes
    n = (1 << 24) // 256
    assert f(256, n, 1) == sum((256 * i + 1) // keys for i in range(n)) % 2 ** 32
