"""The rules that choose the gated block's tile, split and launch
(shard_placement_amd/csrc/product_shape.h), built with g++ into a host-only
library: no GPU and no HIP involved."""
import ctypes
import os
import subprocess
import tempfile

from tests.shape_rules import HDR, Shape, round8

SRC = r"""
#include "product_shape.h"
static void put(const tide::Shape& s, long long* o) {
    const long long v[] = {s.bi, s.bj, s.bk, s.halves, s.tiles_i, s.tiles_j, s.splits, s.split_depth};
    for (int k = 0; k < 8; ++k) o[k] = v[k];
}
extern "C" int by_rows(long long T, long long N, long long K, int keep, int direct) {
    return tide::gated_by_rows(T, N, K, keep != 0, direct != 0);
}
extern "C" int past(long long rows, long long depth) { return tide::past_the_cache(rows, depth); }
extern "C" int gradients_of(long long T, long long turn, long long K, int dx, int dw, long long* in,
                            long long* weight, int* in_first) {
    const tide::Gradients g = tide::choose_gated_gradients(T, turn, K, dx != 0, dw != 0);
    put(g.in, in);
    put(g.weight, weight);
    *in_first = g.in_first;
    return g.pair;
}
extern "C" void choose_gated_of(long long I, long long J, long long depth, long long* o) {
    put(tide::choose_gated(I, J, depth), o);
}
"""
_lib = None


def lib():
    global _lib
    if _lib is None:
        with tempfile.TemporaryDirectory() as d:
            src, so = os.path.join(d, "gated.cpp"), os.path.join(d, "libgated.so")
            with open(src, "w") as f:
                f.write(SRC)
            subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-fPIC", "-shared",
                            "-I" + HDR, src, "-o", so], check=True)
            _lib = ctypes.CDLL(so)
        ll = ctypes.c_longlong
        _lib.choose_gated_of.argtypes = [ll, ll, ll, ctypes.POINTER(ll)]
        _lib.choose_gated_of.restype = None
        _lib.past.argtypes = [ll, ll]
        _lib.by_rows.argtypes = [ll, ll, ll, ctypes.c_int, ctypes.c_int]
        _lib.gradients_of.argtypes = [ll, ll, ll, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ll),
                                      ctypes.POINTER(ll), ctypes.POINTER(ctypes.c_int)]
    return _lib


def choose(I, J, depth):
    o = (ctypes.c_longlong * 8)()
    lib().choose_gated_of(I, J, depth, o)
    return Shape(*o)


def rows(N):
    """Rows of the two weights together, 16 of one and 16 of the other in turn."""
    return 2 * (-(-N // 16) * 16)


def turn(N):
    """Columns of dg (and of du) in the workspace."""
    return -(-N // 64) * 64


def gradients(T, N, K, dx=True, dw=True):
    """(dx's Shape, the weights', whether they share a launch, whether dx's tiles
    come first in one of 256-wide tiles)."""
    a, b, first = (ctypes.c_longlong * 8)(), (ctypes.c_longlong * 8)(), ctypes.c_int(0)
    pair = lib().gradients_of(T, turn(N), K, dx, dw, a, b, ctypes.byref(first))
    return Shape(*a), Shape(*b), bool(pair), bool(first.value)


def forward(T, N, K, keep=False):
    """The forward product's Shape, or None where it goes by the weights' rows."""
    if lib().by_rows(T, N, K, keep, K % 8 == 0):
        return None
    return choose(rows(N), T, round8(K))


def forms(T, N, K):
    """The launches of a forward call (something kept or not) and of both
    gradients together and alone: kernel form, and whether the contraction is
    split."""
    name = lambda s: (s.bi, s.bj, s.bk, s.halves, s.splits > 1)  # noqa: E731
    out = set()
    for keep in (False, True):
        s = forward(T, N, K, keep)
        once = s is not None and s.tiles_j == 1 and s.bi == 128 and bool(lib().past(rows(N), round8(K)))
        out.add(("forward by rows", min(T, 3)) if s is None else ("forward",) + name(s) + (once,))
    x, w, pair, first = gradients(T, N, K)
    if pair and w.bi == 256:
        out.add(("both, wide", x.bj, w.bj, "dx first" if first else "dW first", x.splits > 1))
    elif pair:
        groups = x.tiles_i * x.tiles_j * x.splits + w.tiles_i * w.tiles_j
        out.add(("both", x.bj, 2 if groups <= 256 else 1, x.splits > 1))
    out.add(("dx",) + name(gradients(T, N, K, dw=False)[0]))
    out.add(("dW",) + name(gradients(T, N, K, dx=False)[1]))
    return out
