"""The rules that choose a layer product's tile, split and launch
(shard_placement_amd/csrc/product_shape.h), built with g++ into a host-only
library: no GPU and no HIP involved."""
import ctypes
import os
import subprocess
import tempfile
from collections import namedtuple

HDR = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "shard_placement_amd", "csrc")

SRC = r"""
#include "product_shape.h"
using namespace tide;
static void put(const Shape& s, long long* o) {
    const long long v[] = {s.bi, s.bj, s.bk, s.halves, s.tiles_i, s.tiles_j, s.splits, s.split_depth};
    for (int k = 0; k < 8; ++k) o[k] = v[k];
}
extern "C" {
double choose_of(int kind, long long I, long long J, long long depth, long long* o) {
    double us = 0.0;
    put(choose((Kind)kind, I, J, depth, &us), o);
    return us;
}
int by_rows(long long T, long long N, long long K, int keep, int direct) {
    return forward_by_rows(T, N, K, keep != 0, direct != 0);
}
int gradients_of(long long T, long long N, long long K, int dx, int dw, long long* in, long long* weight,
                 int* in_first) {
    const Gradients g = choose_gradients(T, N, K, dx != 0, dw != 0);
    put(g.in, in);
    put(g.weight, weight);
    *in_first = g.in_first;
    return g.pair;
}
int tiles() { return (int)(sizeof(kTiles) / sizeof(kTiles[0])); }
double estimate(int kind, int tile, long long I, long long J, long long depth, long long splits, long long* o) {
    Shape s = {kTiles[tile].bi, kTiles[tile].bj, 64, kTiles[tile].halves, 0, 0, 1, 0};
    set_split(&s, I, J, depth, splits);
    put(s, o);
    return product_us((Kind)kind, kTiles[tile], s, I, J, depth);
}
}
"""

Shape = namedtuple("Shape", "bi bj bk halves tiles_i tiles_j splits split_depth")
FORWARD, GRAD_INPUT, GRAD_WEIGHT = range(3)
_lib = None


def lib():
    global _lib
    if _lib is None:
        with tempfile.TemporaryDirectory() as d:
            src, so = os.path.join(d, "shape.cpp"), os.path.join(d, "libshape.so")
            with open(src, "w") as f:
                f.write(SRC)
            subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-fPIC", "-shared",
                            "-I" + HDR, src, "-o", so], check=True)
            L = ctypes.CDLL(so)
        ll, out = ctypes.c_longlong, ctypes.POINTER(ctypes.c_longlong)
        L.choose_of.argtypes, L.choose_of.restype = [ctypes.c_int, ll, ll, ll, out], ctypes.c_double
        L.by_rows.argtypes = [ll, ll, ll, ctypes.c_int, ctypes.c_int]
        L.gradients_of.argtypes = [ll, ll, ll, ctypes.c_int, ctypes.c_int, out, out,
                                   ctypes.POINTER(ctypes.c_int)]
        L.estimate.argtypes = [ctypes.c_int, ctypes.c_int, ll, ll, ll, ll, out]
        L.estimate.restype = ctypes.c_double
        _lib = L
    return _lib


def _out():
    return (ctypes.c_longlong * 8)()


def choose(kind, I, J, depth):
    """(Shape, estimate in us; 0 where none is made)."""
    o = _out()
    us = lib().choose_of(kind, I, J, depth, o)
    return Shape(*o), us


def estimate(kind, tile, I, J, depth, splits):
    o = _out()
    us = lib().estimate(kind, tile, I, J, depth, splits, o)
    return Shape(*o), us


def gradients(T, N, K, dx=True, dw=True):
    """(dx's Shape, dW's, whether they share a launch, whether dx's tiles come
    first in one of 256-wide tiles)."""
    a, b, first = _out(), _out(), ctypes.c_int(0)
    pair = lib().gradients_of(T, N, K, dx, dw, a, b, ctypes.byref(first))
    return Shape(*a), Shape(*b), bool(pair), bool(first.value)


def round8(n):
    return -(-n // 8) * 8


def forward(T, N, K, keep=False):
    """The forward product's Shape, or None where it goes by the weight's rows
    (x and W contiguous and starting on 16 bytes)."""
    if lib().by_rows(T, N, K, keep, K % 8 == 0):
        return None
    return choose(FORWARD, N, T, round8(K))[0]


def forms(T, N, K):
    """The launches that a forward product (z kept or not) and both gradients
    together and alone take: kernel form, and whether the contraction is split."""
    name = lambda s: (s.bi, s.bj, s.bk, s.halves, s.splits > 1)  # noqa: E731
    out = set()
    for keep in (False, True):
        s = forward(T, N, K, keep)
        out.add(("forward by rows", min(T, 3)) if s is None else ("forward",) + name(s))
    x, w, pair, first = gradients(T, N, K)
    if pair and w.bi == 256:
        out.add(("both, wide", x.bj, w.bj, "dx first" if first else "dW first"))
    elif pair:
        groups = x.tiles_i * x.tiles_j * x.splits + w.tiles_i * w.tiles_j
        out.add(("both", x.bj, 2 if groups <= 256 else 1, x.splits > 1))
    out.add(("dx",) + name(gradients(T, N, K, dw=False)[0]))
    out.add(("dW",) + name(gradients(T, N, K, dx=False)[1]))
    return out
