"""Which tile each workgroup of the grouped linear layer takes, worked out on the CPU by the
kernels' own arithmetic (csrc/tiles.hpp)."""
import collections
import ctypes
import os
import subprocess

import numpy as np
import pytest

import grouped_cases

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "table_embedding_bag_amd", "csrc")
F32, F16, BF16 = 0, 1, 2
Plan = collections.namedtuple("Plan", "forward dx dw chunk slots both")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("tiles") / "tiles.so")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-Wall", "-fPIC", "-shared", "-I" + CSRC,
                           "-I" + os.path.join(ROOT, "include"), "-o", out,
                           os.path.join(HERE, "grouped_tiles_host.cpp")])
    lib = ctypes.CDLL(out)
    i64, i32 = ctypes.c_int64, ctypes.c_int32
    lib.row_tiles.restype = lib.rounds.restype = i64
    lib.rounds.argtypes = [i64, i64, i64, i32, i32]
    lib.layout.argtypes = [ctypes.c_uint64, i64, i64, i64]
    lib.plan.argtypes = [i64, i64, i64, i64, i32, i32, ctypes.c_void_p]
    return lib


def _row_tiles(host, offsets, rows, cols, TB, TA, count=True):
    """(workgroups with a tile, lowest row, highest row, times each tile was taken)"""
    off = np.ascontiguousarray(offsets, dtype=np.int64)
    groups, na = len(off) - 1, -(-cols // TA)
    blocks = na * (rows // TB + min(groups, rows))      # as launched
    c = np.clip(off, 0, rows)
    tiles = int((-(-np.maximum(np.diff(c), 0) // TB) * na).sum())
    taken = np.zeros(tiles, dtype=np.int32) if count else None
    lo, hi = ctypes.c_int64(), ctypes.c_int64()
    i64 = ctypes.c_int64
    n = host.row_tiles(off.ctypes.data_as(ctypes.c_void_p), i64(groups), i64(rows), i64(blocks), i64(na),
                       i64(TB), ctypes.byref(lo), ctypes.byref(hi),
                       taken.ctypes.data_as(ctypes.c_void_p) if count else None)
    return n, lo.value, hi.value, taken


@pytest.mark.parametrize("TB,TA", [(256, 256), (128, 128), (64, 64), (32, 128)])
def test_every_tile_is_taken_once(host, TB, TA):
    r = np.random.default_rng(TB)
    for groups, rows, cols in ((1, 1, 1), (3, 700, 300), (70, 5000, 520), (8, 8191, 1000), (200, 130, 129)):
        off = np.concatenate([[0], np.cumsum(r.multinomial(rows, r.dirichlet(np.full(groups, 0.3))))])
        n, lo, hi, taken = _row_tiles(host, off, rows, cols, TB, TA)
        assert n == len(taken) and (taken == 1).all() and (lo, hi) == (0, rows - 1)


def test_groups_that_overlap_by_more_than_the_launch_holds(host):
    """4096 groups, every other one all of 131072 rows: 2^31 tiles of 32 rows x 128 columns, where
    the launch has 2^21 workgroups."""
    off = np.arange(4097) % 2 * 131072
    n, lo, hi, _ = _row_tiles(host, off, 131072, 32768, 32, 128, count=False)
    assert n == 0   # none is taken


@pytest.mark.parametrize("TB,TA", [(256, 256), (64, 64), (32, 128)])
def test_bad_offsets_stay_within_the_rows(host, TB, TA):
    r = np.random.default_rng(TB + 1)
    for i in range(60):
        groups, rows = int(r.integers(1, 300)), int(r.integers(1, 9000))
        spread = int(r.choice([rows, 4 * rows, 2 ** 62]))
        off = r.integers(-spread, spread, groups + 1)
        if i % 3 == 0:
            off = np.arange(groups + 1) % 2 * rows
        n, lo, hi, taken = _row_tiles(host, off, rows, int(r.integers(1, 3000)), TB, TA)
        assert n >= 0 and lo >= 0 and hi < rows and (taken <= 1).all(), (i, groups, rows)


def _plan(host, rows, groups, K, M, dtype, dx=True):
    out = (ctypes.c_int64 * 6)()
    host.plan(rows, groups, K, M, dx, dtype, out)
    return Plan(*out)


def test_products_over_rows_take_the_tiles_of_the_fewest_rounds(host):
    r = np.random.default_rng(9)
    for _ in range(3000):
        rows, groups = int(2 ** r.uniform(0, 17)), int(2 ** r.uniform(0, 8))
        K, M = (int(2 ** r.uniform(0, 13)) for _ in range(2))
        for dtype in (F32, F16, BF16):
            p = _plan(host, rows, groups, K, M, dtype)
            for tile, cols in ((p.forward, M), (p.dx, K)):
                assert (tile == 32) == (rows <= 32 * groups)
                for other in (64, 128) + (() if dtype == F32 else (256,)):
                    assert tile == 32 or host.rounds(rows, groups, cols, tile, dtype) <= \
                        host.rounds(rows, groups, cols, other, dtype)


def test_fp32_takes_no_tiles_of_256(host):
    """They are no faster than four of 128: the weights' gradient of several large groups too."""
    r = np.random.default_rng(10)
    for rows, groups, K, M in [(32768, 16, 4096, 4096), (32768, 16, 2048, 2048), (40000, 1, 8192, 8192)] + [
            (int(2 ** r.uniform(5, 18)), int(2 ** r.uniform(0, 6)), int(2 ** r.uniform(8, 14)), int(2 ** r.uniform(8, 14)))
            for _ in range(2000)]:
        p = _plan(host, rows, groups, K, M, F32)
        assert max(p.forward, p.dx, p.dw) <= 128, (rows, groups, K, M, p)


@pytest.mark.parametrize("case", list(grouped_cases.cases()), ids=grouped_cases.name)
def test_kernel_cases_take_the_tiles_they_name(host, case):
    product, tile, chunked, layout, rows, groups, K, M, dtype = case
    code, size = {"fp32": (F32, 4), "fp16": (F16, 2), "bf16": (BF16, 2)}[dtype]
    p = _plan(host, rows, groups, K, M, code, dx=product == "both")
    took = {"forward": p.forward, "dx": p.dx, "dw": p.dw, "both": p.dw}[product]
    assert took == tile and p.both == (product == "both")
    if product in ("dw", "both"):
        assert (p.slots > 0) == chunked
    operands = (K,) if product == "forward" else (K, M)
    assert min(host.layout(4096, n, n, size) for n in operands) == layout


def test_every_kernel_has_a_case():
    """The kernels that are compiled: forward and dx with tiles of 256 (2-byte values alone), 128, 64
    and 128 x 32, the weights' gradient and both gradients with the square ones."""
    have = {(c[0], c[1], c[3], c[8]) for c in grouped_cases.cases()}
    for dtype, layouts in (("fp32", (1, 2)), ("fp16", (0, 1, 2)), ("bf16", (0, 1, 2))):
        square = (64, 128) if dtype == "fp32" else (64, 128, 256)
        for layout in layouts:
            for product in ("forward", "dx", "dw", "both"):
                for tile in square + ((32,) if product in ("forward", "dx") else ()):
                    assert (product, tile, layout, dtype) in have
