"""The softmax loss's plans, compiled for the CPU: every tile, piece and part is covered once and fits
its workspace, and the sizes of the GPU tests reach every kernel."""
import os
import random
import subprocess

import pytest

from conftest import ROOT

FIELDS = ("f_tile", "f_narrow", "f_tiles", "f_run", "f_segments", "tile", "piece", "pieces", "width", "x_tile", "x_splits",
          "x_each", "w_tile", "w_splits", "w_each", "nx_splits", "nx_run", "nw_splits", "nw_run", "narrow_rows")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("loss_plan") / "plan")
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "table_embedding_bag_amd", "csrc"),
                    os.path.join(ROOT, "tests", "loss_plan_host.cpp"), "-o", exe], check=True)

    def run(cases):
        text = "".join("%d %d %d %d %d\n" % c for c in cases)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")[:-1]
        return [dict(zip(FIELDS, map(int, line.split()))) for line in out]
    return run


def up(n, d):
    return -(-n // d)


def cases(count):
    r = random.Random(0)
    log = lambda hi: int(2 ** r.uniform(0, hi))  # noqa: E731
    for _ in range(count):
        n, v, k, dtype = log(24), log(30), log(14), r.randrange(3)
        if n * k > 1 << 33 or v * k > 1 << 36:
            continue
        yield n, v, k, 0, dtype
        if dtype and k <= 128:
            yield n, v, up(k, 8) * 8, 1, dtype


def test_every_part_is_covered_once(plans):
    sizes = list(cases(4000))
    for (n, v, k, narrow, dtype), p in zip(sizes, plans(sizes)):
        what = (n, v, k, narrow, dtype)
        per = {1: 128, 4: 64}[p["f_narrow"]] if narrow else (128 if p["f_tile"] == 32 else p["f_tile"])
        assert p["f_tiles"] == up(v, per), what
        assert (p["f_segments"] - 1) * p["f_run"] < p["f_tiles"] <= p["f_segments"] * p["f_run"], what
        rows = {1: 64, 4: 256}[p["f_narrow"]] if narrow else p["f_tile"]
        assert up(n, rows) * p["f_segments"] * 512 < 1 << 32, what     # threads of a launch
        if narrow:
            for splits, run, t in ((p["nx_splits"], p["nx_run"], up(v, 64)), (p["nw_splits"], p["nw_run"], up(n, 64))):
                assert (splits - 1) * run < t <= splits * run, what
            assert p["narrow_rows"], what
            continue
        e = 4 if dtype == 0 else 2
        assert (p["pieces"] - 1) * p["piece"] < v <= p["pieces"] * p["piece"], what
        assert p["width"] >= p["piece"] and p["width"] * e % 128 == 0 and p["width"] <= 1 << 20, what
        # tiles of the logits cover a row of their gradients to its end
        assert up(p["piece"], p["tile"]) * p["tile"] >= p["width"], what
        assert up(n, p["tile"]) * up(p["piece"], p["tile"]) * 512 < 1 << 32, what
        for out, depth, name in ((n, p["piece"], "x"), (p["piece"], n, "w")):
            assert (p[name + "_splits"] - 1) * p[name + "_each"] < depth <= p[name + "_splits"] * p[name + "_each"], what
            assert p[name + "_each"] % 64 == 0, what
            t = p[name + "_tile"]
            assert up(out, t) * up(k, t) * p[name + "_splits"] * 512 < 1 << 32, what


def test_gpu_tests_reach_every_kernel(plans):
    """By tile and type: forward, gradients of the logits, and both products."""
    from test_gpu_softmax_loss import SIZES
    seen = set()
    sizes = [(n, v, d, int(dt != "fp32" and d <= 128 and d % 8 == 0), {"fp32": 0, "fp16": 1, "bf16": 2}[dt])
             for n, v, d, dt in SIZES]
    for (n, v, k, narrow, dtype), p in zip(sizes, plans(sizes)):
        if narrow:
            seen |= {("narrow", p["f_narrow"], k > 64, dtype), ("nx", p["nx_splits"] > 1, dtype),
                     ("nw", p["nw_splits"] > 1, dtype)}
            continue
        layout = 2 if k * (4 if dtype == 0 else 2) % 16 == 0 else 1 if dtype == 0 or k % 2 == 0 else 0
        seen |= {("forward", p["f_tile"], layout, dtype), ("logits", p["tile"], layout, dtype), ("x", p["x_tile"], layout, dtype),
                 ("w", p["w_tile"], dtype), ("w splits", p["w_splits"] > 1, dtype), ("pieces", p["pieces"] > 1)}
    want = {("pieces", True), ("pieces", False)}
    for dtype in range(3):
        tiles = (64, 128) if dtype == 0 else (64, 128, 256)
        layouts = (1, 2) if dtype == 0 else (0, 1, 2)
        want |= {(name, t, lay, dtype) for name in ("forward", "logits", "x") for t in tiles for lay in layouts}
        want |= {("forward", 32, lay, dtype) for lay in layouts}
        want |= {("w", t, dtype) for t in tiles} | {("w splits", s, dtype) for s in (True, False)}
        if dtype:
            want |= {("narrow", q, wide, dtype) for q in (1, 4) for wide in (True, False)}
            want |= {(name, s, dtype) for name in ("nx", "nw") for s in (True, False)}
    assert want <= seen, sorted(want - seen, key=str)
