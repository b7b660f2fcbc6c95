"""The keys by which experts are chosen, compiled for the CPU: they keep the order of the logits, and
-infinity comes back as itself, whatever is written over its last bits."""
import os
import subprocess

import numpy as np
import pytest
import torch

from conftest import ROOT


@pytest.fixture(scope="module")
def keys(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("route_keys") / "keys")
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", os.path.join(ROOT, "table_embedding_bag_amd", "csrc"),
                    os.path.join(ROOT, "tests", "route_keys_host.cpp"), "-o", exe], check=True)

    def run(values, number):
        """float32 values' keys, and the values that the keys stand for."""
        text = "".join(f"{b} {number}\n" for b in np.asarray(values, np.float32).view(np.uint32))
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
        both = np.array(out, dtype=np.uint64).reshape(-1, 2).astype(np.uint32)
        return both[:, 0], np.ascontiguousarray(both[:, 1]).view(np.float32)
    return run


def in_order(values):
    v = np.unique(values[~np.isnan(values)])     # sorted, and -0 as 0
    return np.where(v == 0, np.float32(0), v)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_logits_of_16_bits(keys, dtype):
    """Every one: keys that end in a number of 10 bits order them and give them back."""
    every = torch.arange(-(1 << 15), 1 << 15).to(torch.int16).view(dtype).float().numpy()
    v = in_order(np.minimum(every, np.finfo(np.float32).max))
    key, back = keys(v, 1023)
    assert (key[1:] >> 10 > key[:-1] >> 10).all() and key[0] > 0
    finite = v > -np.inf
    # the largest float, which stands for +infinity, has ones in its last bits, and a negative
    # value's last bits come back as ones: below 2^-13 of it, or 2^10 times the least float, 2^-149
    assert (np.abs(back[finite] - v[finite]) <= np.abs(v[finite]) * 2.0 ** -13 + 2.0 ** -139).all()
    assert (back[1:] > back[:-1]).all()
    assert v[0] == -np.inf and back[0] == -np.inf


def test_scores_of_32_bits(keys):
    g = np.random.default_rng(0)
    top = np.finfo(np.float32).max
    v = in_order(np.concatenate([g.standard_normal(5000), [top, -top, 1e-45, -1e-45, 0, -np.inf]]).astype(np.float32))
    for number in (0, 15):
        key, back = keys(v, number)
        assert ((key | 15)[1:] >= (key | 15)[:-1]).all() and key[0] > 15
        assert back[0] == -np.inf and np.isfinite(back[1:]).all()
        assert (np.abs(back[1:].astype(np.float64) - v[1:]) <= np.abs(v[1:]) * 2.0 ** -19 + 2.0 ** -145).all()
    assert (keys(v, 0)[1] == v).all()
