"""The split kernel's shared memory and TMEM by its tile (no GPU): CTAs that
share an SM never ask for more TMEM columns than it has."""
import ctypes
import itertools
import os
import subprocess

import pytest

from int4_quant_b200 import build as B

SOURCE = r"""
#include "arnq_matmul_shape.h"
extern "C" {
int columns(int tokens) { return arnq::split_columns(tokens); }
int smem(int tokens, int stages) { return arnq::split_smem(tokens, stages); }
int limit() { return arnq::kSmemLimit; }
int per_sm() { return arnq::kSmemPerSm; }
}
"""
RESERVED = 1024  # shared memory the device takes for every CTA


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    d = tmp_path_factory.mktemp("shape")
    src, so = d / "shape.cpp", d / "shape.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", B.SRC_DIR,
                    "-o", os.fspath(so), os.fspath(src)], check=True)
    return ctypes.CDLL(os.fspath(so))


def tiles(shape):
    """Every (columns, bytes of an SM's shared memory) that a launch can ask for."""
    return {(shape.columns(t), shape.smem(t, s) + RESERVED) for t in range(16, 257, 16) for s in range(1, 13)
            if shape.smem(t, s) <= shape.limit()}


def test_columns(shape):
    for t in range(16, 257, 16):
        c = shape.columns(t)
        assert c >= max(t, 32) and c & (c - 1) == 0 and (c == 32 or c < 2 * t)


def test_the_partial_sums_and_stages_fit(shape):
    for t, s in itertools.product(range(16, 257, 16), range(1, 13)):
        assert shape.smem(t, s) >= 1024 + max(s * (16384 + t * 128), t * 512)


def test_one_tile_alone(shape):
    for columns, size in tiles(shape):
        assert shape.per_sm() // size * columns <= 512, (columns, size)


def test_any_mix_of_tiles(shape):
    # the least shared memory of each column count is what a mix can use most of
    least = {}
    for columns, size in tiles(shape):
        least[columns] = min(least.get(columns, size), size)
    kinds = sorted(least.items())
    assert [c for c, _ in kinds] == [32, 64, 128, 256]
    counts = [range(shape.per_sm() // size + 1) for _, size in kinds]
    for mix in itertools.product(*counts):
        if sum(n * size for n, (_, size) in zip(mix, kinds)) <= shape.per_sm():
            assert sum(n * columns for n, (columns, _) in zip(mix, kinds)) <= 512, mix


def test_two_large_tiles_still_share_an_sm(shape):
    # where two CTAs an SM are planned: half of it less 2 KB for static shared memory, 1.25 KB in fact
    for t, s in itertools.product(range(16, 257, 16), range(1, 13)):
        plain = 1024 + max(s * (16384 + t * 128), t * 512)
        if plain <= shape.limit() // 2 - 2048:
            assert 2 * (shape.smem(t, s) + 1280 + RESERVED) <= shape.per_sm(), (t, s)
