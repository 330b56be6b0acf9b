"""Rows of a launch (csrc/mx_slabs.h), compiled for the host: every launch stays under HIP's 2^32 threads along a
dimension, and the slabs cover all rows once, up to the contract's 2^30 - 1 rows and 2^22 features."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rank_adapter_gemm_lora_amd", "csrc")

# argv: pairs of "tile blocks threads n_rows"; prints the slabs' size and each slab
PROGRAM = r"""
#include "mx_slabs.h"
#include <stdio.h>
#include <stdlib.h>
int main(int c, char **v)
{
    const long long tile = atoll(v[1]), blocks = atoll(v[2]), threads = atoll(v[3]), n = atoll(v[4]);
    lora::for_slabs(n, lora::slab_rows((int)tile, blocks, (int)threads),
                    [](int64_t r, int64_t m) { printf("%lld %lld\n", (long long)r, (long long)m); });
}
"""


@pytest.fixture(scope="module")
def slabs(tmp_path_factory):
    d = tmp_path_factory.mktemp("slabs")
    (d / "s.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(d / "s.cpp"), "-o", str(d / "s")], check=True)

    def of(tile, blocks, threads, n):
        out = subprocess.run([str(d / "s"), *map(str, (tile, blocks, threads, n))], check=True, capture_output=True, text=True)
        return [tuple(map(int, line.split())) for line in out.stdout.splitlines()]
    return of


def check(got, tile, blocks, threads, n):
    at = 0
    for r, m in got:
        assert r == at and m > 0
        assert -(-m // tile) * blocks * threads < 1 << 32
        at += m
    assert at == n
    for r, m in got[:-1]:
        assert m % tile == 0   # a tile never spans two launches


@pytest.mark.parametrize("n", (0, 1, (1 << 22) + 1, (1 << 24) + 3, (1 << 26) + 3, (1 << 30) - 1))
@pytest.mark.parametrize("threads", (64, 256, 512, 1024))
def test_a_row_a_workgroup(slabs, threads, n):
    """The norm's launches."""
    got = slabs(1, 1, threads, n)
    check(got, 1, 1, threads, n)
    assert len(got) == -(-n // (((1 << 32) - 1) // threads // 8 * 8))


# rows of a tile, features of a tile's workgroups, workgroups, threads: the product's kernels
@pytest.mark.parametrize("rows,features,per,threads", [
    (16, 32, 2, 512), (16, 64, 1, 512), (32, 64, 1, 512), (64, 64, 1, 1024), (64, 128, 1, 1024), (64, 128, 1, 512),
    (64, 128, 1, 256), (128, 128, 1, 512), (128, 256, 1, 256), (256, 256, 1, 512)])
@pytest.mark.parametrize("d", (8, 136, 28672, 1 << 22))
def test_tiles_of_a_product(slabs, rows, features, per, threads, d):
    blocks = -(-d // features) * per
    for n in (1, 35422, (1 << 30) - 1):
        check(slabs(rows, blocks, threads, n), rows, blocks, threads, n)
