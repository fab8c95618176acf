"""How the convolution's prefill spreads its tokens, without a GPU: the sizes that the GPU tests take for
each of its tiles do take them."""
import os
import subprocess

import pytest

from conv_sizes import TILED
from rwkv_wkv_gb300 import build as wbuild

SOURCE = """
#include <cstdio>
#include <cstdlib>
#include "ssm_internal.h"
int main(int n, char **v) {
    for (int i = 1; i + 1 < n; i += 2) {
        const wkv7::ConvTiles t = wkv7::conv_tiles(std::atoi(v[i]), std::atoi(v[i + 1]));
        std::printf("%d %u %u %u\\n", t.tokens, t.threads, t.tiles, t.blocks);
    }
}
"""


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    where = tmp_path_factory.mktemp("conv_tiles")
    (where / "tiles.cpp").write_text(SOURCE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(wbuild.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-I", wbuild.CSRC, "-I", wbuild.INCLUDE, "-I", cuda, str(where / "tiles.cpp"), "-o",
                    str(where / "tiles")], check=True)

    def ask(*sizes):
        out = subprocess.run([str(where / "tiles"), *(str(x) for s in sizes for x in s)], check=True, capture_output=True, text=True)
        return [tuple(int(x) for x in line.split()) for line in out.stdout.splitlines()]

    return ask


def test_sizes_of_the_gpu_tests(tiles):
    got = tiles(*((ch, total) for ch, total, _ in TILED))
    assert [t[0] for t in got] == [tile for _, _, tile in TILED]
    # fewer threads than a tile's tokens and the overhang behind it are among them, for both of the long tiles
    for tile in (32, 64):
        assert any(t[0] == tile and t[1] < tile + 1 for t in got)


def test_every_token_and_channel_once(tiles):
    sizes = [(ch, total) for ch in (8, 120, 136, 504, 520, 4096, 2 ** 24) for total in (1, 8, 9, 1000, 19425, 77761, 2 ** 31 - 256)]
    for (ch, total), (tokens, threads, n, blocks) in zip(sizes, tiles(*sizes)):
        assert threads % 32 == 0 and threads <= 128
        assert (n - 1) * tokens < total <= n * tokens
        assert (blocks - 1) * threads * 4 < ch <= blocks * threads * 4
