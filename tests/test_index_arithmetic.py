"""Index arithmetic of the device code at the largest accepted sizes, without a
GPU: the functions that the kernels call, compiled for the host."""
import os
import subprocess

import pytest

from bit_nf4_quantized_09_b200 import build

PROGRAM = r"""
#include <cstdio>
#include "kernels.h"
#include "tiles.cuh"
// grids as "ctas threads": first words and strides of threads all over the grid
int main() {
    long long ctas;
    int threads;
    while (std::scanf("%lld %d", &ctas, &threads) == 2) {
        const int marks[] = {0, 1, static_cast<int>(ctas / 2), static_cast<int>(ctas - 1)};
        for (int cta : marks)
            for (int t : {0, threads - 1}) {
                const qlora::ClearShare s(cta, static_cast<int>(ctas), t, threads);
                std::printf("%lld %d %d %d %lld %lld\n", ctas, threads, cta, t, static_cast<long long>(s.first),
                            static_cast<long long>(s.stride));
            }
    }
}
"""

# a CTA per row of the row quantiser, 128 threads up to 4096 columns and 256 above; the
# down-projections' tiles
GRIDS = [(1, 128), (148, 192), (1 << 20, 128), ((1 << 23) - 1, 256), (1 << 23, 256), (1 << 24, 128), ((1 << 24) + 5, 128),
         ((1 << 26) + 512, 192), (1 << 30, 256), ((1 << 31) - 1, 256)]


@pytest.fixture(scope="module")
def shares(tmp_path_factory):
    d = tmp_path_factory.mktemp("index")
    (d / "index.cu").write_text(PROGRAM)
    r = subprocess.run([build.NVCC, *build.ARCH, "-std=c++17", "-I" + build.CSRC, "-I" + os.path.join(build.ROOT, "include"),
                        str(d / "index.cu"), "-o", str(d / "index")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(d / "index")], input="\n".join(f"{c} {t}" for c, t in GRIDS), capture_output=True, text=True,
                         check=True)
    return [tuple(map(int, line.split())) for line in out.stdout.splitlines()]


def test_cleared_words_stay_in_the_workspace(shares):
    """A thread's words are its number in the grid, then a whole grid further on:
    nothing wraps to a word in front of the workspace."""
    assert len(shares) == 8 * len(GRIDS)
    for ctas, threads, cta, t, first, stride in shares:
        assert first == cta * threads + t, (ctas, threads, cta, t, first)
        assert stride == ctas * threads, (ctas, threads, stride)
