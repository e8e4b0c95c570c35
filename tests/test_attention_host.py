"""Host-side parts of the attention kernels, compiled from their headers by nvcc and
run without a GPU."""
import os
import subprocess

import pytest

from ternary_weight_w1_b200 import build

PROGRAM = """
#include <cstdio>
#include "attn_chunk.cuh"
namespace chunk = bitlinear::attn::chunk;
int main()
{
    std::printf("%d", chunk::JOIN);
    for (int blocks = 1; blocks <= 192; ++blocks)
        for (int b = 0; b < blocks; ++b)
            std::printf(" %d", chunk::worker_of(b, blocks));
    std::printf("\\n");
    for (double units : {0.0, 100.0, 2.3e6, 1e12})
        std::printf("%llu ", static_cast<unsigned long long>(
                                 chunk::join_wait_ns(1000000000ull, units)));
    std::printf("\\n");
}
"""


@pytest.fixture(scope="module")
def output(tmp_path_factory):
    d = tmp_path_factory.mktemp("host")
    src, exe = d / "host.cu", d / "host"
    src.write_text(PROGRAM)
    subprocess.run([build.nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17",
                    "-I", build.CSRC, str(src), "-o", str(exe)], check=True, capture_output=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True,
                          env=dict(os.environ, CUDA_VISIBLE_DEVICES="")).stdout.splitlines()


def test_blocks_wait_only_for_blocks_that_start_before_them(output):
    # blocks start in the order of their numbers; a worker joins the parts that the
    # next `join` workers leave
    join, *workers = map(int, output[0].split())
    assert join >= 1
    at = 0
    for blocks in range(1, 193):
        worker = workers[at:at + blocks]
        at += blocks
        assert sorted(worker) == list(range(blocks))
        block = {w: b for b, w in enumerate(worker)}
        for w in range(blocks):
            for other in range(w + 1, min(w + 1 + join, blocks)):
                assert block[other] < block[w], (blocks, w, other)
    assert at == len(workers)


def test_waits_for_other_blocks_are_limited_by_the_work_of_a_launch(output):
    # a run of 32768 rows of 8 key heads behind a million keys is 2.3 million units, of
    # 0.45 us each: blocks a second apart are sound there
    none, few, long, most = map(int, output[1].split())
    assert none == 10 ** 9 and none < few < none + 10 ** 6
    assert long >= 10 ** 9 + 5 * 2.3e6 * 450
    assert most == 61 * 10 ** 9
