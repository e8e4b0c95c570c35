"""Host-side parts of the attention kernels, compiled from their headers by nvcc and
run without a GPU."""
import itertools
import os
import subprocess

import pytest

from ternary_weight_w1_b200 import build

PROGRAM = """
#include <cstdio>
#include "attn_chunk.cuh"
#include "row_set.cuh"
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
    // addresses and strides in steps of 8 elements; the sets lie in 16-byte units
    for (int sa = 2; sa <= 5; ++sa)
        for (int sb = 2; sb <= 5; ++sb)
            for (int wa = 1; wa <= 2; ++wa)
                for (int wb = 1; wb <= 2; ++wb)
                    for (int n = 1; n <= 4; ++n)
                        for (int at = 0; at <= 48; ++at) {
                            const bitlinear::RowSet a{reinterpret_cast<void *>(1024 + 16 * 24),
                                                      8 * sa, 8 * wa};
                            const bitlinear::RowSet b{reinterpret_cast<void *>(1024 + 16 * at),
                                                      8 * sb, 8 * wb};
                            std::printf("%d", bitlinear::share_memory(a, b, n) ? 1 : 0);
                        }
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


def test_row_sets_that_share_memory(output):
    # against the sets' elements one by one, with equal and with other strides
    got = iter(output[2])
    seen = set()
    for sa, sb, wa, wb, n in itertools.product(range(2, 6), range(2, 6), (1, 2), (1, 2),
                                               range(1, 5)):
        a = {24 + i * sa + w for i in range(n) for w in range(wa)}
        for at in range(49):
            b = {at + i * sb + w for i in range(n) for w in range(wb)}
            assert next(got) == str(int(bool(a & b))), (sa, sb, wa, wb, n, at)
            seen.add(bool(a & b))
    assert next(got, None) is None and seen == {False, True}
