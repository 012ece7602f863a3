"""The rows that a thread of the page operators takes, up to the most that a call
may have: the kernels' own loop, compiled for the host."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verification_04_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "sv_pages.cuh"

// argv: a start and the next: how many rows lie between them.  Or from, to, threads: the lowest and highest row that any of the first, middle and last threads takes, and how many.
int main(int argc, char** argv)
{
    long long from, to;
    unsigned n;
    int start, next;
    if (argc == 3 && sscanf(argv[1], "%d", &start) == 1 && sscanf(argv[2], "%d", &next) == 1) {
        printf("%d\n", sv::packed_count(start, next));
        return 0;
    }
    if (argc != 4 || sscanf(argv[1], "%lld", &from) != 1 || sscanf(argv[2], "%lld", &to) != 1 || sscanf(argv[3], "%u", &n) != 1)
        return 1;
    const unsigned threads[3] = {0, n / 2, n - 1};
    for (unsigned me : threads) {
        long long low = 0, high = -1, count = 0;
        sv::every(from, to, me, n, [&](auto r) {
            const long long x = r;
            if (count == 0 || x < low)
                low = x;
            if (count == 0 || x > high)
                high = x;
            ++count;
        });
        printf("%lld %lld %lld\n", low, high, count);
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    nvcc = shutil.which("nvcc") or os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    if not os.path.exists(nvcc):
        pytest.skip("needs nvcc")
    d = tmp_path_factory.mktemp("rows")
    (d / "rows.cu").write_text(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    "-o", str(d / "rows"), str(d / "rows.cu")], check=True)
    return str(d / "rows")


MOST, THREADS = 2 ** 31 - 1, 152 * 1024


@pytest.mark.parametrize("start,rows,threads", [(0, 0, 1024), (3, 10, 1024), (0, 5000, 1024), (MOST, MOST, THREADS), (MOST - 1, MOST, THREADS), (0, MOST, THREADS),
                                                (7, MOST, THREADS), (MOST - THREADS, MOST, THREADS), (MOST - THREADS + 1, MOST - 5, THREADS)])
def test_every_thread_stays_within_the_rows(program, start, rows, threads):
    out = subprocess.run([program, str(start), str(rows), str(threads)], check=True, capture_output=True, text=True, timeout=60).stdout
    got = [tuple(int(v) for v in line.split()) for line in out.splitlines()]
    for me, (low, high, count) in zip((0, threads // 2, threads - 1), got):
        want = range(start + me, rows, threads)
        assert count == len(want)
        assert not count or (low, high) == (want[0], want[-1])


def test_no_row_is_counted_in_32_bits():
    """No loop of the page kernels steps a 32-bit row by the number of threads."""
    with open(os.path.join(CSRC, "sv_pages.cuh")) as f:
        loops = [line.strip() for line in f if "for (" in line and "nthr" in line]
    assert loops and all(line.startswith("for (long long ") for line in loops)


@pytest.mark.parametrize("start,next,count", [(0, 0, 0), (3, 10, 7), (0, MOST, MOST), (MOST, MOST, 0), (5, 4, -1), (-1, 3, -1), (-1, -1, -1), (-3, -2, -1), (MOST, 0, -1),
                                              (2000000000, -2000000000, -1), (-2000000000, 100, -1), (-2000000000, 2000000000, -1), (MOST, -MOST - 1, -1)])
def test_starts_whose_difference_wraps(program, start, next, count):
    got = subprocess.run([program, str(start), str(next)], check=True, capture_output=True, text=True, timeout=60).stdout
    assert int(got) == count
