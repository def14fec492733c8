"""What keeps the paged attention's memory accesses in range, taken from the kernel's own host functions.

A small program is compiled from the kernel's headers and prints their results; nothing runs on a GPU.
"""
import subprocess

import pytest

from haar_wavelet_patching_b200 import build

MAPS = r"""
#include <stdio.h>
#include <stdlib.h>
#include "pages.cuh"
int main(int argc, char **argv)
{
    // P, page size, heads, channels; strides of page, token, head.
    int64_t x[7];
    for (int i = 0; i < 7; ++i)
        x[i] = atoll(argv[1 + i]);
    const tok::PagesView v{nullptr, x[4], x[5], x[6]};
    const tok::PoolMap m = tok::pool_map(v, x[0], x[1], x[2], x[3]);
    for (uint64_t d : m.dims)
        printf("%lld ", (long long)d);
    for (uint64_t s : m.strides)
        printf("%lld ", (long long)s);
    printf("%lld\n", (long long)m.none);
}
"""

SPANS = r"""
#include <stdio.h>
#include <stdlib.h>
#include "pages.cuh"
int main(int argc, char **argv)
{
    for (int i = 2; i + 1 < argc; i += 2)
        printf("%d ", (int)tok::span_joins(atoi(argv[i]), atoi(argv[i + 1]), atoi(argv[1])));
}
"""


def program(folder, text):
    """The compiled program as a function of its arguments: the numbers that it prints."""
    source, target = folder / "case.cu", folder / "case"
    source.write_text(text)
    subprocess.run([build._nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "--expt-relaxed-constexpr",
                    "-I", build.INCLUDE, "-I", build.CSRC, str(source), "-o", str(target)], check=True)
    return lambda *args: [int(v) for v in subprocess.run([str(target), *map(str, args)], check=True, capture_output=True,
                                                         text=True).stdout.split()]


@pytest.fixture(scope="module")
def pool_map(tmp_path_factory):
    return program(tmp_path_factory.mktemp("maps"), MAPS)


@pytest.mark.parametrize("P", [0, 1, 2, 1000])
@pytest.mark.parametrize("page,H,D", [(1, 1, 8), (16, 2, 64), (64, 8, 128), (24, 3, 80)])
@pytest.mark.parametrize("order", ["tokens", "heads", "broadcast"])
def test_copies_of_no_page_lie_behind_the_map(pool_map, P, page, H, D, order):
    """The page that stands for none is behind the map's pages, so its copies read nothing; the map reaches no
    element that the pool has not, and without pages only one row of channels (of the queries, which have one)."""
    token, head = (H * D, D) if order == "tokens" else (D, page * D) if order == "heads" else (D, 0)
    stride = page * H * D
    numbers = pool_map(P, page, H, D, stride, token, head)
    dims, strides, none = numbers[:4], numbers[4:7], numbers[7]
    assert none >= dims[3] and none < 2 ** 31
    reach = 2 * dims[0] + sum((n - 1) * s for n, s in zip(dims[1:], strides))  # bytes from the first element to behind the last
    has = 2 * ((P - 1) * stride + (page - 1) * token + (H - 1) * head + D) if P else 2 * D
    assert dims[0] == D and all(d >= 1 for d in dims) and reach == has
    assert all(s % 16 == 0 and s >= 16 for s in strides)


def test_spans_that_no_cta_has_written_are_not_followed(tmp_path):
    """After a wait that ran out a unit's span is what the workspace held: never a place behind the CTAs', never a long loop."""
    ctas, low, high = 148, -2 ** 31, 2 ** 31 - 1
    spans = [(a, b) for a in (low, -1, 0, 5, 147, 148, high) for b in (low, -1, 0, 5, 147, 148, high)]
    got = program(tmp_path, SPANS)(ctas, *(v for s in spans for v in s))
    assert [bool(g) for g in got] == [0 <= a <= b < ctas for a, b in spans]
