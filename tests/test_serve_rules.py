"""Rules that the packed and paged kernels apply to what they read on the
device, compiled for the host and checked there (no GPU needed)."""
import os
import subprocess

import pytest

from int4_quantized_attention_b200 import build

MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include "ra_cache.h"
#include "ra_serve.h"
int main() {
  long long a[8];
  while (scanf("%lld %lld %lld", a, a + 1, a + 2) == 3) printf("%d\n", (int)ra::row_fits((int)a[0], (int)a[1], (int)a[2]));
}
"""


@pytest.fixture(scope="module")
def row_fits(tmp_path_factory):
    d = tmp_path_factory.mktemp("rules")
    src, exe = d / "rules.cu", d / "rules"
    src.write_text(MAIN)
    subprocess.run([build.NVCC, "-std=c++17", "-arch=sm_100a", "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"),
                    "-o", str(exe), str(src)], check=True, capture_output=True, text=True)

    def run(rows):
        text = "".join(" ".join(map(str, r)) + "\n" for r in rows)
        out = subprocess.run([str(exe)], input=text, check=True, capture_output=True, text=True).stdout
        return [bool(int(x)) for x in out.split()]

    return run


def test_row_lengths_up_to_the_largest_int(row_fits):
    # a length is held against the table row without overflow, for every page size and any 32 bits
    top = 2 ** 31 - 1
    rows = []
    for shift in (4, 5, 6, 7):
        for pages in (1, 2, 7, 1000, (2 ** 30 >> shift) - 1):
            room = pages << shift
            lens = {0, 1, room - 1, room, room + 1, room + (1 << shift), -1, -top - 1, 10 ** 6, top, top - 1}
            lens |= {top - d for d in range(1, (1 << shift) + 2)} | {top // 2, top // 2 + 1}
            rows += [(n, pages, shift) for n in sorted(lens)]
    assert row_fits(rows) == [0 <= n <= p << s for n, p, s in rows]
