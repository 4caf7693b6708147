"""How many rows per key head the attention's host side expects of a call
(csrc/attention_rows.h), which decides the kernel: exactly theirs for steps
whose requests all add as many tokens."""

import os
import subprocess

import pytest

from spec_verify_gb300 import build

PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include "attention_rows.h"
int main(int n, char** a) {
  for (int i = 1; i + 2 < n; i += 3)
    std::printf("%lld\\n", (long long)smp::attention_rows(std::atoll(a[i]), std::atoll(a[i + 1]), std::atoll(a[i + 2])));
}
"""


@pytest.fixture(scope="module")
def rows(tmp_path_factory):
    where = tmp_path_factory.mktemp("rows")
    (where / "rows.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, str(where / "rows.cpp"), "-o", str(where / "rows")], check=True)

    def run(cases):
        out = subprocess.run([os.path.join(where, "rows"), *(str(x) for c in cases for x in c)], check=True,
                             capture_output=True, text=True)
        return [int(x) for x in out.stdout.split()]
    return run


def test_equal_requests_count_as_they_are(rows):
    cases = [(add * batch, batch, group) for add in (1, 2, 3, 4, 5, 6, 17, 443) for batch in (1, 2, 8, 32, 1 << 20)
             for group in (1, 4, 5, 8)]
    assert rows(cases) == [t // b * g for t, b, g in cases]


def test_ragged_steps_count_a_quarter_more_than_their_average(rows):
    cases = [(127, 32, 4), (31, 8, 8), (3, 2, 1), (2, 3, 4), (1, 1 << 20, 65535), ((1 << 31) - 1, 2, 65535)]
    for (t, b, g), got in zip(cases, rows(cases)):
        assert got == -(-(t * g * 5 // 4) // b) and got * b >= t * g
