"""The guard of row ranges that come from device memory (csrc/kvc_rows.h), compiled for the host."""
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_compression_probe_gb300", "csrc")
PROGRAM = """
#include <cstdio>
#include "kvc_rows.h"
int main() {
  long long off, len, rows;
  while (std::scanf("%lld %lld %lld", &off, &len, &rows) == 3) std::putchar(kvc::rows_fit(off, len, rows) ? '1' : '0');
}
"""


@pytest.fixture(scope="module")
def rows_fit(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    (d / "rows.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-fwrapv", "-I", CSRC,
                    "-o", str(d / "rows"), str(d / "rows.cpp")], check=True)

    def call(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        r = subprocess.run([str(d / "rows")], input=text, text=True, capture_output=True)
        assert r.returncode == 0, r.stderr
        return [c == "1" for c in r.stdout]
    return call


def test_ranges_in_and_out_of_the_rows(rows_fit):
    """Against whole numbers of any size: offsets and lengths at their ends, no sum passes 63 bits."""
    ends = [0, 1, 2, 99, 100, 101, 2 ** 31 - 1, 2 ** 31, 2 ** 62, 2 ** 63 - 101, 2 ** 63 - 100, 2 ** 63 - 1, -1, -100, -2 ** 31, -2 ** 63]
    rng = random.Random(1)
    cases = [(o, n, r) for o in ends for n in ends for r in ends if r >= 0]
    cases += [(rng.randrange(-50, 300), rng.randrange(-5, 200), rng.randrange(0, 250)) for _ in range(2000)]
    want = [o >= 0 and n >= 0 and o + n <= r for o, n, r in cases]
    assert rows_fit(cases) == want
