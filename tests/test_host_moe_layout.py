"""CPU test of the sorted order's row arithmetic (csrc/moe_layout.h), compiled for the host: every count, alignment and number
of rows that the C entry accepts, up to 2^31 - 1, where a count and an alignment together, or a row and 64, are past an int."""
import os
import subprocess

import pytest

from test_host_rht_exact import HERE, _hipcc

TOP = 2 ** 31 - 1


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not available")
    out = str(tmp_path_factory.mktemp("moe_layout") / "moe_layout_host")
    subprocess.run([hipcc, "-x", "hip", "--cuda-host-only", "-O2", "-std=c++17", os.path.join(HERE, "host", "moe_layout_host.hip"), "-o", out],
                   check=True, capture_output=True, text=True)

    def run(lines):
        return subprocess.run([out], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True).stdout.splitlines()
    return run


def test_padded_runs(layout):
    cases = [(0, 1), (0, TOP), (1, TOP), (2, TOP), (TOP, TOP), (TOP, 1), (TOP - 1, 2), (7, 64), (64, 64), (65, 64), (2 ** 30, 2 ** 30), (5, 2 ** 30 - 1),
             (2 ** 30 - 1, 2 ** 30 - 1), (700_000_000, 1_500_000_000), (TOP - 63, 64), (2 ** 31 - 2 ** 20 - 5, 2 ** 20), (1_400_000_000, 715_827_882)]
    cases = [(c, a) for c, a in cases if -(-c // a) * a <= TOP]
    got = layout([f"pad {c} {a}" for c, a in cases])
    assert [int(g) for g in got] == [-(-c // a) * a for c, a in cases]


def test_rows_without_a_pair(layout):
    cases = [(0, 0, 0), (0, 1, 0), (0, 1, 1), (3, 200, 63), (TOP, TOP, 0), (TOP - 1, TOP, 0), (TOP - 1, TOP, 5), (TOP - 64, TOP, 0), (TOP - 1000, TOP, 63),
             (TOP - 129, TOP - 1, 7), (TOP - 40, TOP, 41)]
    got = layout([f"rows {a} {b} {lane}" for a, b, lane in cases])
    for (a, b, lane), line in zip(cases, got):
        rows = range(a + lane, b, 64)
        assert line == f"{len(rows)} {rows[0] if rows else 0} {rows[-1] if rows else 0}", (a, b, lane)
