"""The prefill's cut of a call's weight into shares, compiled for the host from the kernels' own header."""
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]
NEVER = 2 ** 63 - 1


@pytest.fixture(scope="module")
def shares(tmp_path_factory):
    """Rows (total, min_weight, long_total, grid) -> one list of numbers a row."""
    from paged_attention_decode_kv_gb300 import build_lib
    exe = tmp_path_factory.mktemp("shares") / "prefill_shares_host"
    cmd = [build_lib.nvcc(), *build_lib.ARCH, "-std=c++17", f"-I{build_lib.CSRC}",
           str(ROOT / "tests" / "prefill_shares_host.cu"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(rows):
        text = "\n".join(" ".join(map(str, row)) for row in rows)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, timeout=60)
        assert out.returncode == 0
        return [list(map(int, line.split())) for line in out.stdout.splitlines()]

    return run


def test_number_of_shares(shares):
    """One for each block while there are few, twice as much a share where items are long, and the whole grid at any
    larger weight, past 2^39 too (one prompt of two million tokens, 64 query and 8 kv heads of 128)."""
    rows = [(1, 128, NEVER, 152), (128, 128, NEVER, 152), (1280, 128, NEVER, 152), (1280, 128, 1000, 152),
            (1280, 1024, NEVER, 152)]
    assert [r[0] for r in shares(rows)] == [1, 1, 10, 5, 1]
    large = [(2 ** b + d, 128, long, 152) for b in range(20, 47) for d in (-1, 0, 1, 129) for long in (1000, NEVER)]
    assert all(r[0] == 152 for r in shares(large))


@pytest.mark.parametrize("grid", [1, 7, 152, 400])
def test_shares_are_even(shares, grid):
    """No share is more than 1 % larger than the others once they are a few hundred tokens, at any total up to 2^46;
    they add up."""
    totals = [int(2 ** (b + f)) + d for b in range(18, 46) for f in (0, 0.3, 0.585, 0.99) for d in (-1, 0, 1)]
    for total, (ctas, weight) in zip(totals, shares([(t, 128, NEVER, grid) for t in totals])):
        last = total - (ctas - 1) * weight
        assert ctas == grid and weight >= 128
        assert weight <= last <= weight + max(grid, 0.01 * weight), total
