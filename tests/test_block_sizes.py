"""Sizes at the ends of their ranges, without a GPU: what the size functions of the operators around the
projections say, each asked in a process of its own (a division by zero ends the process)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _ask(expression):
    code = f"from bit_rank_compensated_b200 import svdq\nlib = svdq.load()\nprint({expression})"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (expression, r.returncode, r.stderr[-500:])
    return eval(r.stdout)  # noqa: S307


def test_one_group_for_all_rows_whatever_its_size():
    """rows_per_group is at least 1, without an upper limit: from the number of rows on it is one group, of the
    same workspace; near 2^31 it passes 32 bits together with the rows."""
    sizes = [(M, K) for M in (1, 2, 3, 5, 300, 4608, 2 ** 30) for K in (8, 1153, 4096, 16384)]
    large = [2 ** 31 - 1, 2147480000, 2 ** 30 + 1]
    got = _ask(f"[[lib.svdq_layer_norm_workspace_bytes(M, K, 1, r) for r in [M] + {large}] for M, K in {sizes}]")
    for (M, K), (want, *rest) in zip(sizes, got):
        assert rest == [want] * len(large), (M, K)
        assert M < 300 or want >= 2 * K * 4 * 2


@pytest.mark.parametrize("M", [2 ** 30 + 1, 2 ** 31 - 1])
def test_more_rows_than_are_taken(M):
    assert _ask(f"[lib.svdq_layer_norm_workspace_bytes({M}, 64, 1, r) for r in (1, {M}, 2 ** 31 - 1)]") == [0, 0, 0]
