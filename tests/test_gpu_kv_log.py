"""W4A16_LOG: the attention over the paged 8-bit cache prints the kernels it launched."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import sys
sys.path[:0] = [%r, %r]
import w4a16_group_quantised_gb300 as w
from kv_reference import Problem
from test_gpu_kv_attention import run
w.load_library()
for new in ([1, 1], [1, 1], [40, 40], [1, 40]):
    run(w, Problem([n + 20 for n in new], new, 8, 2, 128, 16, "int8", "heads", "bf16", seed=1))
"""


def lines(mode):
    r = subprocess.run([sys.executable, "-c", SCRIPT % (ROOT, os.path.join(ROOT, "tests"))],
                       env=dict(os.environ, W4A16_LOG=str(mode)), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    return [line for line in r.stderr.splitlines() if line.startswith("w4a16: kv_attention ")]


def test_each_choice_once(cuda_lib):
    got = lines(1)
    assert [line.split("kernel=")[1].split()[0] for line in got] == ["few_rows", "many_rows", "few_rows+many_rows"]
    assert "tokens=2 seqs=2 longest=1 heads=8/2 D=128 page=16 int8 bf16" in got[0]


def test_every_call_and_none(cuda_lib):
    assert len(lines(2)) == 4
    assert lines(0) == []
