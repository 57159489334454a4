"""A kernel that allocates tensor memory lets the next kernel on the stream start only after that: a successor that allocates
before it waits would else hold what this one still needs, and each would wait for the other."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a16_group_quantised_gb300", "csrc")


def kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for part in re.split(r"\b__global__\b", text)[1:]:
            end = re.search(r"\n}\n", part).end()
            name = re.search(r"(\w+_kernel\w*)\s*\(", part).group(1)
            yield os.path.basename(path), name, part[:end]


FOUND = [k for k in kernels() if "tmem_alloc(" in k[2]]


def test_there_are_such_kernels():
    assert len(FOUND) >= 2


@pytest.mark.parametrize("path, name, body", FOUND, ids=[k[1] for k in FOUND])
def test_early_launch_after_the_allocation(path, name, body):
    starts = [m.start() for m in re.finditer(r"grid_dependents_launch\(\)|kv_begin\(\)", body)]
    assert starts and min(starts) > body.index("tmem_alloc("), path
