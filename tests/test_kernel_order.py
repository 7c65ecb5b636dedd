"""Order of what a kernel takes and waits for, read from its source: two kernels that each hold what the
other waits for would never end, which no test on a GPU may try."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rope_kv_cache_gb300", "csrc")


def kernels():
    """(file, name, body) of every __global__ function."""
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name)).read()
        text = re.sub(r"//[^\n]*", "", text)
        for m in re.finditer(r"__global__[^;{]*?(\w+)\s*\((?:[^()]|\([^()]*\))*\)\s*\{", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            yield name, m[1], text[m.end():i]


ALL = list(kernels())
TMEM = [k for k in ALL if "tcgen05.alloc" in k[2]]


def test_kernels_are_found():
    assert {"rows_kernel", "prefix_kernel"} == {k[1] for k in TMEM}
    assert len(ALL) >= 8


@pytest.mark.parametrize("file,name,body", TMEM, ids=[k[1] for k in TMEM])
def test_tensor_memory_is_taken_after_the_wait_for_the_grids_in_front(file, name, body):
    """What is held while a grid in front still needs its own may be what that grid waits for. A kernel
    without such a wait is no dependent launch."""
    waits = [m.start() for m in re.finditer(r"griddepcontrol\.wait", body)]
    if waits:
        assert max(waits) < body.index("tcgen05.alloc")
    else:
        host = open(os.path.join(CSRC, "ropekv_attention.cu")).read()
        calls = re.findall(r"constexpr auto kern = ropekv_attn::%s\b.*?return launch\((.*?)\);" % name, host, re.S)
        assert calls and all(c.split(",")[4].strip() == "false" for c in calls), "launched as a dependent"
