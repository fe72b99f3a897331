"""Rules of the 4-bit cache's kernels that hold by their sources, checked without a GPU."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "q8_int8_block_gb300", "csrc")


def source(name):
    """A source file without its comments, and whatever of csrc it includes."""
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    return text, [h for h in re.findall(r'#include "([^"]+)"', text) if os.path.exists(os.path.join(CSRC, h))]


@pytest.mark.parametrize("name", ["q8_kv4.cu", "q8_kv4_attn.cu"])
def test_kernels_that_start_early_use_no_read_only_loads(name):
    """A kernel launched as the dependent of the one in front starts while that still writes; ld.global.nc
    (__ldg, or what const __restrict__ allows) asks for data that is constant while the kernel runs, and
    may be moved across the wait."""
    seen, todo = set(), [name]
    while todo:
        at = todo.pop()
        if at in seen:
            continue
        seen.add(at)
        text, more = source(at)
        todo += more
        found = re.findall(r"__ldg|ld\.global[.\w:]*\.nc|__restrict__", text)
        assert not found, (at, found)
    assert "griddepcontrol.wait" in "".join(source(f)[0] for f in seen)
