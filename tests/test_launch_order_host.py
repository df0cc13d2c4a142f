"""Rules of the kernel sources that no run can show reliably: no GPU needed."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "io_aware_exact_35_b200", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


def _kernels(text):
    """(name, parameters, body) of every kernel."""
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\(.*?\)\s*)?(\w+)\(", text, re.S):
        at, depth = m.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        parameters, at = text[m.end():at - 1], text.index("{", at)
        end, depth = at + 1, 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        yield m.group(1), parameters, text[at:end]


WAITS = r"griddepcontrol\.wait|wait_for_splits\(\)|chain_start\(\)|griddep_wait\(\)"


@pytest.mark.parametrize("source", ["fa_rope.cu", "fa_pages.cu", "fa_shared.cu", "fa_decode.cu"])
def test_what_an_earlier_kernel_still_writes_is_not_promised_to_be_constant(source):
    """A kernel that starts before the one ahead of it has ended and then waits for it
    must not take that one's results as `const T* __restrict__`, which promises memory
    that nobody writes while the kernel lives."""
    text = open(os.path.join(CSRC, source)).read()
    seen = 0
    for name, parameters, body in _kernels(text):
        if not re.search(WAITS, body):
            continue
        seen += 1
        promised = re.findall(r"const\s+float\d?\s*\*\s*__restrict__\s+(\w+)", parameters)
        assert not promised, f"{name}: {promised}"
    assert seen > 0


@pytest.mark.parametrize("source", SOURCES)
def test_copies_land_before_their_shared_memory_is_freed(source):
    """A kernel that fetches by TMA waits for the barriers of its copies on the way
    out, whether or not the computing warps gave up before they asked for them."""
    for name, _, body in _kernels(open(os.path.join(CSRC, source)).read()):
        if re.search(r"tma_load_3d\(|load_rows<", body):
            assert re.search(r"mbar_wait_drain\(&?\w*full", body), name
