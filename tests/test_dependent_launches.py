"""Rules of the kernels that may start while the kernel before them still runs (programmatic dependent launch).

Read from the sources, since a run cannot show them: a kernel that breaks one may still give right results for
years.  What the earlier kernel writes is not constant while the later one lives, so the later one must not read
it through the read-only path: no `const ... * __restrict__` parameter and no __ldg, other than for a caller's
inputs, which are complete before the earlier kernel starts.
"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "jagged_embedding_gb300", "csrc")
WAITS = ("wait_previous()", "wait_for_launch()", "griddepcontrol.wait")
INPUTS = {"dout"}              # a caller's inputs among the parameters
INPUT_LOADS = {"in.ids"}       # and among the loads


def _close(text, at, pair):
    """Index past the bracket that closes the one at `at`."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced")


def dependent_kernels():
    """(file, name, parameters, body) of every kernel that waits for the launch before it."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
        for m in re.finditer(r"__global__\s+void\s+", text):
            at = m.end()
            if text.startswith("__launch_bounds__", at):
                at = _close(text, text.index("(", at), "()")
            open_ = text.index("(", at)
            end = _close(text, open_, "()")
            body_at = text.index("{", end)
            body = text[body_at:_close(text, body_at, "{}")]
            if any(w in body for w in WAITS):
                found.append((os.path.basename(path), text[at:open_].strip(), text[open_ + 1:end - 1], body))
    return found


KERNELS = dependent_kernels()


def test_the_kernels_are_found():
    names = {k[1] for k in KERNELS}
    assert {"count_kernel", "scan_kernel", "scatter_kernel", "head_count_kernel", "number_kernel", "grad_small_kernel",
            "attn_fwd_kernel", "attn_dq_kernel", "attn_dkv_kernel"} <= names


@pytest.mark.parametrize("kernel", KERNELS, ids=lambda k: k[1])
def test_no_read_only_loads_of_what_the_launch_before_writes(kernel):
    _, _, params, body = kernel
    constant = set(re.findall(r"\bconst\s[^,()]*\*\s*__restrict__\s+(\w+)", params))
    assert constant <= INPUTS, constant - INPUTS
    loads = {m.strip() for m in re.findall(r"__ldg\(\s*(?:reinterpret_cast<[^>]*>\s*\()?\s*([\w.\->]+)", body)}
    assert loads <= INPUT_LOADS, loads - INPUT_LOADS


@pytest.mark.parametrize("kernel", [k for k in KERNELS if k[1].startswith("attn_")], ids=lambda k: k[1])
def test_tensor_memory_is_taken_after_the_wait(kernel):
    """Taken before it, a block could hold what the launch it waits for has yet to take, and neither would go on.
    A kernel that lets the next launch begin has its own by then."""
    body = kernel[3]
    wait, take = body.index("wait_for_launch()"), [m.start() for m in re.finditer(r"take_tmem\(|tc::alloc\(", body)]
    assert take and wait < min(take)
    let = body.find("let_next_launch()")
    assert let < 0 or max(take) < let
