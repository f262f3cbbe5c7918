"""Kernels that start beside the kernel before them read what that one writes: none of their pointers may promise the
compiler memory that nobody writes while they run (it would read through the cache for such, or ahead of the wait)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunkwise_linear_attention_gb300", "csrc")
WAIT = "griddepcontrol.wait"


def kernels(text):
    """(name, parameters, body) of every kernel."""
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^)]*\)\s*)?(\w+)\s*\(([^)]*)\)\s*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), m.group(2), text[m.end():i]


def test_no_read_only_promises():
    found = set()
    for f in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, f)) as h:
            text = h.read()
        waits = [k for k in kernels(text) if WAIT in k[2]]
        assert text.count(WAIT) == sum(k[2].count(WAIT) for k in waits), f  # each is in a kernel that was looked at
        for name, params, body in waits:
            found.add(name)
            assert "__restrict__" not in params and "__restrict" not in body and "__ldg(" not in body, (f, name)
            # the wait comes first of all that runs
            before = [x.strip() for x in body[:body.index("asm volatile")].splitlines()]
            assert all(x.startswith(("constexpr ", "__shared__ ")) for x in before if x), (f, name, before)
            assert WAIT in body[body.index("asm volatile"):].splitlines()[0], (f, name)
    assert found == {"c8_join_kernel", "qn_join_kernel"}
