"""What the expert layer's kernels compile to, read off the gfx950 assembly (no GPU): the orders that no run shows
when they are wrong."""

import re

import pytest

from group_scale_factor_amd import _build

PRODUCTS = {s.rsplit("/", 1)[1].split("_")[0]: s for s in _build.EXPERT_SOURCES if "grouped_mm" in s}
READ_BYTES = {"b32": 4, "b64": 8, "b96": 12, "b128": 16}


@pytest.fixture(scope="module")
def assembly():
    return {kind: _build.device_assembly(source) for kind, source in PRODUCTS.items()}


def kernels(text, name):
    """Instructions of the kernels whose mangled name holds `name`."""
    found = {}
    for m in re.finditer(r"^(_Z\w*%s\w*):[^\n]*\n(.*?)^\.Lfunc_end" % name, text, re.S | re.M):
        lines = [line.split(";")[0].strip() for line in m.group(2).splitlines()]
        found[m.group(1)] = [line for line in lines if line and not line.startswith(".") or line.startswith(".LBB")]
    return found


def lds_bytes_read(instructions):
    """Bytes that a lane reads from LDS."""
    total = 0
    for line in instructions:
        m = re.match(r"ds_read(2?)(?:st64)?_([bui]\d+)", line)
        if m:
            total += READ_BYTES[m.group(2)] * (2 if m.group(1) else 1)
    return total


@pytest.mark.parametrize("kind", ["mx", "fp8"])
def test_multiplying_slots_of_paired_waves_read_no_weights(assembly, kind):
    """The lead waves load the next w and its scales while the others multiply, into the place that those read a slot
    before: a slot with products may read nothing but its group's second half of t (four fragments of 32 bytes a lane,
    and a block-128 scale for each)."""
    found = kernels(assembly[kind], "mm_paired_kernel")
    assert len(found) == 2
    for name, lines in found.items():
        at = [i for i, line in enumerate(lines) if line == "s_barrier"]
        slots = [lines[a + 1: b] for a, b in zip(at, at[1:])]
        slots = [s for s in slots if any("mfma" in line for line in s)]
        assert len(slots) >= 2, name      # of lead's and of the others' loop
        for s in slots:
            assert sum("mfma" in line for line in s) == 32, name
            assert lds_bytes_read(s) == 4 * 32 + (0 if kind == "mx" else 4 * 4), name
