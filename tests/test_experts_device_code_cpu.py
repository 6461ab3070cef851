"""What the expert layer's kernels compile to, read off the gfx950 assembly (no GPU): the orders that no run shows
when they are wrong."""

import re

import pytest

from group_scale_factor_amd import _build

PRODUCTS = {s.rsplit("/", 1)[1].split("_")[0]: s for s in _build.EXPERT_SOURCES if "grouped_mm" in s}
TOKENS = [s for s in _build.EXPERT_SOURCES if s.endswith("moe_tokens.hip")][0]
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


def narrowed_lane_reads(lines):
    """(reads of a lane by number, those of them that run while a branch holds lanes back). A branch on a condition
    of the lanes saves the mask to a register and narrows it; the mask is whole again when that register comes back."""
    at = {line.split(":")[0]: i for i, line in enumerate(lines) if line.startswith(".LBB")}
    held = [None] * len(lines)      # mask registers saved and not yet back, on any way there
    work = [(0, frozenset())]
    while work:
        i, state = work.pop()
        while i < len(lines):
            if held[i] is not None and state <= held[i]:
                break
            state = held[i] = state | (held[i] or frozenset())
            line = lines[i]
            m = re.match(r"s_(and|andn2|or)_saveexec_b64 ([^,\s]+), (\S+)", line)
            if m:       # "andn2": on to the other side of a branch, whose mask lies in the second register
                state = (state - {m.group(3)} if m.group(1) != "and" else state) | {m.group(2)}
            m = re.match(r"s_xor_b64 (s[^,\s]+), exec, (\S+)", line)
            if m:       # the lanes of the other side
                state = state - {m.group(2)} | {m.group(1)}
            m = re.match(r"s_andn2_b64 exec, exec, (\S+)", line)
            if m:
                state = state | {m.group(1)}
            m = re.match(r"s_or_b64 exec, exec, (\S+)", line)
            if m:
                state = state - {m.group(1)}
            m = re.match(r"s_(c?branch\S*) (\.LBB\S+)", line)
            if m:
                work.append((at[m.group(2)], state))
            if line.startswith(("s_branch", "s_endpgm")):
                break
            i += 1
    reads = [i for i, line in enumerate(lines) if re.match(r"v_readlane_b32 s\d+, v\d+, s\d+", line)]
    return reads, [i for i in reads if held[i]]


def test_token_moves_read_slots_from_lanes_that_are_there():
    """A token's positions and weights lie one to a lane: a lane past the row's columns may not have left, or be held
    back, where they are read. (The gradient of the sum keeps masks in vector lanes, which this walk does not follow.)"""
    text = _build.device_assembly(TOKENS)
    found = {**kernels(text, "gather_kernel"), **kernels(text, "combine_kernel")}
    assert len(found) == 6
    for name, lines in found.items():
        reads, narrowed = narrowed_lane_reads(lines)
        assert reads and not narrowed, name


def test_the_build_check_finds_early_scalar_reads():
    """By hand: the pair, what stands between it, and whether it is too close. Also over a branch."""
    load = "buffer_load_dwordx4 v1, s[8:11], s40 offen lds"
    m0 = "s_mov_b32 m0, s3\ns_nop 0\n"
    for between, close in [("", True), (m0, True), (m0 + "v_mov_b32_e32 v9, 0\ns_add_i32 s3, s3, 1\n", True),
                           (m0 + "s_nop 2\n", False), ("s_nop 3\n", True), ("s_nop 4\n", False)]:
        for write, read in [("v_readfirstlane_b32 s9, v3", True), ("v_readlane_b32 s40, v250, 3", True),
                            ("v_cmp_eq_u32_e64 s[10:11], v0, v1", True), ("v_readfirstlane_b32 s12, v3", False),
                            ("s_mov_b32 s9, s4", False)]:
            text = "_Zk:  ; @_Zk\n%s\n%s;;#ASMSTART\n%s\n;;#ASMEND\ns_endpgm\n.Lfunc_end0:\n" % (write, between, load)
            found = _build.early_scalar_reads(text)
            assert found == ([(write, load)] if close and read else []), (between, write)
    loop = ("_Zk:\ns_nop 7\n.LBB0_1:\n%s\n%s\nv_readlane_b32 s40, v2, 1\ns_cbranch_scc1 .LBB0_1\ns_endpgm\n"
            ".Lfunc_end0:\n")
    assert len(_build.early_scalar_reads(loop % ("s_nop 1", load))) == 1
    assert _build.early_scalar_reads(loop % ("s_nop 3", load)) == []


@pytest.mark.parametrize("kind", ["mx", "fp8"])
def test_loads_to_lds_say_that_they_write_m0(assembly, kind):
    """Nothing that the compiler makes itself may rely on m0 around them."""
    lines = [line for found in (kernels(assembly[kind], n) for n in ("mm_tile_kernel", "mm_paired_kernel"))
             for lines in found.values() for line in lines]
    writes = [line for line in lines if re.match(r"s_mov_b32 m0, s\d+$", line)]
    assert len(writes) == sum("offen lds" in line for line in lines) > 0
    assert len([line for line in lines if re.search(r"\bm0\b", line)]) == len(writes)
    source = open(PRODUCTS["mx"].rsplit("/", 1)[0] + "/grouped_mm.h").read()
    assert source.count("offen lds") == source.count(': "m0", "memory");')


@pytest.mark.parametrize("kind", ["mx", "fp8"])
def test_barriers_of_staged_tiles_wait_for_the_reads_before_them(assembly, kind):
    """Behind a barrier the next loads write where the wave has just read: its reads are waited for at the barrier
    itself, and on every way to it in the tiles of paired waves, which wait in the slot."""
    for name, lines in kernels(assembly[kind], "mm_tile_kernel").items():
        before = [lines[i - 1] for i, line in enumerate(lines) if line == "s_barrier"]
        assert len(before) == 2, name
        assert all(line.startswith("s_waitcnt vmcnt(") and "lgkmcnt(0)" in line for line in before), (name, before)
    for name, lines in kernels(assembly[kind], "mm_paired_kernel").items():
        reading = False
        for line in lines:
            reading = (reading or line.startswith("ds_read")) and not re.match(r"s_waitcnt .*lgkmcnt\(0\)", line)
            assert line != "s_barrier" or not reading, name


def test_products_of_any_scales_take_the_instruction_without_scales(assembly):
    """Paired waves that multiply the sums by block-128 scales give the products none: every product of the row groups,
    and those that start from nothing of the token groups, whose others add to a total and take the scales."""
    for name, lines in kernels(assembly["fp8"], "mm_paired_kernel").items():
        products = [line for line in lines if "mfma" in line]
        plain = [line for line in products if line.startswith("v_mfma_f32_16x16x128_f8f6f4 ")]
        scaled = [line for line in products if line.startswith("v_mfma_scale_f32_16x16x128_f8f6f4 ")]
        assert len(plain) + len(scaled) == len(products) and plain, name
        assert all(re.search(r"\], 0$", line) for line in plain), name
        if "ILb0ELb0E" in name:
            assert not scaled, name
        else:
            assert scaled and not any(re.search(r"\], 0, ", line) for line in scaled), name


def registers(operand):
    """Scalar registers of an operand, by number."""
    m = re.match(r"s(\d+)$|s\[(\d+):(\d+)\]$", operand)
    if not m:
        return []
    return [int(m.group(1))] if m.group(1) else list(range(int(m.group(2)), int(m.group(3)) + 1))


def loads_from_unset_buffers(lines, given):
    """Loads to LDS before the first barrier whose buffer, or whose step of it, may lie in scalar registers that nothing
    on the way has set; the first `given` are set at the start. A copy of an unset register is unset, too."""
    at = {line.split(":")[0]: i for i, line in enumerate(lines) if line.startswith(".LBB")}
    unset = [None] * len(lines)
    work = [(0, frozenset(range(given, 106)))]
    found = set()
    while work:
        i, state = work.pop()
        while i < len(lines):
            if unset[i] is not None and state <= unset[i]:
                break
            state = unset[i] = state | (unset[i] or frozenset())
            line = lines[i]
            name, _, rest = line.partition(" ")
            ops = [op.strip() for op in rest.split(",")]
            if "offen lds" in line:
                used = registers(ops[1]) + registers(ops[2].split()[0])
                found.update((i, r) for r in used if r in state)
            elif name.startswith(("s_mov_b", "s_and_b")) and len(registers(ops[0])) > 0:
                to = registers(ops[0])
                froms = [registers(op) for op in ops[1:]]
                for n, r in enumerate(to):
                    bad = any(n < len(f) and f[n] in state for f in froms)
                    state = state | {r} if bad else state - {r}
            elif name.startswith(("s_", "v_")) and not name.startswith(("s_cmp", "s_cbranch", "s_branch", "s_bitcmp")):
                state = state - set(registers(ops[0]))
                if name.startswith("v_") and len(ops) > 1:      # a carry or a condition beside the vector result
                    state = state - set(registers(ops[1]) if "_co_" in name else [])
            m = re.match(r"s_(c?branch\S*) (\.LBB\S+)", line)
            if m:
                work.append((at[m.group(2)], state))
            if line.startswith(("s_branch", "s_endpgm")):
                break
            i += 1
    first = lines.index("s_barrier")
    return sorted({(lines[i], r) for i, r in found if i < first})


@pytest.mark.parametrize("kind", ["mx", "fp8"])
def test_no_first_load_goes_by_a_buffer_that_was_not_set(assembly, kind):
    """A tile with nothing to load (rows in no group) issues its loads all the same, out of range of its buffers: their
    sizes have to be set for it, too, where it is the first one of its workgroup. (Later tiles find the last one's.)"""
    text = assembly[kind]
    for name, lines in kernels(text, "mm_paired_kernel").items():
        block = text[text.index(".amdhsa_kernel " + name):]
        given = int(re.search(r"\.amdhsa_user_sgpr_count (\d+)", block).group(1)) + 1     # and the workgroup's number
        assert loads_from_unset_buffers(lines, given) == [], name
