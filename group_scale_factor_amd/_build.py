"""Compiles the gfx950 HIP libraries in-tree with hipcc (no JIT cache, no torch extension)."""

import os
import re
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SOURCES = [os.path.join(PKG, "csrc", name)
           for name in ("mx_rearrange.hip", "mx_unrearrange.hip", "mx_quantize.hip", "mx_pad.hip")]
EXPERT_SOURCES = [os.path.join(PKG, "csrc", name)
                  for name in ("moe_tokens.hip", "fp8_quantize.hip", "mx_grouped_mm.hip", "fp8_grouped_mm.hip")]
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(PKG, "libmxrearrange.so")
EXPERTS_LIBRARY = os.path.join(PKG, "libmoeexperts.so")
ARCH = "gfx950"

HIPCC_FLAGS = [
    "--offload-arch=" + ARCH,
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-Wall",
    # no packed fp32 instructions in any generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    path = os.path.join(rocm, "bin", "hipcc")
    return path if os.path.exists(path) else "hipcc"


# DPP instructions whose DPP operand is the second operand of the operation
# (v_subrev_u32_dpp and the like). On gfx950 a v_subrev_u32_dpp has been
# measured to return the operands' difference the other way round, so the
# generated code must hold none of them.
REVERSED_DPP = re.compile(r"\bv_\w*rev\w*_dpp\b")


def device_assembly(source):
    """gfx950 assembly of one source, compiled with the library's flags."""
    flags = [f for f in HIPCC_FLAGS if f not in ("-fPIC", "-shared")]
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "device.s")
        res = subprocess.run([hipcc()] + flags + ["--cuda-device-only", "-S", "-I", INCLUDE, "-o", out, source],
                             capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("hipcc -S failed for %s:\n%s" % (source, res.stderr))
        with open(out) as f:
            return f.read()


# A scalar register that a vector instruction writes (v_readfirstlane, v_readlane, a comparison) may be read by a
# vector memory instruction five wait states later at the earliest. The compiler sees to that for its own memory
# instructions and does not look into an asm block's.
SCALAR_WAIT_STATES = 5


def _scalars(operand):
    """Numbers of the scalar registers that an operand names."""
    m = re.match(r"s(\d+)$|s\[(\d+):(\d+)\]$", operand)
    if not m:
        return set()
    return {int(m.group(1))} if m.group(1) else set(range(int(m.group(2)), int(m.group(3)) + 1))


def early_scalar_reads(assembly):
    """(vector instruction, memory instruction) pairs of one source's assembly that stand too close."""
    found = []
    for body in re.findall(r"^_Z\w+:[^\n]*\n(.*?)^\.Lfunc_end", assembly, re.S | re.M):
        lines = [line.split(";")[0].strip() for line in body.splitlines()]
        lines = [line for line in lines if line and (not line.startswith(".") or line.startswith(".LBB"))]
        ways_in = {}     # label -> the branches to it
        for i, line in enumerate(lines):
            m = re.match(r"s_c?branch\S* (\.LBB\w+)", line)
            if m:
                ways_in.setdefault(m.group(1), []).append(i)

        def walk(i, states, wanted, load, seen):
            # back from `load` over every way to it, as far as the wait states reach
            while i >= 0 and states < SCALAR_WAIT_STATES and (i, states) not in seen:
                seen.add((i, states))
                line = lines[i]
                if line.startswith(".LBB"):
                    for branch in ways_in.get(line.split(":")[0], []):
                        walk(branch, states, wanted, load, seen)
                    if i > 0 and lines[i - 1].startswith(("s_branch", "s_endpgm", "s_setpc")):
                        return       # nothing comes from above
                else:
                    name, _, operands = line.partition(" ")
                    if name.startswith("v_") and _scalars(operands.split(",")[0].strip()) & wanted:
                        found.append((line, load))
                        return
                    states += int(operands) + 1 if name == "s_nop" else 1
                i -= 1

        for i, line in enumerate(lines):
            if line.startswith(("buffer_", "global_", "scratch_", "flat_")):
                words = [w for op in line.split(None, 1)[1].split(",") for w in op.split()[:1]]
                wanted = set().union(*map(_scalars, words))
                if wanted:
                    walk(i - 1, 0, wanted, line, set())
    return found


def check_device_code():
    """Raise if any source compiles to a reversed-operand DPP instruction, or to a memory instruction too close behind
    the vector instruction that writes its scalar registers."""
    sources = SOURCES + EXPERT_SOURCES
    with ThreadPoolExecutor(4) as pool:
        for src, text in zip(sources, pool.map(device_assembly, sources)):
            bad = sorted(set(m.group(0) for m in REVERSED_DPP.finditer(text)))
            if bad:
                raise RuntimeError("%s: generated code holds %s" % (os.path.basename(src), ", ".join(bad)))
            for write, read in early_scalar_reads(text):
                raise RuntimeError("%s: fewer than %d wait states between '%s' and '%s'"
                                   % (os.path.basename(src), SCALAR_WAIT_STATES, write, read))


def _link(library, sources, verbose):
    """One library from its sources. It replaces the old one in one step from a file of this process's own, so
    concurrent builds neither collide nor expose a half-written library."""
    tmp = "%s.tmp%d" % (library, os.getpid())
    cmd = [hipcc()] + HIPCC_FLAGS + ["-I", INCLUDE, "-o", tmp] + sources
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    msgs = "\n".join(l for l in (res.stdout + res.stderr).splitlines() if "packed-fp32-ops" not in l)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + msgs)
    if verbose and msgs.strip():
        print(msgs)
    os.replace(tmp, library)


def build(verbose=False):
    """Compile libmxrearrange.so and libmoeexperts.so next to this file. Always recompiles."""
    check_device_code()
    with ThreadPoolExecutor(2) as pool:
        for done in [pool.submit(_link, LIBRARY, SOURCES, verbose),
                     pool.submit(_link, EXPERTS_LIBRARY, EXPERT_SOURCES, verbose)]:
            done.result()
    return LIBRARY


if __name__ == "__main__":
    print(build(verbose=True))
