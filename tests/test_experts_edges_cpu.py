"""Sizes at the edges of the expert layer's operators, in the headers and in the binding (no GPU)."""

import os
import shutil
import subprocess

import pytest

import group_scale_factor_amd as gsf

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_a_sort_of_no_tokens_needs_no_workspace(tmp_path):
    calls = [(0, 1, 1, 0), (0, 8, 2048, 0), (0, 1, 2049, 0), (0, 64, 4096, 0), (0, 1, 4097, -1), (0, 0, 4096, -1),
             (1, 1, 4096, 4 * 4097 * 2)]
    src, exe = tmp_path / "probe.c", str(tmp_path / "probe")
    src.write_text('#include <stdio.h>\n#include "moe/moe_tokens.h"\nint main(void) {\n' + "".join(
        '  printf("%%lld\\n", (long long)moe_sort_tokens_workspace_bytes(%d, %d, %d));\n' % c[:3] for c in calls)
        + "  return 0;\n}\n")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-I", INCLUDE, "-o", exe, str(src)], check=True)
    lines = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in lines] == [c[3] for c in calls]
    assert [gsf.moe_sort_tokens_workspace_bytes(*c[:3]) for c in calls] == [c[3] for c in calls]
