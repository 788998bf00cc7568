"""The sources of the serving operators' kernels, which start while the kernel before them still runs: no load that the
compiler or the read-only cache may serve from before their wait."""
import os
import re

import pytest

from lattice_vq_weight_gb300 import build

FILES = sorted(f for f in os.listdir(build.CSRC) if f.endswith((".cu", ".cuh")) and (
    f == "lq_serve.cuh" or '#include "lq_serve.cuh"' in open(os.path.join(build.CSRC, f)).read()
    or '#include "lq_attn_paged.cuh"' in open(os.path.join(build.CSRC, f)).read()))


def code(name):
    text = open(os.path.join(build.CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_the_files_are_found():
    assert {"lq_kv_plan.cu", "lq_rope.cu", "lq_kv_paged.cu", "lq_attn_paged.cu", "lq_attn_paged_tiles.cu",
            "lq_verify.cu"} <= set(FILES)


@pytest.mark.parametrize("name", FILES)
def test_no_read_only_loads(name):
    found = re.findall(r"__ldg\s*\(|ld\.global(?:\.\w+)*\.nc|__restrict__", code(name))
    assert not found, f"{name}: {len(found)} loads or pointers promised to be read-only while the kernel runs"
