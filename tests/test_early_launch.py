"""Kernels that start before the kernel ahead has ended (csrc/tm_launch.cuh) must not
read through the read-only path: it wants memory that stays the same from a kernel's
start on, and theirs comes before the writes of the kernel ahead. Checked in the
sources, since a stale line would show only now and then."""
import glob
import os
import re

from long_context_prefill_trianglemix_b200 import build

READ_ONLY = re.compile(r"__ldg|__ldca|\.nc\b|__restrict__")


def code(path):
    """The source without its comments."""
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def early_kernels():
    """(file, name, body) of every kernel that waits for the one ahead."""
    out = []
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu*"))):
        for part in re.split(r"(?=__global__)", code(path))[1:]:
            if "pdl_wait()" in part:
                out.append((os.path.basename(path), part))
    return out


def test_the_kernels_are_found():
    files = [f for f, _ in early_kernels()]
    assert len(files) >= 9 and {"tm_rope.cu", "tm_kv8.cu", "tm_select.cu", "tm_kv8_attn.cuh",
                                "tm_weights.cuh"} <= set(files)


def test_no_early_kernel_reads_through_the_read_only_path():
    """Their files hold nothing but such kernels and their helpers; tm_attn.cu's own kernels are
    launched in order."""
    files = {f for f, _ in early_kernels()} | {"tm_kv8.cuh", "tm_launch.cuh"}
    assert "tm_attn.cu" not in files
    for f in sorted(files):
        found = READ_ONLY.findall(code(os.path.join(build.CSRC, f)))
        assert not found, (f, found)
