"""Properties of the kernels' sources that no run can show, checked on the text."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "randomized_norm_clipping_gb300", "csrc")


def _text(path):
    """A source without its comments."""
    with open(path) as f:
        s = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", s, flags=re.S)


def _kernels(text):
    """(name, body) of every __global__ function."""
    for m in re.finditer(r"__global__\s+void\b", text):
        at = text.index("{", m.end())
        head = re.sub(r"__launch_bounds__\s*\((?:[^()]|\([^()]*\))*\)", "", text[m.end():at])
        name = re.search(r"(\w+)\s*\(", head.replace("__cluster_dims__(2, 1, 1)", "")).group(1)
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        yield name, text[at:end]


KERNELS = [(os.path.basename(p), n, b) for p in sorted(glob.glob(os.path.join(CSRC, "*.cu")))
           for n, b in _kernels(_text(p))]

# Accesses to the shared memory of another CTA of the cluster.
REMOTE = re.compile(r"\b(st_cluster_f4|st_cluster_f32|ld_cluster_f4|st_async_f4"
                    r"|mbar_arrive_remote\w*)\s*\(")
JOINED = re.compile(r"\b(cluster_sync_all|cluster_wait)\s*\(")


def test_the_kernels_are_found():
    names = {n for _, n, _ in KERNELS}
    assert {"embed_norm_finish_kernel", "linear_gemm_pair_kernel", "dropout_kernel"} <= names


@pytest.mark.parametrize("file,name,body", [k for k in KERNELS if REMOTE.search(k[2])],
                         ids=lambda v: v if isinstance(v, str) and len(v) < 60 else "")
def test_cluster_barrier_before_the_first_remote_access(file, name, body):
    """A CTA of a cluster may be addressed only once it is known to run."""
    joined = JOINED.search(body)
    assert joined and joined.start() < REMOTE.search(body).start(), f"{file}: {name}"


# The files whose kernels may start while the kernel before them still writes
# what they read (launch.cuh).
AFTER = [p for p in sorted(glob.glob(os.path.join(CSRC, "*.cu*")))
         if '#include "launch.cuh"' in open(p).read() or p.endswith(("launch.cuh", "linear.cuh"))]


@pytest.mark.parametrize("path", AFTER, ids=os.path.basename)
def test_early_kernels_read_by_coherent_loads(path):
    """Loads of the read-only path are defined only for data that nobody writes
    while the kernel lives."""
    text = _text(path)
    for what in (r"\b__ldg\s*\(", r"\bld\.global\.nc\b",
                 r"\bconst\s+[\w:]+\s*\*\s*__restrict__"):
        found = re.search(what, text)
        assert found is None, text[max(0, found.start() - 60): found.end() + 60]


def test_early_kernels_are_looked_at():
    names = {os.path.basename(p) for p in AFTER}
    assert {"embed.cu", "dropout.cu", "linear.cu", "linear_gemm.cu", "linear_few.cu"} <= names


@pytest.mark.parametrize("path", AFTER, ids=os.path.basename)
def test_early_kernels_read_behind_their_wait(path):
    """The loads of a cache policy are volatile assembly, which the compiler keeps in
    the order of the wait; what the built-in ones are is not said."""
    text = _text(path)
    assert re.search(r"\b__ld(cg|cs|ca|cv|lu)\s*\(", text) is None
    for m in re.finditer(r'asm\s+(volatile)?\s*\(\s*"ld\.', text):
        assert m.group(1), text[m.start(): m.start() + 80]
