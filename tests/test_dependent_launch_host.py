"""Kernels that start before the kernel in front of them is done (CPU only, from the sources).

`const T* __restrict__` and `__ldg` say that memory does not change while the kernel runs, which allows a read to be
moved in front of griddepcontrol.wait. They are for what no kernel of a chain writes: weights, their scales, and the
caller's tables and lengths."""
import glob
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "sparse_head_latent_b200", "csrc")
READ_ONLY = {"scale"}  # the weights' block scales
READ_ONLY_LDG = {"scale", "p.cache_len", "p.n_nodes", "p.parents", "p.table", "p.v_scale"}


def _kernels():
    """(name, parameters, body) of every __global__ function that calls griddep_wait."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cuh"))):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        for part in src.split("__global__")[1:]:
            m = re.search(r"(\w+_kernel)\(", part)
            start = part.index("{", m.end())
            depth, end = 0, start
            for end in range(start, len(part)):
                depth += {"{": 1, "}": -1}.get(part[end], 0)
                if depth == 0:
                    break
            body = part[start:end]
            if "griddep_wait()" in body:
                yield m.group(1), part[m.end():start], body


def test_nothing_a_chain_writes_is_declared_unchanging():
    names = []
    for name, params, body in _kernels():
        names.append(name)
        unchanging = set(re.findall(r"const \w+\*\s*__restrict__ (\w+)", params))
        assert unchanging <= READ_ONLY, (name, unchanging)
        loaded = set(re.findall(r"__ldg\(\s*([\w.]+)", body))
        assert loaded <= READ_ONLY_LDG, (name, loaded)
    assert {"gemm_m64_kernel", "gemm_m64_w8_kernel", "sum_segments_kernel", "tree_attn_kernel",
            "tree_combine_kernel"} <= set(names)
