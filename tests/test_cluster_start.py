"""Shared memory of another CTA may be accessed only once that CTA runs: in every kernel of the
packed-layer blocks a barrier of the whole cluster comes before the first access (read from the
sources; the order of execution is the order of the text in these kernels)."""
import os
import re

import pytest

from diffusion_transformer_denoiser_dit_b200 import binding

CSRC = os.path.join(os.path.dirname(binding.__file__), "csrc")
REMOTE = re.compile(r"\b(st_cluster_v[24]|ld_cluster_f[24]|mbar_arrive_cluster|mma_commit_pair|tma_load_2d_pair)\(")
BARRIER = re.compile(r"\b(cluster_sync_all|cluster_all_started)\(\)")


def kernels():
    """{name: body} of the kernels that touch the shared memory of their cluster."""
    found = {}
    for f in ("op_linear.cu", "op_linear_tc.cu", "op_attention.cu", "op_attention_rows.cu", "op_rotary.cu"):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())
        for m in re.finditer(r"__global__ void[^;{]*?(\w+)\(const", text):
            body = text[m.end():]
            body = body[:body.index("\n}")]
            if REMOTE.search(body):
                found[m.group(1)] = body
    return found


def test_the_kernels_are_found():
    assert set(kernels()) == {"linear_pair_kernel", "linear_split_kernel", "attention_tc_kernel", "attention_rows_kernel"}


@pytest.mark.parametrize("name", ["linear_pair_kernel", "linear_split_kernel", "attention_tc_kernel", "attention_rows_kernel"])
def test_the_cluster_has_started_before_its_memory_is_touched(name):
    body = kernels()[name]
    barrier = BARRIER.search(body)
    assert barrier and barrier.start() < REMOTE.search(body).start()
