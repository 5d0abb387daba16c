"""Kernels that are resident while their predecessor on the stream still runs read what it may write by
coherent loads only: the read-only path requires memory that nothing writes during the whole kernel."""
import os

from causal_video_diffusion_b200 import build as cuda_build

# sources of the kernels that launch_overlapped starts, and the headers they share
SOURCES = ("cache_q8.cu", "q8.cuh", "rope_append.cuh", "window_attn.cu", "block_norm.cu", "block_norm.h",
           "sm100.cuh", "internal.h")


def test_read_only_loads_are_of_the_coefficient_tables_alone():
    found = []
    for name in SOURCES:
        with open(os.path.join(cuda_build.CSRC, name)) as f:
            for line in f:
                code = line.split("//")[0]
                if "__ldg" in code or "ld.global.nc" in code or "__restrict__" in code:
                    found.append((name, code.strip()))
    assert found == [("rope_append.cuh", "m.cs[u] = __ldg(src);")]
