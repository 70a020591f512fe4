"""Chained launches: a kernel of the serving side starts while the one before it may still write."""
import os
import re

import context_causal_attention_tcgen05_gb300 as cpa

CSRC = os.path.join(os.path.dirname(cpa.__file__), "csrc")


def test_chained_kernels_read_by_ordinary_loads():
    """Read-only loads are for memory that nothing writes while the kernel lives, and may be moved in front of the wait
    for the kernel before."""
    chained = [f for f in os.listdir(CSRC) if re.search(r"grid_dependency_wait|serve\.cuh", open(os.path.join(CSRC, f)).read())]
    assert {"kv_attn.cu", "kv_attn_rows.cu", "kv_cache.cu", "kv_plan.cuh", "rotary.cu", "serve.cuh"} <= set(chained)
    for f in chained:
        code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())
        if f != "api.cu":  # (whose kernels are launched in order)
            assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", code), f
