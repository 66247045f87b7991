"""Warps of the tensor-memory prefill kernels wait for one another with a limit.

Their roles leave a block when a wait has run out (PA_DEVERR_TIMEOUT), each warp by its own look
at the barrier: one may leave while its neighbour, which looked a moment later, goes on.  A named
barrier among warps that may have left waits for good, so there is none: the roles meet at
mbarriers alone, whose waits give up, and the block's own barrier stands where every role ends.
A wait that runs out is not provoked on a device; this reads the sources.
"""
import os
import re

import pytest

import paged_kv_cache_72_gb300.build as b


def code(name):
    text = open(os.path.join(b.CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", ["pa_prefill.cu", "pa_prefill_quant.cuh"])
def test_no_named_barriers(name):
    assert not re.search(r"\b(bar|barrier)(\.cta)?\.(sync|red)\b", code(name))


def test_roles_end_at_one_barrier_of_the_block():
    text = code("pa_prefill_quant.cuh")
    roles = text[text.index("setmaxnreg_dec"):text.index("tmem_dealloc")]
    assert roles.count("__syncthreads") == 1
    assert "__syncthreads" in roles[roles.rindex("tc_fence_before"):]


def test_waits_of_the_quantized_prefill_are_bounded():
    text = code("pa_prefill_quant.cuh")
    # a try stands in the bounded loop alone
    loop = text[text.index("auto wait_warp"):text.index("auto give_up")]
    assert text.count("mbar_try_wait") == loop.count("mbar_try_wait") == 2
    assert "c.abort" in loop and "kWaitCycles" in loop
