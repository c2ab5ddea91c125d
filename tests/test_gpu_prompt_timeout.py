"""Prompt attention's bounded waits, without a fault: a test-only setting makes the
warp that announces each CTA's work start with a wait that nothing ends. It runs
out after a short limit, and every other role (the loaders, both issuers, the
softmax warps, for the 4-bit cache the warps that make its tiles) gives up in its
own first wait. The call must report DDT_DEV_TIMEOUT and end by itself, and the
context's next call must be normal."""
import pytest
import torch

from packed_ref import Packed, check_close
from speculative_decoding_draft_depth_gb300 import ddt

pytestmark = pytest.mark.gpu

WAIT_CYCLES = 2_000_000  # about 1 ms at the SM clock


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,ctx", [([40], [100]), ([300, 0, 20], [700, 5, 2000])])
def test_waits_run_out_and_the_context_recovers(bits, d, lens, ctx):
    p = Packed(lens, ctx, 8, 2, d, 16, bits, seed=64)
    p.fill_context()
    p.fill_new()
    want, tol = p.attention64()
    first = p.attend()
    check_close(first, want, tol)
    assert p.h.ddt_device_status() == 0
    p.h.ddt_debug_arm_prompt_timeout(WAIT_CYCLES)
    p.attend()
    assert p.h.ddt_device_status() == ddt.DEV_TIMEOUT
    # (one-shot)
    again = p.attend()
    assert p.h.ddt_device_status() == 0
    assert torch.equal(again.view(torch.int16), first.view(torch.int16))
    p.h.ddt_debug_arm_prompt_timeout(WAIT_CYCLES)
    p.h.ddt_debug_arm_prompt_timeout(0)  # disarm
    again = p.attend()
    assert p.h.ddt_device_status() == 0
    assert torch.equal(again.view(torch.int16), first.view(torch.int16))


def test_the_kernel_of_few_rows_has_no_waits():
    """It runs as ever; the setting is still there for the next tensor-core launch."""
    p = Packed([1, 1, 1], [100, 700, 3], 8, 2, 128, 16, 4, seed=65)
    p.fill_context()
    p.fill_new()
    want, tol = p.attention64()
    p.h.ddt_debug_arm_prompt_timeout(WAIT_CYCLES)
    check_close(p.attend(), want, tol)
    assert p.h.ddt_device_status() == 0
    p.h.ddt_debug_arm_prompt_timeout(0)
