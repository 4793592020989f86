"""What the kernels latch in their device error words (no GPU): bit 0 where a
bounded wait ran out, bit 1 only for a number outside its tensor, which
mhc_get_last_device_error() reports as MHC_ERR_TIMEOUT and MHC_ERR_RANGE."""

import os
import re

from mhc_pre_gb300 import build as mbuild


def test_a_wait_that_runs_out_latches_bit_0():
    """Every word outside the attention sublayer has waits only."""
    seen = 0
    for name in sorted(os.listdir(mbuild.CSRC)):
        if name.startswith(("qk_norm_rope", "paged_attn")):
            continue
        text = open(os.path.join(mbuild.CSRC, name)).read()
        for bits in re.findall(r"atomicOr\(&g_\w*error, (\w+)\)", text):
            assert bits == "1u", name
            seen += 1
    assert seen >= 10


def test_the_attention_sublayers_bits():
    """Waits next to a timer or the test hook latch bit 0, everything else bit 1."""
    waits = ranges = 0
    for name in sorted(os.listdir(mbuild.CSRC)):
        if not name.startswith(("qk_norm_rope", "paged_attn")):
            continue
        lines = open(os.path.join(mbuild.CSRC, name)).read().split("\n")
        for i, line in enumerate(lines):
            m = re.search(r"atomicOr\(&g_\w*error, (\w+)\)", line)
            if not m:
                continue
            near = "\n".join(lines[max(0, i - 2):i + 1])
            timed = re.search(r"globaltimer\(\) - \w+ > |forced_wait_runs_out|sbase & 1023u", near)
            assert m.group(1) in (("1u", "ATTN_ERR_TIMEOUT") if timed else ("2u", "ATTN_ERR_RANGE")), (name, i + 1)
            waits += bool(timed)
            ranges += not timed
    assert waits >= 4 and ranges >= 6
