"""Threads that read a ring's slot from shared memory fence their reads before they give it back (no GPU).

The next copy writes the slot through the async proxy, which no barrier alone orders behind plain reads: the compiler has put
such reads off until after the arrival, and where the copy was quicker they gave the next stage's data.  That shows only
where data come late, so the order is read from the sources."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dit_tq2_g128_gb300", "csrc")
RINGS = {  # barriers that give a slot back to a copy
    "moe_gemm.cu": r"ctl->c_empty\[",
    "attention_paged.cu": r"ctl->empty\[",
    "gemm_tc_ws.cu": r"ctl->codes_empty\[",
    "gemv.cu": r"empty\[",
}


def unfenced(text, ring):
    """The arrivals at a ring's barrier that no fence stands within six lines before."""
    lines = text.splitlines()
    at = [i for i, l in enumerate(lines) if re.search(r"mbar_arrive\(&" + ring, l)]
    assert at
    return [lines[i].strip() for i in at if not any("fence_proxy_async_smem();" in l for l in lines[max(0, i - 6):i + 1])]


def test_the_check_itself():
    assert unfenced("x = *p;\nmbar_arrive(&ctl->empty[s]);", RINGS["attention_paged.cu"]) == ["mbar_arrive(&ctl->empty[s]);"]
    assert not unfenced("x = *p;\nfence_proxy_async_smem();\nmbar_arrive(&ctl->empty[s]);", RINGS["attention_paged.cu"])


SOURCES = list(RINGS)


@pytest.mark.parametrize("source", SOURCES)
def test_reads_are_fenced(source):
    with open(os.path.join(CSRC, source)) as f:
        assert unfenced(f.read(), RINGS[source]) == []
