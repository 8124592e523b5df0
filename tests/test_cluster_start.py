"""No kernel touches another CTA's shared memory before a cluster barrier has told it that all CTAs have begun (no GPU).

What a CTA that has not begun holds is not its own yet, and what is stored there is undefined: nothing but a barrier of the
whole cluster says that it has.  A race of this kind hardly ever shows, so the order is read from the sources."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dit_tq2_g128_gb300", "csrc")
# an access by a mapped address (`lead` is one kept as a pointer), and what ends a thread's wait for the whole cluster
ACCESS = re.compile(r"at_cta\([^;]*?\)(?:->|\[)|\*at_cta\(|\blead->|sk_mapa\(")
BARRIER = re.compile(r"\bcluster_(?:sync|wait)\(\);")


def kernels(text):
    """The bodies of a source's kernels (comments left out)."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__[^;{]*?\)\s*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield text[m.end():i]


def early(body):
    """Whether a kernel's first remote access comes before any cluster barrier."""
    access, barrier = ACCESS.search(body), BARRIER.search(body)
    return bool(access) and (barrier is None or access.start() < barrier.start())


def test_the_check_itself():
    assert early("int a; at_cta(sh, 1)->x = 2; cluster_sync();")
    assert early("push(sk_mapa(p, 1)); cluster_sync();")
    assert not early("Shared *lead = at_cta(sh, 0); cluster_arrive(); cluster_wait(); lead->x = 1;")
    assert early("cluster_arrive(); lead->x = 1; cluster_wait();")
    assert not early("cluster_sync();")


@pytest.mark.parametrize("source", ["sample.cu", "moe.cu", "skinny_mma.cu"])
def test_all_ctas_have_begun(source):
    with open(os.path.join(CSRC, source)) as f:
        bodies = list(kernels(f.read()))
    assert any(ACCESS.search(b) for b in bodies)
    assert not any(early(b) for b in bodies)
