"""Orders between CTAs and launches that no run shows reliably, read from the kernels' sources: what another CTA or
launch may do early or late has to be held back by an instruction that PTX orders, not by how a compiler happens to
schedule the code."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "offload_streamed_gb300", "csrc")


def code(name):
    """A source file without its comments."""
    src = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", src, flags=re.S)


@pytest.mark.parametrize("name,kernel", [("tl_ortho.cu", "ortho_small_kernel(")])
def test_ctas_part_after_their_remote_reads(name, kernel):
    """A CTA that reads another's shared memory arrives with release semantics before the other may leave: a relaxed
    arrival is not ordered after the loads."""
    src = code(name)
    body = src[src.index(kernel):]
    body = body[:body.index("\n}\n")]
    after = body[body.rindex("ld_cluster_f32x4("):]
    assert re.search(r"\bcluster_arrive\(\)|\bcluster_sync\(\)", after), "no releasing arrival after the remote reads"
    assert "relaxed" not in after
    ptx = code("tl_ptx.cuh")
    for fn, words in (("cluster_arrive", "barrier.cluster.arrive.release;"), ("cluster_wait", "barrier.cluster.wait.acquire;")):
        assert re.search(r"void %s\(\) \{ asm volatile\(\"%s\"" % (fn, re.escape(words)), ptx), fn
