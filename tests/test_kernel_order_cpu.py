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


@pytest.mark.parametrize("name,kernel", [("tl_ortho.cu", "ortho_small_kernel("), ("tl_fp8.cu", "fp8_few_kernel(")])
def test_ctas_part_after_their_remote_reads(name, kernel):
    """A CTA that reads another's shared memory has done so before the other may leave: every relaxed arrival at the
    cluster's barrier, which is not ordered after the reads, comes after one at a barrier of the CTA, and the warp that
    waits there arrives at the cluster's with release semantics."""
    src = code(name)
    body = src[src.index(kernel):]
    body = body[:body.index("\n}\n")]
    last = body.rindex("ld_cluster_f32x4(")
    relaxed = [m.start() for m in re.finditer(r"cluster_arrive_relaxed\(\)", body)]
    if relaxed:
        (handed,) = re.finditer(r"cta_barrier_arrive\((\d), (\w+)\);", body)
        assert last < handed.start() < min(relaxed)
        taken = body.index("cta_barrier_sync(%s, %s);" % handed.groups())
        assert re.match(r"\s*cluster_arrive\(\);", body[taken:].split(";", 1)[1])
    else:
        assert re.search(r"\bcluster_arrive\(\)|\bcluster_sync\(\)", body[last:])
    assert re.search(r"\bcluster_wait\(\)", body[last:])
    ptx = code("tl_ptx.cuh")
    for fn, words in (("cluster_arrive", "barrier.cluster.arrive.release;"), ("cluster_wait", "barrier.cluster.wait.acquire;")):
        assert re.search(r"void %s\(\) \{ asm volatile\(\"%s\"" % (fn, re.escape(words)), ptx), fn
