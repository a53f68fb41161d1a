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


def body_of(src, start):
    body = src[src.index(start):]
    return body[:body.index("\n}\n")]


@pytest.mark.parametrize("name,start", [("tl_fp8.cu", "fp8_few_kernel("), ("tl_ortho.cu", "ortho_small_kernel("),
                                        ("tl_ortho.cu", " ortho_kernel("), ("tl_norm.cu", "norm_reduce_kernel(")])
def test_early_kernels_read_what_was_written(name, start):
    """A kernel that may begin before the one ahead has completed reads none of that one's results as read-only data:
    such a load need not come after the wait, nor see what was written before it."""
    src = code(name)
    body = body_of(src, start)
    assert "griddepcontrol.wait" in body or "grid_dependency_wait()" in body
    assert "__ldg" not in body
    calls = re.findall(r"scale_words<\d+(?:, (\w+))?>\(p\.\w", body)
    assert all(c == "true" for c in calls), calls
    if calls:
        words = body_of(src, "void scale_words(")
        assert re.search(r"EARLY \? ld_written_u32\([^:]*\) : __ldg\(", words)
        assert re.search(r"uint32_t ld_written_u32\([^{]*\{[^}]*asm volatile\(\"ld\.relaxed\.gpu\.global", src)
        rest = words.replace(re.search(r"EARLY \? [^;]*;", words).group(0), "")
        assert rest.count("__ldg") == 1 and "__ldg(at + j * s.k_step)" in rest  # the tiles' bytes
