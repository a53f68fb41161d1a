"""Orders in the row operators' kernels that no run shows reliably, read from their sources (see test_kernel_order_cpu.py)."""
import re

import pytest

from test_kernel_order_cpu import code


def kernel(name, start):
    src = code(name)
    body = src[src.index(start):]
    return body[:body.index("\n}\n")]


@pytest.mark.parametrize("name,start", [("tl_grouped.cu", "grouped_few_kernel("), ("tl_grouped_dw.cu", "grouped_dw_narrow_kernel(")])
def test_ctas_part_after_their_remote_reads(name, start):
    """Relaxed arrivals at the cluster's barrier follow an arrival at one of the CTA, past which a warp arrives releasing."""
    body = kernel(name, start)
    last = body.rindex("ld_cluster_f32x4(")
    (relaxed,) = re.finditer(r"cluster_arrive_relaxed\(\)", body)
    (handed,) = re.finditer(r"cta_barrier_arrive\((\d), (\w+)\);", body)
    assert last < handed.start() < relaxed.start()
    taken = body.index("cta_barrier_sync(%s, %s);" % handed.groups())
    assert re.match(r"\s*cluster_arrive\(\);", body[taken:].split(";", 1)[1])
    assert re.search(r"\bcluster_wait\(\)", body[last:])


@pytest.mark.parametrize("name,start", [("tl_grouped.cu", "grouped_few_kernel("), ("tl_grouped_dw.cu", "grouped_dw_narrow_kernel(")])
def test_copies_are_handed_over_after_they_landed(name, start):
    """Each thread's proxy fence stands between its wait for its copies and its warp's arrival."""
    body = kernel(name, start)
    (hand,) = re.finditer(r"auto hand_over = \[&\] \{(.*?)\};", body, flags=re.S)
    assert re.search(r"fence_proxy_async_shared\(\);\s*__syncwarp\(\);\s*if \(lane == 0\) mbar_arrive\(full_bar", hand.group(1))
    calls = [m.start() for m in re.finditer(r"hand_over\(\);", body)]
    assert len(calls) == 3
    for at in calls:
        assert body[:at].rindex("cp_async_wait<") > body[:at].rfind("cp_async_commit()")


def test_the_second_launches_wait():
    """Kernels that may begin early wait before they read what the one ahead writes, and not as read-only data."""
    src = code("tl_route.cu")
    place = kernel("tl_route.cu", "sort_place_kernel(")
    assert place.index("grid_dependency_wait()") < place.index("place_all(")
    body = src[src.index("void place_entries("):src.index("void place_all(")]
    assert "__ldg" not in body
    few = kernel("tl_adapter.cu", "expand_few_kernel(")
    assert few.index("grid_dependency_wait()") < few.index("p.parts") and "__ldcg(p.parts" in few
    assert few.index("grid_dependency_wait()") < few.index("p.h[") < few.index("y =")
