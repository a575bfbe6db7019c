"""bench.py --paged, on CPU: its cases have names of their own, floors, and cover each call and kernel."""

import bench


def test_the_paged_cases():
    operators, cases = bench.paged_cases()
    names = [c["name"] for c in cases]
    assert len(set(names)) == len(names) and names[:len(operators.listed())] == [c["name"] for c in operators.listed()]
    assert {c["op"] for c in cases} == {"attn", "accept", "commit", "update", "compact"}
    assert {c["mode"] for c in cases if c["op"] == "accept"} == {"specsample", "specexec"}
    for c in cases:
        w = operators.work(c)
        assert w["bytes"] > 0 and w["flops"] >= 0
    # both forms of update and compaction: below and past the single kernel's 32768 pages
    for op in ("update", "compact"):
        pages = [c["pages"] for c in cases if c["op"] == op]
        assert min(pages) <= 32768 < max(pages)
