"""What follows a wait of the experts' products that runs out, read from the source
(CPU only: no call makes such a wait run out, and none is broken to see it)."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "moe_expert_routing_token_b200", "csrc", "expert_matmul.cu")


def kernel(name):
    """The body of a kernel, comments taken out."""
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    at = text.index("{", text.index(f" {name}("))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(name)


@pytest.mark.parametrize("name", ["expert_rows_kernel", "expert_weight_kernel"])
def test_only_whole_sums_are_handed_over(name):
    """acc_full reaches both CTAs of a pair, whose abort flags are their own: it is
    committed only while no wait of the issuing lane has run out."""
    body = kernel(name)
    commits = [m.start() for m in re.finditer(r"ptx::umma_commit_pair\(ptx::smem_u32\(&c->acc_full", body)]
    assert len(commits) == 1
    lane = body[body.index("warp == 1"):]
    assert body[:commits[0]].rstrip().endswith("if (ok)")
    # ok is what the loop's waits leave: cleared where a stage's wait runs out, and the loop over tiles ends on it
    assert re.search(r"for \([^{]*tile < tiles && ok", lane)
    waits = re.findall(r"bar_wait<true>\(full[^;]*;", lane)
    assert waits and ("ok = false" in lane or re.search(r"ok = over \? ptx::bar_wait", lane))


@pytest.mark.parametrize("name", ["expert_rows_kernel", "expert_weight_kernel"])
def test_every_wait_is_bounded_and_looked_at(name):
    """Each waiting call stands in a condition or is assigned, and carries a limit."""
    body = kernel(name)
    calls = list(re.finditer(r"ptx::(?:bar_wait<\w+>|mbar_wait(?:_cluster)?)\(", body))
    assert len(calls) >= 5
    for m in calls:
        depth, end = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(body[end], 0)
            end += 1
        assert "kWaitNs" in body[m.end():end], body[m.start():end]
        before = body[:m.start()].rstrip()
        assert before.endswith(("!", "?", ":", "&&", "(0xffffffffu,")), before[-40:]
