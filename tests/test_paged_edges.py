"""Paged-cache and beam operators at the edges of what they take: what a CPU can check."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def source(name):
    return open(os.path.join(ROOT, "confidence_gated_kv_logits_gb300", "csrc", name)).read()


def test_softmax_warps_leave_their_loop_together():
    """Barriers of some of a block's warps wait without a limit, so after a wait that gave up (2 s) no warp may leave the
    others at one: the loop over pieces ends by a decision of all warps, and nothing that can give up lies between the
    second of its decisions and the next turn."""
    role = source("k_paged_attend_many.cu").split("// ---- softmax and epilogue ----")[1].split("\ntemplate ")[0]
    loop = re.search(r"\n    while \((.*)\) \{\n", role)
    assert loop.group(1) == "!soft_any(!next_piece())"
    body = role[loop.end():role.index("\n    }\n", loop.end())]
    leave = re.findall(r"\n      (.*(?:break|return);.*)", "\n".join(x for x in body.split("\n") if re.match(r"      \S", x)).join("\n\n"))
    assert len(leave) == 1 and leave[0].startswith("if (soft_any(")
    before, after = body.split(leave[0])
    assert "bar_wait" in before and "soft_sync" not in before
    assert "bar_wait" not in after and "next_piece" not in after
