"""A warp whose lanes each wait, and each leave on their own answer, can part for good
when a wait gives up: some lanes go to the kernel's last barrier while the others meet
in the loop.  That can not be run, so the source is read: each bounded wait is one
thread's, or the warp takes its answer together."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "top_routing_expert_moe_gb300", "csrc")
WAIT = re.compile(r"\b(?:wait_bar<\w+>|mbar_wait|mbar_wait_cl)\(")


def enclosing(src, at):
    """The calls and statements whose parentheses hold position ``at``, inmost first."""
    depth, names = 0, []
    for i in range(at - 1, -1, -1):
        if src[i] in ";{}" and depth == 0:
            break
        if src[i] == ")":
            depth += 1
        elif src[i] == "(":
            depth -= 1
            if depth < 0:
                depth = 0
                names.append(re.search(r"([\w:]*)\s*$", src[:i]).group(1))
    return names


def role(src, at):
    """The condition of the inmost branch on a warp or thread index around ``at``."""
    depth, i = 0, at
    while i > 0:
        i -= 1
        if src[i] == "}":
            depth += 1
        elif src[i] == "{":
            if depth:
                depth -= 1
                continue
            head = src[:i].rstrip()
            m = re.search(r"(?:if|else if) \(([^;{}]*)\)$", head)
            if m and re.search(r"\b(warp|lane|tid|threadIdx\.x|elected)\b", m.group(1)):
                return m.group(1)
    return ""


@pytest.mark.parametrize("name", ["mx4_gemm.cu", "gemm_tc.cu", "route.cu"])
def test_a_warp_gives_up_together(name):
    src = re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), open(os.path.join(CSRC, name)).read())
    seen = 0
    for m in WAIT.finditer(src):
        line = src[src.rfind("\n", 0, m.start()) + 1:m.start()]
        if "bool" in line and "=" not in line:
            continue                                        # its definition
        seen += 1
        one_thread = re.search(r"lane == 0|tid == 0|threadIdx\.x == 0|elected|threadIdx\.x & 31\) == 0", role(src, m.start()) + line)
        together = {"agreed", "__all_sync", "__shfl_sync"} & set(enclosing(src, m.start()))
        assert one_thread or together, (name, src[:m.start()].count("\n") + 1, role(src, m.start()))
    assert seen >= 3
