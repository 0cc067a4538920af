"""Waits that one lane makes for its warp, read from the source (host only): a run cannot show a missing order."""
import os
import re

from nf4_layer_streamed_b200 import build


def _functions(text):
    """(name, body) of every braced definition whose head is on one or two lines."""
    for m in re.finditer(r"\b(\w+)\([^;{}]*\)\s*\{", text):
        depth, i = 1, m.end()
        while depth and i < len(text):
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), text[m.end():i - 1]


def test_a_wait_by_one_lane_hands_its_order_to_the_warp():
    """mbarrier.try_wait acquires for the lane that makes it and a vote orders no memory: where a voted wait succeeds,
    __syncwarp stands between the vote and the return."""
    found = []
    for name in sorted(os.listdir(build.CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(build.CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for fn, body in _functions(text):
            if "mbarrier.try_wait" not in body or "__any_sync" not in body:
                continue
            found.append(fn)
            success = re.search(r"if \(__any_sync\([^;{]*\bok\)\)\s*(\{[^}]*\}|[^;]*;)", body).group(1)
            assert re.search(r"__syncwarp\(\);\s*return true;", success), (name, fn)
    assert found == ["warp_wait"]
