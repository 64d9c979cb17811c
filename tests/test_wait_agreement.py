"""CPU check on the CUDA sources: where a whole warp waits on a barrier, its lanes agree on the answer.

A bounded wait answers each lane for itself.  Lanes that left on an answer of their own would leave the others alone in
the warp-wide instructions that follow (tensor-memory accesses, full-mask shuffles), and the bounded wait would become
an unbounded one.  So a bare mbar_wait stands only where one lane waits, or where every lane goes on whatever the
answer; everything else goes through mbar_wait_warp or __all_sync."""
import glob
import os
import re

from bit_mixture_experts_top_b200 import build

ALONE = {"101": "one lane of the weight loader", "102": "one lane of the activation loader",
         "201": "one lane issues the MMAs", "202": "one lane issues the MMAs", "203": "one lane issues the MMAs",
         "711": "one lane of the loader", "712": "one lane of the loader", "9001": "one thread",
         "301": "every lane goes on, and the warp votes before it signals the stage",
         "302": "every lane goes on, and the warp votes before it signals the stage",
         "2101": "every thread of the group goes on to the group's barriers and shuffles"}


def _waits():
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\b(mbar_wait\w*|warp_wait)\(([^;{]*?wctx|[^;{]*?\bw), (\d+)", text):
            before = text[max(0, m.start() - 40):m.start()]
            yield os.path.basename(path), m.group(1), m.group(3), re.search(r"__all_sync\([^,]*, *$", before) is not None


def test_every_wait_of_a_whole_warp_has_one_answer():
    waits = list(_waits())
    assert len(waits) >= 25
    for path, name, code, agreed in waits:
        if name in ("mbar_wait_warp", "warp_wait") or agreed:
            continue
        assert name == "mbar_wait" and code in ALONE, (path, name, code)
