"""What the epilogues of the tensor-core kernels do when a wait runs out, checked
on the source text (no GPU needed; no wait is made to run out).

The epilogue's warps read TMEM with instructions that whole warps execute, so a
warp agrees on the outcome of its wait first. Where the epilogue's warps meet at a
barrier of their own, a warp that has given up goes on taking part in it."""
import os
import re

from test_source_rules import SOURCES, _code

KERNELS = [p for p in SOURCES if re.search(r"acc_full", open(p).read())]


def test_epilogue_warps_vote():
    assert len(KERNELS) >= 6
    for p in KERNELS:
        waits = re.findall(r"[^;{}]*\bmbar_wait\(&acc_full[^;{}]*", _code(p))
        for w in waits:
            assert "__all_sync(0xffffffffu, mbar_wait(&acc_full" in w, f"{os.path.basename(p)}: {w.strip()}"


def test_a_warp_that_gave_up_keeps_the_warpgroups_barriers():
    for p in KERNELS:
        code = _code(p)
        calls = [m.start() for m in re.finditer(r"\bepi_bar\(\);", code)]
        if not calls:
            continue
        loop = code[code.index("bool dead"):]
        gave_up = loop[loop.index("if (dead)"):]
        gave_up = gave_up[:gave_up.index("continue;")]
        went_on = loop[loop.index("if (dead)") + len(gave_up):]
        assert gave_up.count("epi_bar();") == went_on.count("epi_bar();") == 2, p
        # nothing leaves the loop before the barriers
        assert "break;" not in re.sub(r"if \(c0 >= cols\) break;", "", went_on[:went_on.rindex("epi_bar();")]), p
