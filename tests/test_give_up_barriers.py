"""The softmax groups of the e4m3 grouped-query kernel meet in named barriers
that have no time limit.  A wait that runs out in some of a group's warps must
therefore lead every warp through the same barriers.  This is a model of the
group's loop over its tiles, run for every combination of warps that give up;
which statements come before which is read from the kernel's source."""
import itertools
import os
import re

import pytest

WARPS = 4
SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "sequence_sharded_mla_gb300", "csrc", "gqa_fp8.cu")


def group_loop():
    """The loop's text, without comments."""
    text = open(SOURCE).read()
    a = text.index("for (int j = t0 + ((g ^ grp) & 1); j < t1; j += 2) {")
    return re.sub(r"//[^\n]*", "", text[a:text.index("g += t1 - t0;", a)])


def warp(tiles, gives_up, first_cleared_early):
    """The barriers of one warp, in order: yields (barrier, vote) and receives
    the vote of all.  gives_up(tile, wait) tells whether that wait runs out."""
    ok, first = True, True
    for j in range(tiles):
        ok_s = ok and not gives_up(j, "logits")
        move = first
        if not first:
            move = yield "move", not ok_s
        if move:
            if (yield "limit", not ok_s):
                ok = False
                break
            ok_pv = first or not gives_up(j, "rescale")
            if (yield "references", not ok_pv):
                ok = False
                break
        if not first and gives_up(j, "weights"):
            ok = False
            continue
        if first_cleared_early:
            first = False
        if gives_up(j, "values"):
            ok = False
            continue
        first = False
    yield "epilogue", not ok


def meet(warps):
    """Runs the warps barrier by barrier; False if they wait in different ones."""
    at = [next(w) for w in warps]
    while True:
        if len({b for b, _ in at}) != 1:
            return False
        if at[0][0] == "epilogue":
            return True
        vote = any(v for _, v in at)
        at = [w.send(vote) for w in warps]


def test_model_follows_the_source():
    body = group_loop()
    order = ["&misc->s_full[sb]", "if (!first) {", "mx > kMost || !ok_s)", "if (move) {",
             "kGroupThreads, !ok_s)", "ok_pv = first ||", "kGroupThreads, !ok_pv)",
             "if (!first && !__all_sync(0xffffffffu, poll(&misc->pv_done", "&misc->v_full[st], phase)))"]
    at = -1
    for k in order:
        at = body.index(k, at + 1)
    assert len(re.findall(r"ok = false;\s+continue;", body)) == 2
    assert body.count("named_bar_or(") == 3 and body.count("first = false;") == 1


@pytest.mark.parametrize("tiles", [1, 2, 3])
def test_warps_that_give_up_meet_the_others(tiles):
    body = group_loop()
    early = body.index("first = false;") < body.rindex("&misc->v_full[st], phase)))")
    waits = [(j, k) for j in range(tiles) for k in ("logits", "rescale", "weights", "values")]
    for who in range(1, 2 ** WARPS):
        for n in (1, 2):
            for which in itertools.combinations(waits, n):
                # the warps of `who` give up at the first wait, the others at
                # the second or not at all
                def gives_up(w):
                    mine = which[0] if who >> w & 1 else which[-1] if n == 2 else None
                    return lambda j, k: (j, k) == mine

                assert meet([warp(tiles, gives_up(w), early) for w in range(WARPS)]), (who, which)
