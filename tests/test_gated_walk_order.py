"""The order of the gated rule's walk (csrc/fw_gated_tc.cu), on the CPU: its
three kinds of warps (workers, the MMAs' issuer, the copies') as programs over
mbarriers that know a phase by its parity alone, run through every
interleaving of a few chunks.  A wait has to see the phase that it means, not
one two further on (it would then wait for ever), and no copy may land in a
place that a product or a worker still reads."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "delta_rule_linear_dpfp_gb300", "csrc", "fw_gated_tc.cu")


def programs(fwd, tied, nch, workers):
    """(per role its steps, per barrier its arrivals).  Steps: ("wait", barrier,
    phase), ("arrive", barrier), ("mma", place, barrier), ("fetch", place),
    ("read" / "done", place).  tied: the forward's copies arrive for the state,
    and its answers' product has two barriers."""
    def my(it):
        return (f"my{it & 1}", it // 2) if tied else ("my", it)

    mma, copy, work = [], [], [("arrive", "zr")]
    for it in range(nch):
        b = it & 1
        mma += [("wait", f"fullA{b}", it // 2), ("wait", "zr", it), ("mma", f"A{b}", "m1")]
        mma += [("mma", f"A{b}", my(it)[0])] if fwd else []
        mma += [("wait", f"fullB{b}", it // 2), ("wait", "ur", it), ("mma", f"B{b}", "m2")]
    copy += [("arrive", "zr")] if fwd and tied else []
    for it in range(min(2, nch)):
        copy += [("fetch", f"A{it}"), ("fetch", f"B{it}")]
    for it in range(nch):
        copy += [("wait", "zr", it)]
        copy += [("arrive", "zr")] if fwd and tied else []
        copy += [("fetch", f"B{(it + 1) & 1}")] if 0 < it < nch - 1 else []
        copy += [("wait", *my(it))] if fwd else [("arrive", "ur"), ("wait", "ur", it)]
        copy += [("fetch", f"A{it & 1}")] if it + 2 < nch else []
    for it in range(nch):
        b = it & 1
        work += [("wait", f"fullB{b}", it // 2), ("read", f"B{b}"), ("wait", "m1", it), ("arrive", "ur")]
        work += [("wait", *my(it))] if fwd else []
        work += [("wait", "m2", it), ("done", f"B{b}"), ("arrive", "zr")]
    need = {"fullA0": 1, "fullA1": 1, "fullB0": 1, "fullB1": 1, "m1": 1, "m2": 1, "my": 1, "my0": 1, "my1": 1,
            "zr": workers + (1 if fwd and tied else 0), "ur": workers + (0 if fwd else 1)}
    return [mma, copy] + [work] * workers, need


def explore(fwd, tied, nch=5, workers=2):
    """None, or what goes wrong in some interleaving."""
    progs, need = programs(fwd, tied, nch, workers)
    names = sorted(need)
    at = {n: i for i, n in enumerate(names)}
    # program counters; per barrier (phases completed, arrivals of the present one); products and copies in flight
    first = ((0,) * len(progs), ((0, 0),) * len(names), (), ())
    seen, todo = {first}, [first]
    while todo:
        pcs, bars, products, copies = todo.pop()

        def arrive(bars, n):
            done, have = bars[at[n]]
            new = (done + 1, 0) if have + 1 == need[n] else (done, have + 1)
            return bars[:at[n]] + (new,) + bars[at[n] + 1:]

        after = []
        if products:                                     # (they end in the order of their issue)
            after.append((pcs, arrive(bars, products[0][1]), products[1:], copies))
        for c in set(copies):
            rest = list(copies)
            rest.remove(c)
            after.append((pcs, arrive(bars, "full" + c), products, tuple(rest)))
        for r, prog in enumerate(progs):
            if pcs[r] == len(prog):
                continue
            step, nb, np, nc = prog[pcs[r]], bars, products, copies
            if step[0] == "wait":
                done = bars[at[step[1]]][0]
                if (done & 1) == (step[2] & 1):           # the phase of this parity is not the last completed one
                    continue
                if done != step[2] + 1:
                    return f"role {r} takes phase {done - 1} of {step[1]} for its phase {step[2]}"
            elif step[0] == "arrive":
                nb = arrive(bars, step[1])
            elif step[0] == "mma":
                np = products + ((step[1], step[2]),)
            elif step[0] == "fetch":
                place = step[1]
                if any(p == place for p, _ in products):
                    return f"a copy into {place} under a product that reads it"
                for w in range(2, len(progs)):            # (a worker between its read and its done)
                    past = progs[w][:pcs[w]]
                    if past.count(("read", place)) != past.count(("done", place)):
                        return f"a copy into {place} under a worker that reads it"
                nc = tuple(sorted(copies + (place,)))
            after.append((pcs[:r] + (pcs[r] + 1,) + pcs[r + 1:], nb, np, nc))
        if not after and any(pcs[r] < len(p) for r, p in enumerate(progs)):
            stuck = [p[pcs[r]] for r, p in enumerate(progs) if pcs[r] < len(p)]
            return f"nothing can go on: {stuck}"
        for s in after:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return None


@pytest.mark.parametrize("nch", [1, 2, 3, 4, 7])
@pytest.mark.parametrize("fwd", [True, False], ids=["forward", "backward"])
def test_every_interleaving_ends(fwd, nch):
    assert explore(fwd, tied=True, nch=nch) is None


def test_the_copies_have_to_be_tied():
    """Workers alone on the forward's state barrier: they may go through a whole
    chunk while the copies' warp still means to see the one before, which would
    then wait for ever."""
    assert "nothing can go on" in explore(True, tied=False)


def test_the_source_is_what_is_modelled():
    with open(SOURCE) as f:
        text = f.read()
    text = text[text.index("FW_DEV void walk("):text.index("gated_tc_walk_kernel")]
    assert "mbar_init(zr, WORKERS + (MODE == kFwd ? 1 : 0))" in text
    assert "mbar_init(ur, WORKERS + (MODE == kFwd ? 0 : 1))" in text
    assert re.findall(r"wait\(my\b.*", text) == ["wait(my + (it & 1), (it >> 1) & 1);"] * 2
    assert re.findall(r"mma_commit\(my\b.*", text) == ["mma_commit(my + (it & 1));"]
    copies = text[text.index("// the copies"):text.index("bulk_wait_all();\n            if (!ok)")]
    assert len(re.findall(r"if \(MODE == kFwd\)\n\s*mbar_arrive\(zr\);", copies)) == 2
    assert re.search(r"wait\(zr, it & 1\);\n\s*if \(!ok\)\n\s*break;\n\s*if \(MODE == kFwd\)\n\s*mbar_arrive\(zr\);", copies)
