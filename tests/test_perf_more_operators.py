"""The cases of perf/more_operators.py: names, ranges and what a pass cannot do without (CPU)."""
import random

import perf.more_operators as operators


def test_listed_cases():
    cases = operators.listed()
    names = [c["name"] for c in cases]
    assert 4 <= len(cases) <= 12 and len(set(names)) == len(names)
    ops = [c["op"] for c in cases]
    assert set(ops) == {"slots", "append", "select", "sparse", "logprobs"} and all(ops.count(o) >= 2 for o in set(ops))
    work = [operators.work(c) for c in cases]
    assert all(w["bytes"] > 0 and w["flops"] > 0 for w in work)
    assert max(w["bytes"] for w in work) >= 16 * min(w["bytes"] for w in work)


def test_drawn_cases_stay_below_the_largest_listed_one():
    largest = {}
    for c in operators.listed():
        w = operators.work(c)
        for k in w:
            largest[k] = max(largest.get(k, 0), w[k])
    rng = random.Random(0)
    seen = set()
    for _ in range(400):
        c = operators.draw(rng)
        assert "name" not in c
        w = operators.work(c)
        assert w["bytes"] <= largest["bytes"] and w["flops"] <= largest["flops"], c
        if c["op"] == "select":
            assert c["first"] + c["last"] < c["keep"] and c["keep"] < -(-c["hi"] // c["P"])      # there is a choice
        seen.add(repr(c))
    assert len(seen) > 390
    assert operators.draw(random.Random(5)) == operators.draw(random.Random(5))
