"""The row-tile weights kernel's barriers as its source has them, run on the CPU.

Ring sizes, arrival counts, and the barrier and parity of every wait and arrival are read from
csrc/kv4_wtile.cu and evaluated; only the roles' loops are restated here.  Each warp that
arrives is a role of its own.  Roles advance in random order; every wait must be for the phase that it
means (a role's i-th wait on a barrier is for the i-th completion), and all must come to their end.
"""

import os
import random
import re

import pytest

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "context_ring_attention_step_gb300",
                    "csrc", "kv4_wtile.cu")
SOURCE = re.sub(r"//[^\n]*", "", open(PATH).read())
COMMENTED = open(PATH).read()


def py(expr):
    """A C expression over whole numbers that are not negative, as Python."""
    expr = re.sub(r"\(uint32_t\)|C::|WTile<D>::", "", " ".join(expr.split())).replace("/", "//")
    m = re.fullmatch(r"(.+?) \? (.+?) : (.+)", expr)
    return "(%s if %s else %s)" % (py(m[2]), m[1], py(m[3])) if m else expr


def value(expr, names):
    return int(eval(py(expr), {}, names))


def constants(d):
    names = {"D": d}
    names["kLseStages"] = int(re.search(r"constexpr int kLseStages = (\d+);", SOURCE)[1])
    body = SOURCE[SOURCE.index("struct WTile {"):]
    for name, expr in re.findall(r"static constexpr int (k\w+) = ([^;]+);", body[:body.index("};")]):
        names[name] = value(expr, names)
    names.update(N=names["kN"], QS=names["kQStages"], LS=names["kLseStages"])
    for name, off in re.findall(r"const uint32_t (b_\w+) = smem_u32\(bars(?: \+ ([^)]+))?\);", SOURCE):
        names[name] = 8 * value(off or "0", names)
    return names


def args_at(text, start):
    """The arguments of a call whose opening bracket is at `start`."""
    out, depth, last = [], 0, start + 1
    for i in range(start, len(text)):
        depth += text[i] in "([{"
        depth -= text[i] in ")]}"
        if (text[i] == "," and depth == 1) or depth == 0:
            out.append(text[last:i].strip())
            last = i + 1
        if depth == 0:
            return out


def calls(text, name):
    return [args_at(text, m.end() - 1) for m in re.finditer(r"\b%s\(" % name, text)]


def section(begin, end):
    """The source of one role, by the headings over the roles."""
    a = COMMENTED.index(begin)
    return re.sub(r"//[^\n]*", "", COMMENTED[a:COMMENTED.index(end, a)])


ISSUE = section("- MMA issuers", "- query tiles")
QUERY = section("- query tiles", "- log-sum-exps and limits")
LSE = section("- log-sum-exps and limits", "- exponentials and sums")
SUM = section("- exponentials and sums", "- expansion")
EXPAND = section("- expansion", "template <int D>\ncudaError_t launch(")
WAITS = {a[3]: a[:2] for a in calls(SOURCE, "mbar_wait")}


def advance(text, ring, names, at, phase):
    """`if (++at == RING) { at = 0; phase ^= 1; }`, as the source has it."""
    assert re.search(r"if \(\+\+%s == %s\) \{ %s = 0; %s \^= 1; \}" % (at, ring, at, phase), text)
    names[at] += 1
    if names[at] == names[ring]:
        names[at] = 0
        names[phase] ^= 1


def run(d, items, seed):
    rnd, base = random.Random(seed), constants(d)
    need, got, done = {}, {}, {}
    init = re.search(r"if \(tid == 0\) \{(.*?)fence_mbar_init", SOURCE, re.S)[1]
    for bound, body in re.findall(r"for \(int i = 0; i < (\w+); \+\+i\) \{(.*?)\n    \}", init, re.S):
        for i in range(value(bound, base)):
            for at, count in calls(body, "mbar_init"):
                at = value(at, dict(base, i=i))
                assert at not in need, "two barriers in one place"
                need[at], got[at], done[at] = value(count, base), 0, 0

    def wait(names, site, seen, late=0):
        at, parity = (value(e, names) for e in WAITS[site])
        phase = seen.get(at, 0) - late
        seen[at] = seen.get(at, 0) + 1
        return at, parity, phase

    def arrive(names, expr):
        return (value(expr, names),)

    def issuer(kt):
        v = dict(base, kt=kt, g=0, qs=0, qph=0, ls=0, lph=0)
        seen = {}
        sb, back = (re.search(r"const uint32_t %s = ([^;]+);" % n, ISSUE)[1] for n in ("sb", "back"))
        commits = [a[0] for a in calls(ISSUE, "umma_commit")]
        assert commits[:3] == ["b_sfull + 8 * (4 * kt + sb)", "b_qempty + 8 * qs", "b_lempty + 8 * ls"] and "kempty" in commits[3]
        for v["item"], tiles in enumerate(items):
            v["set"] = value(re.search(r"set = ([^;]+);", ISSUE)[1], v)
            yield wait(v, "160", seen)
            for _ in range(tiles):
                yield wait(v, "161", seen)
                yield wait(v, "168", seen)
                v["sb"], v["back"] = value(sb, v), value(back, v)
                if v["g"] >= v["back"]:
                    yield wait(v, "162", seen)
                for e in commits[:3]:
                    yield arrive(v, e)
                advance(ISSUE, "QS", v, "qs", "qph")
                advance(ISSUE, "LS", v, "ls", "lph")
                v["g"] += 1
            yield arrive(v, commits[3])

    def query():
        v, seen = dict(base), {}
        (at, _), = calls(QUERY, "mbar_expect_tx")
        for v["g"] in range(sum(items)):
            v["qs"] = value(re.search(r"qs = ([^;]+);", QUERY)[1], v)
            yield wait(v, "163", seen, 1)
            yield arrive(v, at)

    def lse():
        v, seen = dict(base, ls=0, lph=0), {}
        (at,), = calls(LSE, "mbar_arrive")
        for _ in range(sum(items)):
            yield wait(v, "164", seen, 1)
            yield arrive(v, at)
            advance(LSE, "LS", v, "ls", "lph")

    def summing(warp):
        v, seen = dict(base, gp=warp >> 2), {}
        v["kt"] = value(re.search(r"kt = (gp [^,;]+)", SUM)[1], v)
        (empty,), (lempty,) = calls(SUM, "mbar_arrive")
        for v["g"] in range(sum(items)):
            v["ls"], v["sb"] = (value(re.search(r"%s = ([^;]+);" % n, SUM)[1], v) for n in ("ls", "sb"))
            yield wait(v, "165", seen)
            yield wait(v, "166", seen)
            yield arrive(v, empty)
            yield arrive(v, lempty)

    def expanding(warp):
        v, seen = dict(base), {}
        v["kGroups"], v["kT"] = (value(re.search(r"%s = ([^,;]+)[,;]" % n, EXPAND)[1], dict(v, kGroups=base["kExpandWarps"] // 4))
                                 for n in ("kGroups", "kT"))
        first = re.search(r"kt0 = kGroups == 1 \? 0 : \(warp - 4 - kSumWarps\) >> 2;", EXPAND)
        assert first
        v["kt0"] = 0 if v["kGroups"] == 1 else warp >> 2
        (full,), = calls(EXPAND, "mbar_arrive")
        for v["item"] in range(len(items)):
            v["set"] = value(re.search(r"set = ([^;]+);", EXPAND)[1], v)
            for v["kt"] in range(v["kT"]):
                yield wait(v, "167", seen, 1)
                yield arrive(v, full)

    roles = [issuer(k) for k in range(base["kKeyTiles"])] + [query(), lse()]
    roles += [summing(w) for w in range(base["kSumWarps"])] + [expanding(w) for w in range(base["kExpandWarps"])]
    at = [next(r, None) for r in roles]
    while any(a is not None for a in at):
        ready = []
        for i, a in enumerate(at):
            if a is None:
                continue
            if len(a) == 3:
                bar, parity, phase = a
                assert phase <= done[bar] <= phase + 1, "a wait more than one phase away"
                if (done[bar] & 1) == parity:
                    assert done[bar] == phase, "a wait that holds after its phase"
                    continue
                assert done[bar] == phase + 1, "a wait that passes before its phase"
            ready.append(i)
        assert ready, "all roles wait"
        # (a few of the roles at a time, so that some fall far behind)
        i = min(rnd.sample(ready, min(len(ready), 3))) if seed & 1 else rnd.choice(ready)
        if len(at[i]) == 1:
            bar, = at[i]
            got[bar] += 1
            if got[bar] == need[bar]:
                got[bar], done[bar] = 0, done[bar] + 1
        at[i] = next(roles[i], None)
    assert not any(got.values())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_no_wait_is_a_phase_off(d):
    for seed in range(24):
        rnd = random.Random(100 * d + seed)
        run(d, [rnd.randint(1, 5) for _ in range(rnd.randint(1, 9))], seed)


def test_every_wait_is_in_the_model():
    assert sorted(WAITS) == [str(s) for s in range(160, 169)]
    assert sum(len(calls(t, "mbar_wait")) for t in (ISSUE, QUERY, LSE, SUM, EXPAND)) == 9


@pytest.mark.parametrize("site,part,was,now", [
    ("162", 1, "(g - back)", "g"), ("160", 1, "C::kSets", "2"), ("166", 1, "C::kSRing", "QS"), ("163", 1, "^ 1", "^ 0"),
    ("167", 0, "kt0 + kt + set", "kt0 + kt"), ("165", 0, "ls", "0"), ("162", 0, "C::kKeyTiles - 1 - kt", "kt")])
def test_the_model_sees_a_changed_wait(monkeypatch, site, part, was, now):
    """A wait with another parity or another barrier is found (at one head_dim at least: not all differ at each)."""
    wait = list(WAITS[site])
    assert was in wait[part]
    wait[part] = wait[part].replace(was, now)
    monkeypatch.setitem(WAITS, site, wait)
    off = 0
    for d in (64, 128, 256):
        for seed in range(6):
            try:
                run(d, [3, 1, 4, 2, 5, 1], seed)
            except (AssertionError, KeyError):
                off += 1
    assert off > 0


def test_nothing_is_under_way_when_the_block_ends():
    """Where some role gives a wait up, another may have issued its last product or copy and left its loop
    without a failed wait: products are awaited before tensor memory is given back, and copies before the block's
    shared memory is, whether that role's own waits held or not."""
    for text, loop, drain in ((ISSUE, "while (ok && wk.next()) {", "umma_commit(b_drain + 8 * kt);"),
                              (QUERY, "while (ok && wk.next()) {", "mbar_wait_drain(b_qfull")):
        i, depth = text.index(loop) + len(loop), 1
        while depth:                                             # behind the loop
            depth += (text[i] == "{") - (text[i] == "}")
            i += 1
        between = text[i:text.index(drain)]
        assert "ok" not in between, between
