"""The barriers of the decode over several tokens (csrc/kda_tokens.cu), run as a model on the CPU: teams that
prepare blocks, the warp that moves the states, and the working warps, over lists of heads with few blocks and
windows of pairs that end anywhere among them. Every role has to end, and nothing may be overwritten before it
is read.

What the teams do before their first step is taken from the source, statement by statement; the rest of the
roles is written out here as it stands there.
"""
import os
import random
import re

import pytest

from kimi_delta_attention_17_gb300 import build

SOURCE = os.path.join(os.path.dirname(os.path.abspath(build.__file__)), "csrc", "kda_tokens.cu")
BLOCK, TEAM = 8, 96
FULL, EMPTY, TEAM_BAR, WINDOW, BEGIN = 1, 9, 11, 13, 14


def first_statements(source):
    """What a team does from its first head on, up to its steps: [(statement, "all" or "team 1")]."""
    body = source[source.index("TokenTask task = {0, -1"):source.index("for (int step = team;; step += kTeams)")]
    body = re.sub(r"//[^\n]*", "", body)
    found, only = [], "all"
    for line in (x.strip() for x in body.split("\n")[1:]):
        if line == "if (team == 1) {":
            only = "team 1"
        elif line == "}":
            only = "all"
        elif line:
            found.append((line.rstrip(";"), only))
    return found


class Barriers:
    """Named barriers: each opens when as many threads have come as its first one expected."""

    def __init__(self):
        self.phase, self.came, self.count = {}, {}, {}

    def arrive(self, at, threads, count):
        if self.came.get(at, 0) == 0:
            self.count[at] = count
        assert self.count[at] == count, "barrier %d: two counts at once" % at
        self.came[at] = self.came.get(at, 0) + threads
        assert self.came[at] <= count, "barrier %d: too many" % at
        phase = self.phase.setdefault(at, 0)
        if self.came[at] == count:
            self.came[at], self.phase[at] = 0, phase + 1
        return phase

    def open(self, at, phase):
        return self.phase[at] > phase


class Cta:
    def __init__(self, counts, teams, pairs, window, first):
        self.counts, self.teams, self.pairs, self.window, self.first = counts, teams, pairs, window, first
        self.bar, self.prep = Barriers(), teams * TEAM
        self.work, self.full, self.empty = 64 * pairs, 64 + TEAM, 64 * pairs + TEAM + 32
        self.block, self.ring, self.held = [None, None], [None] * 4, [None] * window
        self.values = [None] * (teams + 2)
        self.arrived, self.buffer, self.stored = [0, 0], [None, None], []
        self.reading = [0, 0]  # working warps that are in block 0 or 1
        self.done = []

    def sync(self, at, threads, count):
        phase = self.bar.arrive(at, threads, count)
        while not self.bar.open(at, phase):
            yield

    def team(self, team):
        st = dict(task=dict(place=-1, before=-1, older=-1, count=0, t0=0, head=-1), next=None, second=None)
        cursor = [0]

        def next_head(task):
            task.update(older=task["before"], before=task["place"], place=-1, head=task["head"] + 1)
            while cursor[0] < len(self.counts):
                at = cursor[0] % self.window
                if at == 0:
                    yield from self.sync(WINDOW, TEAM, self.prep)
                    for i in range(team, self.window, self.teams):  # each team its part
                        self.held[i] = (cursor[0], self.counts[cursor[0] + i] if cursor[0] + i < len(self.counts) else BLOCK)
                    yield from self.sync(WINDOW, TEAM, self.prep)
                assert self.held[at][0] == cursor[0] - at  # the window that this team is in
                cursor[0] += 1
                if self.held[at][1] > 0:
                    task.update(place=cursor[0] - 1, count=self.held[at][1], t0=0)
                    return

        def advance(task):
            to = dict(task)
            if to["place"] >= 0:
                to["t0"] += BLOCK
                if to["t0"] >= to["count"]:
                    yield from next_head(to)
            return to

        def fetch(task, step):
            if task["place"] >= 0:
                self.values[step % (self.teams + 2)] = (task["place"], task["t0"])

        def pass_full(step):
            assert self.reading[step & 1] == 0, "block %d passed on while it is read" % (step & 1)
            for p in range(self.pairs):
                self.bar.arrive(FULL + 2 * p + (step & 1), TEAM, self.full)

        def at_empty(step):
            yield from self.sync(EMPTY + (step & 1), TEAM, self.empty)

        first_end = True
        for statement, only in self.first:
            if only == "team 1" and team != 1:
                continue
            if statement == "next_head(task)":
                yield from next_head(st["task"])
            elif statement in ("next = advance(task)", "second = advance(next)"):
                to, of = re.match(r"(\w+) = advance\((\w+)\)", statement).groups()
                st[to] = yield from advance(st[of])
            elif statement == "task = next":
                st["task"] = st["next"]
            elif statement == "if (tid == 0 && team == 0) sm.ring[0] = task":
                self.ring[0] = dict(st["task"]) if team == 0 else self.ring[0]
            elif statement == "if (tid == 0 && team == 0) sm.ring[1] = next":
                self.ring[1] = dict(st["next"]) if team == 0 else self.ring[1]
            elif statement == "tc::bar_sync(kBarBegin, kPrep + 32)":
                yield from self.sync(BEGIN, TEAM, self.prep + 32)
            elif statement == "first_end = task.place >= 0":
                first_end = st["task"]["place"] >= 0
            elif statement == "fetch(task, team)":
                fetch(st["task"], team)
            else:
                assert statement == "bool first_end = true", "the model does not know: " + statement
            yield
        step = team
        while True:
            task = st["task"]
            if task["place"] < 0:
                if step >= 2:
                    yield from at_empty(step)
                if first_end:
                    self.block[step & 1] = dict(task, step=step)
                    pass_full(step)
                    if self.teams == 1 and step >= 1:
                        yield from at_empty(step - 1)
                    yield from at_empty(step)
                return
            yield
            if step >= 2:
                yield from at_empty(step)
            assert self.reading[step & 1] == 0, "block %d filled while it is read" % (step & 1)
            self.block[step & 1] = dict(task, step=step)
            self.ring[(step + 2) & 3] = dict(st["second"])
            yield
            pass_full(step)
            yield
            first_end = self.teams == 1 or st["next"]["place"] >= 0
            if self.teams == 2:
                st["task"] = st["second"]
                st["next"] = yield from advance(st["task"])
            else:
                st["task"], st["next"] = st["next"], st["second"]
            st["second"] = yield from advance(st["next"])
            fetch(st["task"], step + self.teams)
            step += self.teams

    def mover(self):
        def store(head, place):
            if place >= 0:
                assert self.buffer[head & 1] == ("out", place), "a state goes before it is done with"
                self.stored.append(place)

        def at_empty(step):
            yield from self.sync(EMPTY + (step & 1), 32, self.empty)

        yield from self.sync(BEGIN, 32, self.prep + 32)
        step = 0
        while True:
            if step >= 2:
                yield from at_empty(step)
            task = dict(self.ring[step & 3])
            if task["place"] < 0:
                if step >= 1:
                    yield from at_empty(step - 1)
                yield from at_empty(step)
                store(task["head"] - 2, task["older"])
                store(task["head"] - 1, task["before"])
                return
            if task["t0"] == 0:
                store(task["head"] - 2, task["older"])
                yield  # the copy takes its time
                self.buffer[task["head"] & 1] = ["in", task["place"], 0]
                self.arrived[task["head"] & 1] += 1
            yield
            step += 1

    def worker(self, warp):
        step = 0
        while True:
            bar = FULL + (warp & ~1) + (step & 1)
            yield from self.sync(bar, 32, self.full)
            self.reading[step & 1] += 1
            task = self.block[step & 1]
            assert task["step"] == step
            if task["place"] < 0:
                self.reading[step & 1] -= 1
                self.bar.arrive(EMPTY + (step & 1), 32, self.empty)
                return
            buf, last = task["head"] & 1, task["t0"] + BLOCK >= task["count"]
            if task["t0"] == 0:
                while self.arrived[buf] <= task["head"] >> 1:
                    yield
                assert self.arrived[buf] == (task["head"] >> 1) + 1 and self.buffer[buf][:2] == ["in", task["place"]]
            assert self.values[step % (self.teams + 2)] == (task["place"], task["t0"])
            yield from self.sync(bar, 32, 64)
            assert self.values[step % (self.teams + 2)] == (task["place"], task["t0"])
            yield from self.sync(bar, 32, 64)
            assert self.block[step & 1] is task
            if warp == 0:
                self.done.append((task["place"], task["t0"]))
            if last:
                self.buffer[buf][2] += 1
                if self.buffer[buf][2] == 2 * self.pairs:
                    self.buffer[buf] = ("out", task["place"])
            self.reading[step & 1] -= 1
            self.bar.arrive(EMPTY + (step & 1), 32, self.empty)
            step += 1

    def run(self, rng):
        roles = {"mover": self.mover(), **{"team %d" % t: self.team(t) for t in range(self.teams)},
                 **{"warp %d" % w: self.worker(w) for w in range(2 * self.pairs)}}
        idle, slow = 0, rng.choice([None, *roles])
        while roles:
            before = (dict(self.bar.phase), dict(self.bar.came), list(self.arrived), len(roles))
            names = list(roles)
            rng.shuffle(names)
            for name in names:
                if name == slow and rng.random() < 0.9:
                    continue
                for _ in range(rng.randint(1, 4)):  # roles run at their own speeds
                    if next(roles[name], "end") == "end":
                        del roles[name]
                        break
            same = before == (self.bar.phase, self.bar.came, self.arrived, len(roles))
            idle = idle + 1 if same else 0  # no role does more than a few things between two barriers
            assert idle < 500, "no role comes further: %s wait for ever" % ", ".join(roles)
        blocks = [(i, t) for i, c in enumerate(self.counts) for t in range(0, max(c, 0), BLOCK)]
        assert self.done == blocks and sorted(self.stored) == [i for i, c in enumerate(self.counts) if c > 0]
        assert not any(self.bar.came.values())


@pytest.fixture(scope="module")
def first():
    with open(SOURCE) as f:
        return first_statements(f.read())


def tokens(blocks, rng):
    return BLOCK * (blocks - 1) + rng.randint(1, BLOCK) if blocks else 0


@pytest.mark.parametrize("teams", [1, 2])
@pytest.mark.parametrize("ahead", range(7))
@pytest.mark.parametrize("behind", [0, 1, 2, 5])
def test_few_blocks_before_a_windows_end(first, teams, ahead, behind):
    """So many blocks among the first pairs, in one head, in several, anywhere before the windows' end, none for two
    windows more, and some (or none) behind."""
    rng = random.Random(100 * ahead + 10 * behind + teams)
    for heads in range(1 if ahead else 0, ahead + 1):
        for _ in range(3):
            cuts = sorted(rng.sample(range(1, ahead), heads - 1)) if ahead else []
            sizes = [b - a for a, b in zip([0] + cuts, cuts + [ahead])] if ahead else []
            window = 8
            counts = [0] * (window * 4)
            for place, size in zip(sorted(rng.sample(range(window), heads)), sizes):
                counts[place] = tokens(size, rng)
            for place in rng.sample(range(3 * window, 4 * window), behind):
                counts[place] = tokens(rng.randint(1, 3), rng)
            Cta(counts, teams, 2, window, first).run(rng)


@pytest.mark.parametrize("teams", [1, 2])
@pytest.mark.parametrize("pairs", [1, 2, 4])
def test_any_counts(first, teams, pairs):
    """Lists of any length, dense and sparse, ending before, at and behind a window's end; none at all among them."""
    rng = random.Random(pairs)
    for n in range(150):
        window = rng.choice([1, 2, 3, 4, 8])
        some = rng.choice([0.02, 0.1, 0.3, 0.7, 1.0])
        counts = [tokens(rng.randint(1, 4), rng) if rng.random() < some else 0 for _ in range(rng.randint(0, 40))]
        Cta(counts, teams, pairs, window, first).run(rng)
