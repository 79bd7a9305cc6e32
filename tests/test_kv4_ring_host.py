"""The value ring of the kernel for trees with many rows, as a model: warps that unpack, the warp that issues
products, barriers that tell phases by their parity alone.

A wait for a phase's parity cannot tell it from the phase two before or behind.  The model runs the waits of
fa_kv4_wide.cuh in random orders and speeds and sees whether one passes too early (a place overwritten that a
product has not taken) or never (a warp that asks for a phase two phases old).  Items of a team are three to five
apart, so the kernel waits once more before the last item of a unit; without that wait most schedules go wrong."""
import os
import random
import re

import pytest

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_37_gb300", "csrc", "fa_kv4_wide.cuh")


def place(values, j, n):
    """wide_item of the kernel."""
    if values:
        return 2 * n - 1 if j == n - 1 else 2 * j + 2
    return 0 if j == 0 else 2 * j - 1


def constants():
    with open(HEADER) as f:
        text = f.read()
    items = int(re.search(r"kItems = (\d+);", text).group(1))
    teams = re.search(r"kTeam = D == 256 \? (\d+) : (\d+), kTeams = 4 / kTeam;", text)
    return text, items, [int(x) for x in teams.groups()]


def test_the_model_is_of_this_kernel():
    """The lines that the model stands for, as the kernel has them."""
    text, items, teams = constants()
    flat = re.sub(r"\s+", " ", text)
    for line in ("if (values) return j == n - 1 ? 2 * n - 1 : 2 * j + 2; return j == 0 ? 0 : 2 * j - 1;",
                 "for (int j = W::kTeams == 2 ? (tile0 ^ team) & 1 : 0; j < n; j += W::kTeams) {",
                 "if (item >= W::kItems && !(ok = warp_nap(bar(W::kEmpty + s), (item / W::kItems - 1) & 1, err, kErrTimeoutMma))) break;",
                 "if (W::kTeams == 2 && j + 2 >= n && item >= 3 && "
                 "!(ok = warp_nap(bar(W::kEmpty + (item + 1) % W::kItems), ((item - 3) / W::kItems) & 1, err, kErrTimeoutMma))) break;",
                 "return warp_nap(bar(W::kFull + i % W::kItems), (i / W::kItems) & 1, err, kErrTimeoutRing);"):
        assert line in flat, line
    assert items == 4 and teams == [4, 2]


def run(units, seed, team_warps, extra_wait, items=4):
    """Goes through units of so many tiles: "done", "stuck", or "early" where a wait passed that should not have."""
    rng = random.Random(seed)
    teams = 4 // team_warps
    empty, full, arrived = [0] * items, [0] * items, [0] * items  # phases completed; arrivals at a place's next

    def unpack(values, team):
        item0 = tile0 = 0
        for n in units:
            for j in range((tile0 ^ team) & 1 if teams == 2 else 0, n, teams):
                item = item0 + place(values, j, n)
                s = item % items
                if item >= items:
                    yield empty, s, (item // items - 1) & 1
                    if empty[s] < item // items:
                        raise OverflowError
                yield None  # the work
                if extra_wait and teams == 2 and j + 2 >= n and item >= 3:
                    yield empty, (item + 1) % items, ((item - 3) // items) & 1
                arrived[s] += 1
                if arrived[s] == team_warps:
                    arrived[s] = 0
                    full[s] += 1
                yield None
            item0 += 2 * n
            tile0 += n

    def issue():
        for item in range(2 * sum(units)):
            s = item % items
            yield full, s, (item // items) & 1
            if full[s] != item // items + 1:
                raise OverflowError
            yield None  # the product
            empty[s] += 1

    roles = [unpack(v, t) for v in (0, 1) for t in range(teams) for _ in range(team_warps)] + [issue()]
    speed = [rng.choice((1, 1, 4, 20)) for _ in roles]
    now = [next(r, "end") for r in roles]  # what each waits for
    idle = 0
    try:
        while any(now[k] != "end" for k in range(len(roles))):
            live = [k for k in range(len(roles)) if now[k] != "end"]
            k = rng.choices(live, [speed[x] for x in live])[0]
            if rng.random() < 0.02:
                speed[rng.randrange(len(roles))] = rng.choice((0.2, 1, 4, 20))
            w = now[k]
            if w is None or (w[0][w[1]] & 1) != w[2]:  # the phase of that parity is not the one under way
                now[k] = next(roles[k], "end")
                idle = 0
            else:
                idle += 1
                if idle > 400 and all(now[x] is not None and (now[x][0][now[x][1]] & 1) == now[x][2] for x in live):
                    return "stuck"
    except OverflowError:
        return "early"
    return "done"


def some_units(seed):
    rng = random.Random(seed)
    return [rng.choice((1, 1, 2, 2, 3, 4, 5, 9, 20)) for _ in range(rng.randint(2, 14))]


@pytest.mark.parametrize("team_warps", [2, 4])
def test_every_schedule_ends(team_warps):
    """Random units and speeds, in teams of two warps (d = 64 and 128) and of four (d = 256)."""
    for seed in range(100):
        assert run(some_units(seed), seed, team_warps, True) == "done", seed


@pytest.mark.parametrize("units", [[1] * 40, [2] * 20, [3] * 14, [1, 2] * 12, [1, 1, 2] * 9, [4, 1] * 8, [2, 3, 1, 1] * 6, [64], [1], [2]])
def test_units_of_one_kind(units):
    for seed in range(12):
        assert run(units, seed, 2, True) == "done", seed


def test_the_wait_at_a_units_end_is_needed():
    """The same schedules without it: a team that comes late takes a phase for the one two phases on."""
    ends = [run(some_units(seed), seed, 2, False) for seed in range(100)]
    assert ends.count("done") < 20
