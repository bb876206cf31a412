"""The ring that e4m3 scales go through in the attention, on a model: four loading warps whose copies arrive by themselves,
teams of warps that take the tiles in turn, and waits that give up."""
import random

from tests.test_kv_waits import Bar


def scales(seed, *, teams=None, buffers=None, places=None, lands=True):
    """As attend.cuh has it: a loading warp's arrival counts once its copies have landed, another for which positions are
    there; after a wait that gave up it copies no more but arrives all the same. A warp of the softmax gives a place back
    whether its wait gave up or not, one without rows when the tile's scores are there. Scores go through `buffers` places
    of their own. lands: the loading warps end after their last copies. Returns what went wrong, or None."""
    r = random.Random(seed)
    TM = teams or r.choice([1, 2, 4])
    SB = buffers or (2 if TM == 1 else TM)
    ring = places or r.choice([4, 8, 16])
    if ring <= SB:
        ring = 16
    tiles, stall = r.randint(1, 70), r.choice([0, 0, 0.001, 0.01, 0.2])
    live, idle = r.choice([1, 2]), r.choice([0, 1])  # warps of a team with and without rows
    full, empty = [Bar(8) for _ in range(ring)], [Bar(live + idle) for _ in range(ring)]
    s_full, s_empty = [Bar(1) for _ in range(SB)], [Bar(live + idle) for _ in range(SB)]
    held = [[None] * 4 for _ in range(ring)]  # the tile whose scales a place holds, for each loading warp
    flying, aborted, wrong = [], [False], []

    def wait(bar, parity):
        while not bar.done(parity):
            if aborted[0]:
                return False
            if r.random() < stall:
                aborted[0] = True
            yield
        return True

    def loader(w):
        dead = False
        for t in range(tiles):
            s = t % ring
            if t >= ring and not (yield from wait(empty[s], (t // ring - 1) & 1)):
                dead = True
            if dead:
                full[s].arrive()
            else:
                flying.append((w, s, t))
            yield
            full[s].arrive()
            yield
        while lands and any(f[0] == w for f in flying):
            yield

    def scores():
        for t in range(tiles):
            if t >= SB and not (yield from wait(s_empty[t % SB], (t // SB - 1) & 1)):
                return
            for _ in range(r.randint(0, 3)):
                yield
            s_full[t % SB].arrive()

    def softmax(team, rows):
        for t in range(team, tiles, TM):
            s = t % ring
            if rows:
                got = yield from wait(full[s], (t // ring) & 1)
                for _ in range(r.randint(0, 6)):
                    if not aborted[0] and got and held[s] != [t] * 4:
                        wrong.append("scales of another tile")
                    yield
            yield from wait(s_full[t % SB], (t // SB) & 1)
            s_empty[t % SB].arrive()
            yield
            empty[s].arrive()
            yield

    roles = [loader(w) for w in range(4)] + [scores()]
    roles += [softmax(m, i < live) for m in range(TM) for i in range(live + idle)]
    for _ in range(200000):
        if flying and r.random() < 0.2:
            w, s, t = flying.pop(r.randrange(len(flying)))
            held[s][w] = t
            full[s].arrive()
        g = r.choice(roles)
        try:
            next(g)
        except StopIteration:
            roles.remove(g)
        if not roles:
            break
    else:
        wrong.append("a role does not end")
    if flying:
        wrong.append("a copy outlives the CTA")
    return wrong[0] if wrong else None


def test_scales_are_the_tiles_and_no_copy_outlives_the_cta():
    assert {scales(seed) for seed in range(1500)} == {None}


def test_the_model_sees_what_the_rules_keep_out():
    """A ring whose places go from team to team, loading warps that leave their copies behind."""
    assert "a copy outlives the CTA" in {scales(seed, lands=False) for seed in range(600)}
    assert {scales(seed, teams=2, buffers=2, places=3) for seed in range(600)} != {None}
