"""The static tile order of a grouped launch (dense_gemm.cu, struct Order), restated: every tile is dealt exactly
once, in ascending order within a cluster, whatever the split into long and short tiles; and the clusters without
a further long tile take at least as many short ones."""
import random


def order(c, P, n, big, rounds):
    """Tiles of cluster c of P; `big` long tiles first, then the others, `rounds` of them among the clusters that
    hold one long tile less."""
    mine = (big - c + P - 1) // P if c < big else 0
    r = big % P
    rest, more = P - r, c >= r
    k, out = 0, []
    while True:
        if k < mine:
            t = c + k * P
        else:
            j = k - mine
            if more and j < rounds:
                t = big + j * rest + c - r
            else:
                t = big + rounds * rest + (j - (rounds if more else 0)) * P + c
        if t >= n:
            return out
        out.append(t)
        k += 1


def test_every_tile_once_and_in_order():
    rng = random.Random(3)
    for _ in range(2000):
        big, small = rng.choice([0, rng.randrange(200)]), rng.randrange(800)
        if big + small == 0:
            continue
        P = min(rng.randint(1, 74), big + small)
        r = big % P
        rounds = rng.randint(0, small // (P - r)) if r else 0
        dealt = [order(c, P, big + small, big, rounds) for c in range(P)]
        assert sorted(t for d in dealt for t in d) == list(range(big + small))
        assert all(d == sorted(d) for d in dealt)
        if 0 < r < P:
            short = [sum(t >= big for t in d) for d in dealt]
            assert min(short[r:]) >= rounds and max(short[:r]) <= min(short[r:]) - rounds + 1


def test_a_wrong_share_is_caught():
    """Planted: dealing the extra rounds among all clusters deals some tiles twice."""
    P, big, small, rounds = 10, 4, 60, 3
    wrong = []
    for c in range(P):
        d = order(c, P, big + small, big, rounds)
        wrong += [t if t < big or t >= big + rounds * (P - big) else big + (t - big) % (P - big) for t in d]
    assert sorted(wrong) != list(range(big + small))
