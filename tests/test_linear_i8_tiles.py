"""The row tiles that moe_linear_i8's grid holds, from the library's own count: as many
as any sizes of the groups can make, and no fewer for any draw."""

import random

from test_linear_i8_plan import TOKENS, log_uniform, plans  # noqa: F401 (a fixture)

COUNTED = (64, 256)                     # tokens of a tile; of the library's two counts


def worst(M, E, t):
    """Sizes of E groups, M rows in all, that make the most tiles of t rows: every group that can
    begins a tile with one row, whole tiles go to the first and the rest fills the last one's."""
    used = min(E, M)
    counts = [1] * used + [0] * (E - used)
    counts[0] += (M - used) // t * t
    counts[used - 1] += (M - used) % t
    return counts


def needed(counts, t):
    return sum(-(-c // t) for c in counts)


def test_any_sizes_of_the_groups_fit_the_grid(plans):  # noqa: F811
    rng = random.Random(5)
    cases, sizes = [], []
    for _ in range(3000):
        E, M = log_uniform(rng, 1, 1024), log_uniform(rng, 1, 6000)
        cuts = sorted(rng.randint(0, M) for _ in range(E - 1))
        cases.append((M, 64, 64, False, 0, 0, E))
        sizes.append([b - a for a, b in zip([0] + cuts, cuts + [M])])
    for (M, _, _, _, _, _, E), counts, (_, tiles) in zip(cases, sizes, plans(cases, True)):
        for t, n in zip(COUNTED, tiles):
            assert needed(counts, t) <= n, (M, E, t)
            # a bound one lower would lose rows of these
            w = worst(M, E, t)
            assert sum(w) == M and len(w) == E and needed(w, t) == n, (M, E, t)


def test_rows_without_groups(plans):  # noqa: F811
    rng = random.Random(6)
    cases = [(log_uniform(rng, 1, 1 << 28), 1 + i % 64, 64, False, 0, 0, 0) for i in range(2000)]
    for (M, *_), (p, tiles) in zip(cases, plans(cases, True)):
        assert list(tiles) == [-(-M // t) for t in COUNTED], M
        assert TOKENS.get(p.tile, 64) >= 64
