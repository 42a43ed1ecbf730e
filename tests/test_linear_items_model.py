"""The projection's tile numbering as a host model: pairs of CTAs walk whole tiles, half tiles and the
narrow edge tiles (item_of in csrc/gdn_linear.cu). Every tile belongs to exactly one pair, and no
pair has more than about a tile more to do than the mean."""
import random

PAIRS = 76          # pairs of SMs


def plan(M, N, TN, unit):
    mt, nt = -(-M // 256), N // TN
    edge = -(-(N % TN) // unit) * unit
    last = mt * nt % PAIRS
    halves = 2 * last if TN == 256 and 0 < last <= PAIRS // 2 else 0
    whole = mt * nt - halves // 2
    items = whole + halves + (mt if edge else 0)
    pairs = min(items, PAIRS)
    light = (whole + halves) % pairs
    room = (pairs - light) * (320 // (edge + 64))
    return dict(mt=mt, nt=nt, edge=edge, halves=halves, whole=whole, items=items, pairs=pairs, light=light,
                light_edges=0 if edge == 0 else min(mt, room))


def item_of(p, pair, n):
    """The n-th item of a pair: ("main", index), ("edge", row tile) or None behind the last."""
    main = p["whole"] + p["halves"]
    i = pair + n * p["pairs"]
    if i < main:
        return "main", i
    k = n - ((main - pair + p["pairs"] - 1) // p["pairs"] if pair < main else 0)
    lights = p["pairs"] - p["light"]
    e, first = (0 if p["edge"] else p["mt"]), 0
    if pair >= p["light"]:
        first = (p["light_edges"] - (pair - p["light"]) + lights - 1) // lights
        assert first >= 0
        if k < first:
            e = pair - p["light"] + k * lights
    if k >= first:
        e += p["light_edges"] + pair + (k - first) * p["pairs"]
    return ("edge", e) if e < p["mt"] else None


def test_every_tile_once():
    rng = random.Random(0)
    shapes = [(1, 1), (4100, 2056), (4100, 2040), (8192, 2048), (256, 256), (257, 255)]
    shapes += [(rng.randint(1, 30000), rng.randint(1, 9000)) for _ in range(2000)]
    for M, N in shapes:
        for TN in (128, 256):
            for unit in (32, 128):
                p = plan(M, N, TN, unit)
                seen, loads = set(), []
                for pair in range(p["pairs"]):
                    n = load = 0
                    while (it := item_of(p, pair, n)) is not None:
                        assert it not in seen
                        seen.add(it)
                        load += (p["edge"] + 64) / 320 if it[0] == "edge" else 1 if it[1] < p["whole"] else 0.6
                        n += 1
                    loads.append(load)
                assert len(seen) == p["items"]
                assert max(loads) <= sum(loads) / len(loads) + 1.25, (M, N, TN, unit)
