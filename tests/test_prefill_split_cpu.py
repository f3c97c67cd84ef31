"""The cut of the 4-bit prefill's work (prefill_split in prefill.cu), restated:
ranges in strictly rising order that hold every tile, and no tile in more than
the 32 pieces that the un-rotation's merge has lanes for.  A range holds total /
n of the work and n <= 30 floor(total / heaviest tile), so a tile holds the work
of at most 30 ranges: with one that begins before it and one that ends behind it,
at most 32 pieces.
"""
import random

ROWS, KEYS, PIECES = 256, 128, 32


def split(tokens, length, hq, hkv, sms):
    g, first = hq // hkv, length - tokens
    tiles, old = (tokens * g + ROWS - 1) // ROWS, first * (hq // hkv)

    def before(x):
        return x * (old + ROWS // 2 * (x + 1))

    def weight(x):
        return old + ROWS * (x + 1)

    def chunks_of(x):
        return (first + (min(ROWS * (x + 1), tokens * g) - 1) // g) // KEYS + 1

    head = before(tiles)
    total = head * hkv
    n = min(sms, 256, (PIECES - 2) * (total // weight(tiles - 1)), max(tiles * hkv, total // (2 * KEYS * g)))
    start = [(0, 0)]
    for j in range(1, n):
        u = total // n * j + total % n * j // n
        hk, v = u // head, u % head
        x = max(i for i in range(tiles) if before(i) <= v) if tiles < 64 else _last(before, tiles, v)
        chunks = chunks_of(x)
        snap = 1 if chunks >= 16 else 0
        c = ((v - before(x)) * chunks + weight(x) // 2) // weight(x)
        s = (hk * tiles + x, 0) if c <= snap else (hk * tiles + x + 1, 0) if c >= chunks - snap else (hk * tiles + x, c)
        if s > start[-1]:
            start.append(s)
    if start[-1][0] == tiles * hkv:
        start.pop()
    return tiles, start + [(tiles * hkv, 0)], chunks_of


def _last(before, tiles, v):
    lo, hi = 0, tiles - 1
    while lo < hi:
        mid = (lo + hi + 1) >> 1
        lo, hi = (mid, hi) if before(mid) <= v else (lo, mid - 1)
    return lo


def pieces(tokens, length, hq, hkv, sms=148):
    """Pieces of the tile that has the most; checks that the ranges hold every tile's chunks once."""
    tiles, start, chunks_of = split(tokens, length, hq, hkv, sms)
    seen, count = {}, {}
    for a, b in zip(start, start[1:]):
        assert a < b
        for t in range(a[0], b[0] + (b[1] > 0)):
            lo = a[1] if t == a[0] else 0
            hi = b[1] if t == b[0] else chunks_of(t % tiles)
            assert lo == seen.get(t, 0) and lo < hi
            seen[t], count[t] = hi, count.get(t, 0) + 1
    assert all(seen[t] == chunks_of(t % tiles) for t in range(tiles * hkv)) and len(seen) == tiles * hkv
    return max(count.values())


MANY = [(1, 7360, 5, 5, 30), (100, 28291, 10, 5, 31), (1, 60000, 1, 1, 30)]  # tokens, length, hq, hkv, pieces on 148 SMs


def test_shapes_with_the_most_pieces():
    for tokens, length, hq, hkv, most in MANY:
        assert pieces(tokens, length, hq, hkv) == most


def test_no_tile_has_more_pieces_than_the_merge_has_lanes():
    r = random.Random(3)
    for _ in range(4000):
        hkv, g = r.choice([1, 2, 3, 4, 5, 6, 7, 8, 16, 64]), r.choice([1, 2, 3, 4, 5, 8, 16])
        length = int(2 ** r.uniform(0, 20)) + 1
        tokens = min(length, int(2 ** r.uniform(0, 12)))
        assert pieces(tokens, length, hkv * g, hkv, r.choice([148, 148, 132, 160, 300])) <= PIECES
