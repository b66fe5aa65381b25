"""How attend_cache8 rounds a weight to 8-bit terms, restated on FP16 bits on the
CPU: the bounds that its header gives, and that weights that are alike keep their
sum."""
import numpy as np
import pytest


def bits(x):
    return np.asarray(x, dtype=np.float16).view(np.uint16).astype(np.uint32)


def half(b):
    return (b & 0xffff).astype(np.uint16).view(np.float16).astype(np.float64)


def e4m3(x):
    a = np.abs(x)
    step = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.copysign(np.minimum(np.round(a / step) * step, 448.0), x)


def two_terms(p, turn):
    """An E4M3 and an E5M2 value: from 256 on E5M2 the value and E4M3 the rest, below the other way round; below 2^-6 the
    rest is rounded up where its lower byte and `turn` pass 255."""
    p = np.float16(p).astype(np.float64)
    large = np.where(p >= 256, half((bits(p) + 0x80) & 0xff00), 0.0)
    four = e4m3(p - large)
    five = half((bits(p - large - four) + np.where(p < 2.0 ** -6, turn, 0x80)) & 0xff00)
    return large + four + np.where(p >= 256, 0.0, five)


def three_terms(p, turn):
    """Three E5M2 values; below 2^-8 the third is rounded up or down by `turn`."""
    p = np.float16(p).astype(np.float64)
    x = half((bits(p) + 0x80) & 0xff00)
    y = half((bits(p - x) + 0x80) & 0xff00)
    return x + y + half((bits(p - x - y) + np.where(p < 2.0 ** -8, turn, 0x80)) & 0xff00)


def turns(kind, n):
    """`turn` of the first n keys: 2^8 times the fraction of key times the golden ratio, or, in the kernel of CTA pairs, the
    32 keys' numbers bit by bit backwards, crossed with that of the group of 32."""
    golden = lambda i: (i * 0x9E3779B1 & 0xffffffff) >> 24  # noqa: E731
    key = np.arange(n, dtype=np.uint64)
    if kind == "keys":
        return golden(key).astype(np.int64)
    i = key % 32
    back = sum((i >> b & 1) << (4 - b) for b in range(5))
    return ((back * 8 + 4) ^ golden(key // 32)).astype(np.int64)


WEIGHTS = np.arange(1, int(bits(3584.0)) + 1, dtype=np.uint16).view(np.float16).astype(np.float64)   # every FP16 weight


@pytest.mark.parametrize("terms,part,least", [(two_terms, 2.0 ** -7, 2.0 ** -13), (three_terms, 2.0 ** -9, 2.0 ** -16)])
def test_a_weight_is_within_its_bound(terms, part, least):
    for turn in (0, 1, 100, 0x80, 254, 255):
        off = np.abs(terms(WEIGHTS, turn) - WEIGHTS)
        assert (off <= part * WEIGHTS + least).all()
    assert (terms(np.zeros(3), np.array([0, 128, 255])) == 0).all()


@pytest.mark.parametrize("kind", ["keys", "pairs"])
def test_the_turns_are_spread(kind):
    """Of 2^12 keys from any on the share with turn >= t is right to 2^-7 for each t, of 2^12 that lie 2 to 64 apart to
    2^-5."""
    r = turns(kind, 1 << 18)
    for first, n, stride in [(0, 4096, 1), (777, 4096, 1), (100000, 5000, 1)] + [(5, 4096, s) for s in (2, 3, 8, 16, 17, 32, 64)]:
        some = r[first:first + n * stride:stride]
        at_least = np.array([(some >= t).mean() for t in range(257)])
        assert np.abs(at_least - (1 - np.arange(257) / 256)).max() <= 2.0 ** (-7 if stride == 1 else -5), (first, stride)


@pytest.mark.parametrize("kind", ["keys", "pairs"])
@pytest.mark.parametrize("terms", [two_terms, three_terms])
def test_weights_alike_keep_their_sum(terms, kind):
    n = 4096
    r = turns(kind, n)
    for p in np.exp2(np.arange(-16, 11.7, 0.137)):
        p = float(np.float16(p))
        off = abs(terms(np.full(n, p), r).mean() / p - 1)
        assert off <= 2.0 ** -7, p
