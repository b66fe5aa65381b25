"""Attention over the 8-bit cache where its weights and masks are hardest, on each
of its kernels: tiles of 16, 32 and 64 heads, CTA pairs, and pairs with a tile
that is not full.

Tolerances as in test_cache8_gpu.  Sums of many weights that are alike have one
of their own, below.
"""
import math

import pytest
import torch

import cache8_reference as ref
import test_cache8_gpu as base

pytestmark = pytest.mark.gpu

from mla_attention_prolog_gb300 import binding  # noqa: E402

DEV = base.DEV
HEADS = [16, 20, 64, 128, 130]
# lengths whose last step ends in the first and in the second half of 128 keys (a pair's CTAs bring one each), at 32 keys'
# ends and beside them, and in the first step
TAILS = [1, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 190, 193, 254, 300, 383]


def code(x):
    return ref.nearest(torch.tensor([x], dtype=torch.float64)).item()


@pytest.mark.parametrize("H", HEADS)
def test_reads_nothing_behind_the_ends(H):
    """NaN codes behind each sequence's end, in pages of nobody and in the bytes that fill up a page; results as without."""
    lens = TAILS + [0]
    cache, table, q = base.attend_case(81, lens, H, 512, 64, 48, 3)
    clean = base.run_attend(cache, table, lens, q, 512, 0.1)
    base.check_attend(cache, table, lens, q, 512, 0.1, *clean)
    keep = torch.zeros(cache.codes.shape[:2], dtype=torch.bool)
    for s, n in enumerate(lens):
        t = torch.arange(n)
        keep[table[s].long()[t // 48], t % 48] = True
    cache.codes[~keep] = 0x7f
    cache.exps[~keep.unflatten(1, (16, 3)).any(2)] = 255
    cache.bytes[:, 48 * 576 + 16:] = 0xff
    dirty = base.run_attend(cache, table, lens, q, 512, 0.1)
    for a, b in zip(clean, dirty):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("H", HEADS)
def test_nan_code_of_a_key_and_infinite_query(H):
    lens = [200, 193, 330]
    cache, table, q = base.attend_case(82, lens, H, 128, 64, 64, 8)
    cache.codes[int(table[0, 1]), 3, 5] = 0x7f
    bad = {0, 2, H // 2 + 1, H - 1}
    for i, h in enumerate(sorted(bad)):
        q[1, h, 7 + i] = (math.inf, math.nan, -math.inf, math.nan)[i]
    out, lse = base.run_attend(cache, table, lens, q, 128, 0.1)
    assert out[0].isnan().all() and lse[0].isnan().all()
    for h in range(H):
        assert bool(out[1, h].isnan().all()) == (h in bad) and bool(out[1, h].isnan().any()) == (h in bad), h
        assert bool(lse[1, h].isnan()) == (h in bad), h
    base.check_attend(cache, table[2:], lens[2:], q[2:], 128, 0.1, out[2:], lse[2:])


@pytest.mark.parametrize("H", HEADS)
def test_pages_and_lengths_outside_their_ranges(H):
    cache, table, q = base.attend_case(83, [256] * 4, H, 128, 64, 64, 16)
    status = base.i32([0])
    out, lse = base.run_attend(cache, table, [-5, 1 << 30, 256, 0], q, 128, 0.1, status=status)
    assert status.item() == binding.STATUS_SEQ_RANGE
    base.check_attend(cache, table, [0, 256, 256, 0], q, 128, 0.1, out, lse)
    # pages outside read as rows of zeros: in either half of a step, in a last step
    bad, n = table.clone(), cache.bytes.shape[0]
    lens = [256, 250, 170, 100]
    bad[0, 1], bad[1, 2], bad[1, 3], bad[2, 2], bad[3, 1] = -1, n, 2 ** 31 - 1, -7, n
    status = base.i32([0])
    out, lse = base.run_attend(cache, bad, lens, q, 128, 0.1, status=status)
    assert status.item() == binding.STATUS_PAGE_RANGE
    zero = ref.Pages(torch.cat([cache.bytes, torch.zeros((1, cache.bytes.shape[1]), dtype=torch.uint8)]), cache.C, 64, 16)
    zero.exps[n] = 127
    bad[0, 1] = bad[1, 2] = bad[1, 3] = bad[2, 2] = bad[3, 1] = n
    base.check_attend(zero, bad, lens, q, 128, 0.1, out, lse)


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("q_std,scale,lo,hi", [(1.0, 2.0, 115, 122), (30.0, 1.0, 119, 122), (1e-6, 1e4, 119, 122),
                                               (1.0, 0.07, 60, 200), (1e20, 1e-21, 119, 122), (1.0, 1e-30, 119, 122)])
def test_sharp_flat_and_uneven(H, q_std, scale, lo, hi):
    """Weights of one key, weights all alike, scales from 2^-60 to 2^60 side by side; the bound of the weights moves often."""
    lens = [777, 2000]
    cache, table, q = base.attend_case(84, lens, H, 256, 64, 64, 8, q_std, lo, hi)
    if lo == 60:   # (scores of the largest scales alone would hide the rest: a query that meets few columns)
        q[:, :, 8:] = 0
        q = (q.float() * 2.0 ** -58).to(torch.bfloat16)
    out, lse = base.run_attend(cache, table, lens, q, 256, scale)
    base.check_attend(cache, table, lens, q, 256, scale, out, lse)


@pytest.mark.parametrize("H", HEADS)
def test_rising_scores(H):
    """Each key outweighs the one before: the bound moves at every step."""
    cache, table, q = base.attend_case(85, [1500], H, 128, 0, 64, 1)
    cache.codes[..., 0] = code(1.0)
    q[:] = 0
    q[..., 0] = 1.0
    t = torch.arange(1500)
    cache.exps[table[0].long()[t // 64], t % 64] = (100 + t // 40).to(torch.uint8)
    out, lse = base.run_attend(cache, table, [1500], q, 128, 1.0)
    base.check_attend(cache, table, [1500], q, 128, 1.0, out, lse)


# ------------------------------------------------- many small weights, alike
#
# n keys of weight P each behind others that outweigh them: what they add up to counts.  With P as the kernel holds it (its
# largest at 2^2 to 2^11.75), the sum is off by
#
#   FP16     2^-11 of itself, or 2^-25 / P where that is more: 2^-9 for P >= 2^-16
#   terms    where rounded to nearest: E4M3 to 2^-4 and the rest by E5M2 to 2^-3, 2^-7 of itself; three E5M2 values 2^-9
#            where rounded up or down by turns along the keys: the share of keys that round up is right to 2^-7 over 2^12
#            keys (test_cache8_rounding), of a step of 2^-2 P, or of 2^-16 <= P: 2^-7
#   scores   2^-22 (|s| + 16) in log2 twice, |s| <= 32: 2^-16
#   out      2^-8
ALIKE = 2.0 ** -9 + 2.0 ** -7 + 2.0 ** -16 + 2.0 ** -8


def alike_case(H, n, ahead, seed):
    """n keys of score 0 and a value of 1 in 64 columns, of which `ahead` ({position: score}) stand out, with a value of 0;
    152 rows whose heads scale the scores by 1 to 1.25, all on one sequence.  The shares of the keys alike, 64 bits."""
    B, size = 152, 64
    cache, table, _ = base.attend_case(seed, [n], H, 128, 64, size, 16)
    q = torch.zeros((B, H, 192), dtype=torch.float64)
    step = torch.arange(B * H, dtype=torch.float64).view(B, H)
    q[..., 0] = 1 + (step * 37 % 32) / 128          # (BF16, and E4M3 twice, hold them)
    cache.exps.fill_(127)
    cache.codes[..., 0] = 0
    cache.codes[..., 64:128] = code(1.0)
    pos = torch.tensor(sorted(ahead))
    page = table[0].long()[pos // size]
    score = ref.VALUES[ref.nearest(torch.tensor([ahead[i] for i in sorted(ahead)], dtype=torch.float64)).long()]
    cache.codes[page, pos % size, 0] = ref.nearest(score)
    cache.codes[page, pos % size, 64:128] = 0
    alike = float(n - len(ahead))
    share = alike / (alike + torch.exp2(q[..., :1] * score).sum(-1))
    return cache, table, q.to(torch.bfloat16), share.to(DEV)


def check_alike(H, n, ahead, seed):
    cache, table, q, share = alike_case(H, n, ahead, seed)
    out, lse = base.run_attend(cache, table, [n], q, 128, math.log(2), seqs=[0] * q.shape[0])
    off = ((out[..., 64:].double() - share[..., None]).abs() / share[..., None]).amax(-1)
    assert off.max() <= ALIKE, f"off by {off.max().item():.4f} of the share, on average {off.mean().item():.4f}"
    want = math.log(n - len(ahead)) - torch.log(share)
    assert (lse.double() - want).abs().max() <= 2.0 ** -16 + (n + 16) * 2.0 ** -23 + 2.0 ** -23 * 32


@pytest.mark.parametrize("H", [16, 32, 40, 64, 100, 128, 130])
@pytest.mark.parametrize("at", [0, 200, 6000, 16383])
def test_many_keys_alike_behind_one(H, at):
    """One key of 2^16 to 2^20 times the weight of 16383 others, in the first step, in the next, in the middle, at the end."""
    check_alike(H, 16384, {at: 16.0}, 86)


@pytest.mark.parametrize("H", [16, 40, 128])
@pytest.mark.parametrize("gap", [9.0, 12.0, 18.0])
def test_many_keys_alike_behind_few(H, gap):
    """Nine keys that outweigh the rest, in several steps."""
    check_alike(H, 16000, {i: gap for i in (3, 77, 130, 131, 132, 1000, 5000, 5001, 15999)}, 87)


@pytest.mark.parametrize("H", [16, 40, 128])
@pytest.mark.parametrize("n", [4300, 60000])
def test_many_keys_alike_behind_uneven_first_ones(H, n):
    """A first step whose scores differ widely, so that the bound leaves room above its largest, and the rest 2^-13 of that
    or less."""
    first = {i: 5.0 + 8.0 * math.sin(1.7 * i) for i in range(128)}
    check_alike(H, n, first, 88)


# ------------------------------------------------------------ other widths

WIDTHS = [(16, 560), (96, 464), (144, 432), (256, 320), (272, 304), (384, 192), (400, 112), (512, 16), (512, 48),   # > 512 columns
          (16, 496), (256, 256), (496, 16), (16, 400), (192, 256),                                                  # 4 chunks
          (16, 368), (128, 256), (256, 128), (320, 0), (16, 240), (144, 112), (16, 112), (48, 0)]                   # fewer


@pytest.mark.parametrize("H", [11, 24, 50, 100])
@pytest.mark.parametrize("Lkv,R", WIDTHS)
def test_values_of_some_of_the_columns(H, Lkv, R):
    """Keys of one to five chunks of 128 columns, values in one to four of them, over many steps: one sequence that several
    units share, and a batch that each unit has many steps and several tiles of."""
    cache, table, q = base.attend_case(89, [9000, 700, 1300, 5], H, Lkv, R, 64, 16)
    seqs = [1, 2, 0, 3] + [1, 2] * 150
    g = base.gen(90)
    q = torch.randn((len(seqs), H, Lkv + R), generator=g).to(torch.bfloat16)
    lens = [9000, 700, 1300, 5]
    for some in ([2], list(range(len(seqs)))):
        status = base.i32([0])
        of = [seqs[b] for b in some]
        out, lse = base.run_attend(cache, table, lens, q[some], Lkv, 0.08, seqs=of, status=status)
        assert status.item() == 0
        few = list(range(min(len(some), 6))) + list(range(max(6, len(some) - 4), len(some)))
        base.check_attend(cache, table, lens, q[some][few], Lkv, 0.08, out[few], lse[few], [of[b] for b in few])


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("power", [6, 12, 18, 24, 30, 40])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_so_large_that_one_value_takes_all(H, power, sign):
    """Scores of up to 25 * 2^power, each exact in FP32, equal or at least 2^(power - 3) apart: the weight goes to the keys of
    the largest, wherever the bound of the weights has to move.  Up to 2^12 they share it alike (2^6: e^-8 of it goes to the
    next).  Beyond that FP32 log-sum-exps of up to 36 * 2^18 in log2, by which the pieces of a sequence are joined, are right
    to half a binade or worse, and the shares of equals are not: but the result lies between their values."""
    lens = [1000, 130, 64, 1, 5000]
    cache, table, q = base.attend_case(91, lens, H, 128, 64, 64, 16, 1.0, 121, 122)
    cache.codes[..., 0] = ref.nearest(torch.randint(4, 200, cache.codes.shape[:2], generator=base.gen(92)).double() / 8)
    q[:] = 0
    q[..., 0] = sign
    scale = 2.0 ** (power + 6)          # (the rows' scale is 2^-6)
    out, lse = base.run_attend(cache, table, lens, q, 128, scale)
    for b, n in enumerate(lens):
        t = torch.arange(n)
        rows = cache.rows(table[b].long()[t // 64] * 64 + t % 64)
        s, values = rows[:, 0] * sign * scale, rows[:, :128]
        z = torch.logsumexp(s, 0)
        p = torch.exp(s - z)
        # weights to 2^-7, theirs and the others' (of 2^-11 and less); 36 * 2^12 in log2 to 2^-24, twice: 2^-5.8
        room = 2.0 ** -8 + 2.0 ** -6 + 2.0 ** -11
        if power <= 12:
            want = p @ values
            tol = (room + (2.0 ** -5.8 if power == 12 else 0)) * (p @ values.abs()) + 1e-30
            low, high = want - tol, want + tol
        else:
            best = values[s == s.max()]
            tol = room * best.abs().amax(0) + 1e-30
            low, high = best.amin(0) - tol, best.amax(0) + tol
        got = out[b].double().cpu()
        assert ((got >= low) & (got <= high)).all(), (b, got.isnan().sum().item())
        assert (lse[b].double() - z.item()).abs().max() <= 2.0 ** -21 * abs(z.item()) + 2.0 ** -8 + (math.log(n) if power > 12 else 0)
