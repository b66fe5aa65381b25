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
