"""Attention operators on the GPU: calls at the edges of their contracts.
Tolerances as derived in test_attend_gpu.py."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

from mla_attention_prolog_gb300 import binding  # noqa: E402
from test_attend_gpu import DEV, cache_case, check_cache, check_prompt, prompt_case, run_cache, run_prompt  # noqa: E402


def same(a, b):
    return all(torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16)) for x, y in zip(a[:2], b[:2]))


@pytest.mark.parametrize("device", ["cpu", "cuda"])
def test_a_scale_that_is_a_tensor_is_read_at_each_call(device):
    scale = torch.tensor(0.1, device=device)
    p, c = prompt_case(40, [70, 3], [70, 3], 2, 2, 64, 64), cache_case(41, [70, 3], 16, 512, 64, 64)
    for x in (0.1, 0.5, 0.03):
        scale.fill_(x)
        as_float = float(scale)   # the FP32 number that the tensor holds
        for case, run in ((p, run_prompt), (c, run_cache)):
            assert same(run({**case, "scale": scale}), run({**case, "scale": as_float}))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("q", ["int8", "int8_per_head"])
def test_rows_without_a_key_whatever_their_scale(q, bad):
    """Three of five queries come before the first key; their scale is no number."""
    c = prompt_case(42, [5, 200], [2, 131], 4, 2, 192, 128, q=q)
    want = run_prompt(c)
    check_prompt(c, *want[:2])
    for rows in (slice(0, 3), slice(5, 74)):
        c["q_scale"][rows] = bad
    got = run_prompt(c)
    assert got[2] == 0 and same(got, want)
    for rows in (slice(0, 3), slice(5, 74)):
        assert (got[0][rows] == 0).all() and torch.isneginf(got[1][rows]).all()
    c["q_scale"][3] = bad   # a row that has keys
    got = run_prompt(c)
    assert not torch.isfinite(got[0][3].float()).any() and same([x[4:] for x in got[:2]], [x[4:] for x in want[:2]])


def test_cache_the_largest_batch_nearly_all_of_it_empty():
    """One run passes over all the empty sequences between two others."""
    B = 1 << 17
    lens = [70] + [0] * (B - 2) + [90]
    c = cache_case(43, [70, 90], 1, 64, 16, 16)
    seqs = torch.full((B,), 2, dtype=torch.int32, device=DEV)
    seqs[0], seqs[-1] = 0, 1
    table = torch.cat([c["table"], torch.full_like(c["table"][:1], -1)])
    q = torch.zeros((B, 1, 80), dtype=torch.bfloat16, device=DEV)
    q[0], q[-1] = c["q"][0], c["q"][1]
    for order in (seqs, None):
        d = {**c, "q": q, "table": table, "lens": torch.cat([c["lens"], torch.zeros_like(c["lens"][:1])])}
        if order is None:
            d["table"] = table[2:].repeat(B, 1)
            d["table"][0], d["table"][-1] = table[0], table[1]
            d["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        out, lse, status = run_cache(d, seqs=order)
        assert status == 0
        check_cache(c, out[[0, -1]], lse[[0, -1]])
        assert (out[1:-1] == 0).all() and torch.isneginf(lse[1:-1]).all()


def differ_by_roundings(a, b):
    """Another cut of the same keys: results that are joined from other pieces."""
    return not same(a, b)


@pytest.mark.parametrize("H,lens,shared", [(16, [1024 + 40, 1024] + [0] * 38, 1024), (16, [0, 3] * 20 + [2048 + 1, 2100], 2048),
                                           (128, [1100, 1024, 1500, 2000], 1024), (64, [300] * 8, 256)])
def test_cache_a_prefix_that_is_not_worth_tiles_of_its_own(H, lens, shared):
    """A shared length that saves no work changes nothing, not a bit."""
    c = cache_case(44, lens, H, 512, 64, 64, shared)
    prefix = c["rows"][max(range(len(lens)), key=lens.__getitem__)][:shared]
    if lens[0] < shared:   # cache_case fills the prefix for a first sequence that shares it
        g = torch.Generator(DEV).manual_seed(1)
        c["cache"].view(-1, 576)[prefix] = torch.randn((shared, 576), generator=g, device=DEV).to(torch.bfloat16)
    got = run_cache(c)
    assert got[2] == 0 and same(got, run_cache(c, shared=False))
    check_cache(c, *got[:2])


@pytest.mark.parametrize("dims,page,shared,n", [((16, 512, 64), 64, 1024, 60), ((16, 512, 64), 16, 1040, 60), ((64, 512, 64), 64, 2048, 48),
                                                ((130, 512, 64), 64, 2048, 40), ((5, 256, 32), 48, 672, 64), ((1, 512, 0), 16, 720, 150)])
def test_cache_a_prefix_in_tiles_of_its_own(dims, page, shared, n):
    """Many sequences that end at the prefix, a little behind it or far, among
    empty and shorter ones; in the order of seqs, too."""
    lens = [shared + (0, 1, 63, 64, 200)[i % 5] for i in range(n)] + [0, shared - 1, shared // 2]
    c = cache_case(45, lens, *dims, page, shared)
    got = run_cache(c)
    assert got[2] == 0 and differ_by_roundings(got, run_cache(c, shared=False))
    check_cache(c, *got[:2])
    again = run_cache(c)
    assert same(got, again)
    order = list(reversed(range(len(lens))))
    seqs = torch.tensor(order, dtype=torch.int32, device=DEV)
    got = run_cache(c, seqs=seqs)
    assert got[2] == 0
    check_cache(c, *got[:2], order)


def test_cache_a_nan_in_the_prefix_reaches_only_those_who_share_it():
    shared = 1024
    lens = [shared + i for i in range(60)] + [0, 100, shared - 1, shared - 64]
    c = cache_case(46, lens, 16, 512, 64, 64, shared)
    want = run_cache(c)
    row = int(c["rows"][0][500])
    c["cache"].view(-1, 576)[row, 3] = math.nan
    out, lse, status = run_cache(c)
    assert status == 0 and torch.isnan(out[:60].float()).all() and torch.isnan(lse[:60]).all()
    assert same((out[60:], lse[60:]), (want[0][60:], want[1][60:]))
