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
