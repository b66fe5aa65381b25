"""Attention operators on the GPU: calls at the edges of their contracts.
Tolerances as derived in test_attend_gpu.py."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

from mla_attention_prolog_gb300 import binding  # noqa: E402
from test_attend_gpu import (DEV, POISON, cache_case, check, check_cache, check_prompt, prompt_case, row_attention,  # noqa: E402
                             run_cache, run_prompt)


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


def cut_to(cu, rows):
    """What the contract makes of offsets: [(first row, rows)] of each sequence."""
    inside = [min(max(x, 0), rows) for x in cu]
    return [(a, max(b - a, 0)) for a, b in zip(inside, inside[1:])]


OFFSETS = [([0, 40, 1000], [0, 40, 90]), ([-4, 40, 90], [0, 40, 90]), ([0, 60, 40], [0, 60, 90]), ([95, 95, 200], [0, 40, 90]),
           ([0, 40, 90], [0, 40, 1000]), ([0, 40, 90], [-7, 40, 90]), ([0, 40, 90], [0, 60, 40]), ([0, 40, 90], [91, 300, 1 << 30]),
           ([0, 1 << 30, -(1 << 31)], [0, 50, 90]), ([-5, -2, 90], [-(1 << 31), 30, (1 << 31) - 1])]


@pytest.mark.parametrize("cu_q,cu_k", OFFSETS)
@pytest.mark.parametrize("extra", [0, 40])   # empty sequences behind: one look of a warp, and more
@pytest.mark.parametrize("q", ["bf16", "int8"])
def test_prompt_offsets_outside_the_buffers_are_cut(cu_q, cu_k, extra, q):
    """Sequences are cut to their rows inside the buffers, by definition, and
    rows of none stay as they were."""
    c = prompt_case(47, [40, 50], [40, 50], 4, 2, 64, 64, q=q, pad=0)
    cu_q, cu_k = cu_q + [cu_q[-1]] * extra, cu_k + [cu_k[-1]] * extra
    for name, cu in (("cu_q", cu_q), ("cu_k", cu_k)):
        c[name] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    out, lse, status = run_prompt(c)
    assert status == binding.STATUS_SEQ_RANGE
    own = torch.zeros(90, dtype=torch.bool, device=DEV)
    for (a, n), (b, t) in zip(cut_to(cu_q, 90), cut_to(cu_k, 90)):
        own[a:a + n] = True
        i, j = torch.arange(n, device=DEV)[:, None], torch.arange(t, device=DEV)[None, :]
        k, v = (c[x][b:b + t].double().permute(1, 0, 2).repeat_interleave(2, 0) for x in "kv")
        o, z, to, tz = row_attention(c["qd"][a:a + n].permute(1, 0, 2), k, v, c["scale"], j > i + (t - n))
        check(out[a:a + n].permute(1, 0, 2), o, to, f"out of the rows from {a}")
        check(lse[a:a + n].t(), z, tz, f"lse of the rows from {a}")
    assert (out[~own].view(torch.int16) == POISON).all() and (lse[~own] == 123.0).all()


@pytest.mark.parametrize("name,T,per_head", [("tiny_q", 150, False), ("tiny_q", 150, True), ("v3_decode", 128, False)])
def test_prompt_on_the_codes_scales_keys_and_values_of_the_prolog(name, T, per_head):
    """The prolog's INT8 q and its scales, K and V, as it leaves them, behind it
    in the stream; then a chain of both, with other inputs each time, against
    the same chain with a synchronize between any two."""
    import dataclasses
    from helpers import alloc_outputs, device_inputs, run_prolog
    from mla_attention_prolog_gb300 import workloads as wl
    w = wl.WORKLOADS[name]
    d = dataclasses.replace(w.dims, T=T, max_pos=max(T, w.dims.max_pos), flags=w.dims.flags | (0x8 if per_head else 0))
    dev = torch.device(DEV, torch.cuda.current_device())
    x = device_inputs(wl.make_inputs(w, d), dev)
    outs = alloc_outputs(d, dev)
    p = binding.MlaProlog.from_dims(d)
    H, D, E = d.num_heads, d.nope_dim + d.rope_dim, d.v_dim
    cu_ = torch.tensor([0, T - 30, T], dtype=torch.int32, device=dev)
    first, ends = x["x"].clone(), []
    for apart in (True, False):
        x["x"].copy_(first)
        res = []
        for turn in range(6):
            run_prolog(p, x, outs)
            if apart:
                torch.cuda.synchronize()
            out, lse = torch.zeros((T, H, E), dtype=torch.bfloat16, device=dev), torch.zeros((T, H), device=dev)
            if apart:
                torch.cuda.synchronize()
            binding.attend_prompt(outs["out_q_int8"].t, outs["out_k"].t, outs["out_v"].t, cu_, cu_, out, lse, scale=D ** -0.5,
                                  q_scale=outs["out_scale"].t)
            if apart:
                torch.cuda.synchronize()
            res.append((out, lse))
            if apart and turn == 0:
                a = 0
                for n in (T - 30, 30):
                    f = lambda t: t[a:a + n].double().permute(1, 0, 2)  # noqa: E731
                    s = outs["out_scale"].t.double().reshape(T, -1, 1)[a:a + n].permute(1, 0, 2)
                    i, j = torch.arange(n, device=dev)[:, None], torch.arange(n, device=dev)[None, :]
                    o, z, to, tz = row_attention(f(outs["out_q_int8"].t) * s, f(outs["out_k"].t), f(outs["out_v"].t), D ** -0.5, j > i)
                    check(f(out), o, to, f"out from row {a}")
                    check(lse[a:a + n].t(), z, tz, f"lse from row {a}")
                    a += n
            x["x"].copy_(x["x"].roll(1, 0))
        torch.cuda.synchronize()
        ends.append(res)
    assert p.device_status() == 0
    p.close()
    for apart, together in zip(*ends):
        assert same(apart, together)
