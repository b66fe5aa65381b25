"""Attention operators on the GPU against the definition in 64 bits.

Tolerances, derived per element from the stated precision: the probabilities
and the output are each rounded to BF16 once (2^-8 relative at most), scores
and sums are FP32.  With D the length of a score's sum, n the keys of a row
and A = sum_j p_j |v_j|:

  |d score| <= ds = (D + 3) 2^-24 max_j scale sum_d |q_d k_jd|
  |d out|   <= 2^-8 |out| + A (2^-8 + 2 ds + (n + 16) 2^-23)
  |d lse|   <= ds + (n + 16) 2^-23 + 2^-23 |lse|
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

from mla_attention_prolog_gb300 import binding  # noqa: E402

DEV = "cuda"
H8 = 2.0 ** -8
NAN = float("nan")
POISON = 0x7FA1   # a BF16 NaN


def rand(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def row_attention(q, k, v, scale, hidden=None):
    """(out, lse, out tolerance, lse tolerance) of q [.., n, D] on k [.., m, D]
    and v [.., m, E], all float64; hidden keys are replaced, never read."""
    n = k.shape[-2]
    s = (q @ k.transpose(-1, -2)) * scale
    mag = (q.abs() @ k.abs().transpose(-1, -2)) * scale
    if hidden is not None:
        s = torch.where(hidden, -math.inf, s)
        mag = torch.where(hidden, 0.0, mag)
    if n == 0:
        z = q.new_full(q.shape[:-1], -math.inf)
        o = q.new_zeros(*q.shape[:-1], v.shape[-1])
        return o, z, o + 1e-30, torch.zeros_like(z)
    z = torch.logsumexp(s, -1)
    p = torch.where(torch.isinf(s) & (s < 0), 0.0, torch.exp(s - torch.where(torch.isinf(z) & (z < 0), 0.0, z)[..., None]))
    o, a = p @ v, p @ v.abs()
    ds = (q.shape[-1] + 3) * 2.0 ** -24 * mag.amax(-1)
    eps = ds + (n + 16) * 2.0 ** -23
    return o, z, H8 * o.abs() + a * (H8 + 2 * eps)[..., None] + 1e-30, eps + 2.0 ** -23 * torch.where(torch.isinf(z), 0.0, z.abs())


def check(got, want, tol, what):
    g = got.double()
    same = torch.isinf(want) & (g == want)
    bad = ~(((g - want).abs() <= tol) | same)
    assert not bad.any(), (f"{what}: {int(bad.sum())}/{bad.numel()} outside; first at {bad.nonzero()[0].tolist()}: "
                           f"{g[bad][0].item()} for {want[bad][0].item()} +- {tol.expand_as(want)[bad][0].item()}")


def cu(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


def prompt_case(seed, new, total, H, Hk, D, E, q="bf16", pad=3, std=1.7):
    g = torch.Generator(DEV).manual_seed(seed)
    tq, tk = sum(new) + pad, sum(total) + pad
    c = dict(new=new, total=total, k=rand(g, (tk, Hk, D)), v=rand(g, (tk, Hk, E)), q_scale=None, scale=D ** -0.5,
             cu_q=cu(new), cu_k=cu(total))
    if pad:   # what lies behind the last sequence never reaches a result
        c["k"][-pad:] = NAN
        c["v"][-pad:] = NAN
    if q == "bf16":
        c["q"] = rand(g, (tq, H, D), std)
        c["qd"] = c["q"].double()
    else:
        c["q"] = torch.randint(-127, 128, (tq, H, D), generator=g, device=DEV).to(torch.int8)
        c["q_scale"] = torch.rand((tq, H) if q == "int8_per_head" else (tq,), generator=g, device=DEV) * 0.05
        c["qd"] = c["q"].double() * c["q_scale"].double().reshape(tq, -1, 1)
    return c


def run_prompt(c, causal=True, **kw):
    tq, H, E = c["q"].shape[0], c["q"].shape[1], c["v"].shape[2]
    out = torch.full((tq, H, E), POISON, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    lse = torch.full((tq, H), 123.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    binding.attend_prompt(c["q"], c["k"], c["v"], c["cu_q"], c["cu_k"], out, lse, scale=c["scale"], causal=causal,
                          q_scale=c["q_scale"], status=status, **kw)
    return out, lse, int(status.item())


def check_prompt(c, out, lse, causal=True):
    H, Hk = c["q"].shape[1], c["k"].shape[1]
    a = b = 0
    for n, t in zip(c["new"], c["total"]):
        i, j = torch.arange(n, device=DEV)[:, None], torch.arange(t, device=DEV)[None, :]
        hidden = (j > i + (t - n)) if causal else None
        q = c["qd"][a:a + n].permute(1, 0, 2)
        k = c["k"][b:b + t].double().permute(1, 0, 2).repeat_interleave(H // Hk, 0)
        v = c["v"][b:b + t].double().permute(1, 0, 2).repeat_interleave(H // Hk, 0)
        o, z, to, tz = row_attention(q, k, v, c["scale"], hidden)
        check(out[a:a + n].permute(1, 0, 2), o, to, f"out of the sequence at row {a}")
        check(lse[a:a + n].t(), z, tz, f"lse of the sequence at row {a}")
        a, b = a + n, b + t
    assert (out[a:].view(torch.int16) == POISON).all() and (lse[a:] == 123.0).all()


DIMS = [(2, 2, 192, 128), (4, 2, 128, 128), (8, 1, 64, 64), (2, 2, 48, 32), (3, 3, 80, 112), (2, 1, 256, 128),
        (6, 3, 16, 16)]
LENGTHS = [[1], [127], [128], [129], [255, 1, 257], [1, 7, 100, 513, 33], [300, 0, 40], [640]]


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("lens", LENGTHS, ids=lambda x: "+".join(map(str, x)))
def test_prompt_causal(dims, lens):
    c = prompt_case(1, lens, lens, *dims)
    out, lse, status = run_prompt(c)
    assert status == 0
    check_prompt(c, out, lse)


@pytest.mark.parametrize("q", ["int8", "int8_per_head"])
@pytest.mark.parametrize("dims", [(4, 4, 192, 128), (4, 2, 80, 48)])
def test_prompt_int8(q, dims):
    c = prompt_case(2, [70, 1, 300], [70, 1, 300], *dims, q=q)
    c["q_scale"][5] = 0.0   # a zero row, as the quantisation gives it
    c["qd"][5] = 0.0
    out, lse, status = run_prompt(c)
    assert status == 0
    check_prompt(c, out, lse)


@pytest.mark.parametrize("new,total", [([1], [1000]), ([5, 64], [133, 64]), ([200], [1400]), ([129, 1, 300], [257, 900, 700]),
                                       ([3], [0]), ([5, 260], [2, 131])],
                         ids=lambda x: "+".join(map(str, x)))
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_chunks_and_rows_without_keys(new, total, causal):
    """Queries behind cached tokens, and fewer keys than queries: rows whose
    mask leaves nothing are zero with lse -inf."""
    c = prompt_case(3, new, total, 4, 2, 192, 128)
    out, lse, status = run_prompt(c, causal)
    assert status == 0
    check_prompt(c, out, lse, causal)


def test_prompt_hidden_keys_may_hold_anything():
    """NaN and infinities in keys that the causal rule hides reach no row that
    must not see them, and every row that does."""
    c = prompt_case(4, [300], [300], 2, 2, 192, 128)
    c["v"][200, 0, 5] = math.inf
    c["v"][210, 1, 7] = NAN
    c["k"][250, 0] = NAN
    out, lse, _ = run_prompt(c)
    clean = {**c, "k": c["k"].clone(), "v": c["v"].clone()}
    clean["k"][200:], clean["v"][200:] = 1.0, 1.0
    want, want_lse, _ = run_prompt(clean)
    assert torch.equal(out[:200].view(torch.int16), want[:200].view(torch.int16)) and torch.equal(lse[:200], want_lse[:200])
    assert torch.isinf(out[200:250, 0, 5]).all() and (out[200:250, 0, 5] > 0).all()
    assert torch.isfinite(out[:250, 0, :5]).all() and torch.isfinite(out[:250, 0, 6:]).all()
    assert torch.isnan(out[210:300, 1, 7]).all() and torch.isfinite(out[:300, 1, 8:]).all()
    assert torch.isfinite(out[:210, 1, 7]).all()
    assert torch.isnan(out[250:300, 0]).all() and torch.isnan(lse[250:300, 0]).all()
    assert torch.isfinite(lse[:250, 0]).all()


def test_prompt_large_scores():
    """Scores of several hundred: nothing overflows."""
    c = prompt_case(5, [200, 333], [200, 333], 2, 2, 192, 128, std=60.0)
    out, lse, _ = run_prompt(c)
    check_prompt(c, out, lse)


def test_prompt_offsets_outside_the_buffers():
    c = prompt_case(6, [40, 50], [40, 50], 2, 2, 64, 64, pad=0)
    for bad in ([0, 40, 1000], [-4, 40, 90], [0, 60, 40]):
        c["cu_q"] = torch.tensor(bad, dtype=torch.int32, device=DEV)
        out, lse, status = run_prompt(c)
        assert status == binding.STATUS_SEQ_RANGE
    c["cu_q"] = cu([40, 50])
    out, lse, status = run_prompt(c)
    assert status == 0
    check_prompt(c, out, lse)


def test_prompt_without_lse_and_repeated():
    c = prompt_case(7, [500, 77], [500, 77], 4, 4, 192, 128)
    out, lse, _ = run_prompt(c)
    again, lse2, _ = run_prompt(c)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)
    binding.attend_prompt(c["q"], c["k"], c["v"], c["cu_q"], c["cu_k"], again, None, scale=c["scale"])
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_prompt_on_a_stream_and_in_a_graph():
    c = prompt_case(8, [300, 21], [300, 21], 4, 4, 192, 128)
    want, want_lse, _ = run_prompt(c)
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        binding.attend_prompt(c["q"], c["k"], c["v"], c["cu_q"], c["cu_k"], out, lse, scale=c["scale"])
    s.synchronize()
    assert torch.equal(out[:321].view(torch.int16), want[:321].view(torch.int16))
    with torch.cuda.graph(g):
        binding.attend_prompt(c["q"], c["k"], c["v"], c["cu_q"], c["cu_k"], out, lse, scale=c["scale"])
    # the replay follows the offsets and the inputs
    d = prompt_case(9, [121, 200], [121, 200], 4, 4, 192, 128)
    for k in ("q", "k", "v", "cu_q", "cu_k"):
        c[k].copy_(d[k])
    g.replay()
    torch.cuda.synchronize()
    check_prompt(d, out.clone().index_fill_(0, torch.arange(321, 324, device=DEV), 0).view(torch.int16).index_fill_(
        0, torch.arange(321, 324, device=DEV), POISON).view(torch.bfloat16),
        lse.index_fill(0, torch.arange(321, 324, device=DEV), 123.0))


def test_prompt_many_short_sequences():
    """More sequences than one look of a warp covers, many of them empty; the
    first ones' rows lie behind rows of no sequence."""
    lens = [i * 7 % 5 - 1 if i % 5 else 0 for i in range(700)]
    lens = [max(n, 0) for n in lens] + [150]
    c = prompt_case(20, lens, lens, 2, 1, 64, 64)
    out, lse, status = run_prompt(c)
    assert status == 0
    check_prompt(c, out, lse)
    head = 4   # the same rows, but the first sequences left out: rows before cu_q[0] stay as they were
    first = int(c["cu_q"][head].item())
    sub = {**c, "cu_q": c["cu_q"][head:].contiguous(), "cu_k": c["cu_k"][head:].contiguous()}
    part, plse, status = run_prompt(sub)
    assert status == 0 and first > 0
    assert (part[:first].view(torch.int16) == POISON).all() and (plse[:first] == 123.0).all()
    assert torch.equal(part[first:].view(torch.int16), out[first:].view(torch.int16)) and torch.equal(plse[first:], lse[first:])


def test_prompt_int8_lowest_code_and_negative_scales():
    c = prompt_case(21, [140, 3], [140, 3], 2, 2, 192, 128, q="int8")
    c["q"][:, :, ::5] = -128
    c["q_scale"][::3] *= -1.0
    c["qd"] = c["q"].double() * c["q_scale"].double().reshape(-1, 1, 1)
    out, lse, status = run_prompt(c)
    assert status == 0
    check_prompt(c, out, lse)


def test_prompt_one_query_on_many_keys():
    c = prompt_case(22, [1, 2], [20011, 5000], 4, 2, 192, 128)
    out, lse, status = run_prompt(c)
    assert status == 0
    check_prompt(c, out, lse)


@pytest.mark.parametrize("H", [2, 20, 60])   # clusters of 8, 4 and 2 CTAs on a tile pair's keys
@pytest.mark.parametrize("dims,q", [((192, 128), "bf16"), ((192, 128), "int8"), ((80, 48), "bf16"), ((256, 112), "bf16"),
                                    ((16, 16), "int8_per_head")])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_keys_shared_by_a_cluster(H, dims, q, causal):
    for new, total in (([130], [1531]), ([256], [769]), ([1], [1000])):
        c = prompt_case(26, new, total, H, H // 2, *dims, q=q)
        out, lse, status = run_prompt(c, causal)
        assert status == 0
        check_prompt(c, out, lse, causal)
    again, lse2, _ = run_prompt(c, causal)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


def test_prompt_clusters_with_uneven_sequences():
    """Clusters whose CTAs have a key tile, or none, and rows that see no key."""
    for H in (1, 10, 30):
        c = prompt_case(27, [5, 260], [2400, 131], H, 1, 192, 128)
        out, lse, status = run_prompt(c)
        assert status == 0
        check_prompt(c, out, lse)


@pytest.mark.parametrize("H", [2, 20, 60])
def test_prompt_clusters_and_hidden_keys(H):
    c = prompt_case(28, [300], [1000], H, 2, 192, 128)
    c["v"][900, 0, 5] = math.inf    # seen by the queries from 200 on
    c["v"][910, 1, 7] = NAN
    c["k"][950, 0] = NAN
    out, lse, _ = run_prompt(c)
    clean = {**c, "k": c["k"].clone(), "v": c["v"].clone()}
    clean["k"][900:], clean["v"][900:] = 1.0, 1.0
    want, want_lse, _ = run_prompt(clean)
    h = H // 2   # heads of key head 0
    assert torch.equal(out[:200].view(torch.int16), want[:200].view(torch.int16)) and torch.equal(lse[:200], want_lse[:200])
    assert (out[200:250, :h, 5] == math.inf).all() and torch.isfinite(out[:250, :h, :5]).all()
    assert torch.isnan(out[210:300, h:, 7]).all() and torch.isfinite(out[:210, h:, 7]).all()
    assert torch.isfinite(out[:300, h:, 8:]).all() and torch.isfinite(lse[:250, :h]).all()
    assert torch.isnan(out[250:300, :h]).all() and torch.isnan(lse[250:300, :h]).all()


def test_prompt_and_cache_calls_at_once():
    """Prompts and decoding steps on three streams at the same time."""
    ps = [prompt_case(23, [700, 90], [700, 90], 4, 4, 192, 128), prompt_case(24, [33, 300], [133, 300], 4, 4, 192, 128)]
    cc = cache_case(25, [900, 10, 2000, 64], 128, 512, 64, 64)
    B, H, L = 4, 128, 512
    pouts = [[torch.zeros((*c["q"].shape[:2], 128), dtype=torch.bfloat16, device=DEV), torch.zeros(c["q"].shape[:2], device=DEV)]
             for c in ps]
    cout = [torch.zeros((B, H, L), dtype=torch.bfloat16, device=DEV), torch.zeros((B, H), device=DEV)]
    ws = torch.empty(binding.attend_cache_workspace_bytes(B, H, L, 64), dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, o, s in zip(ps, pouts, streams):
            binding.attend_prompt(c["q"], c["k"], c["v"], c["cu_q"], c["cu_k"], *o, scale=c["scale"], status=status, stream=s)
        binding.attend_cache(cc["q"], cc["cache"], cc["table"], cc["lens"], *cout, ws, scale=cc["scale"], status=status,
                             stream=streams[2])
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for c, (o, z) in zip(ps, pouts):
        n = sum(c["new"])
        o.view(torch.int16)[n:] = POISON
        z[n:] = 123.0
        check_prompt(c, o, z)
    check_cache(cc, *cout)


# ------------------------------------------------------------------ the cache

def cache_case(seed, lens, H, Lkv, R, page, shared=0, spare=3):
    """Paged latent cache; what no sequence holds is NaN."""
    g = torch.Generator(DEV).manual_seed(seed)
    C, B = Lkv + R, len(lens)
    sp = shared // page
    width = max(1, max(-(-n // page) for n in lens)) + 1
    count = sp + sum(max(0, -(-n // page) - (sp if n >= shared else 0)) for n in lens) + spare
    order = torch.randperm(count, generator=g, device=DEV).tolist()
    cache = torch.full((count, page, C), NAN, device=DEV, dtype=torch.bfloat16)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at, rows = sp, []
    for b, n in enumerate(lens):
        keep = sp if n >= shared else 0
        k = -(-n // page)
        table[b, :k] = torch.tensor(order[:keep] + order[at:at + k - keep], dtype=torch.int32)
        at += k - keep
        slots = (table[b].long()[:, None] * page + torch.arange(page)).reshape(-1)[:n].to(DEV)
        new = slots if (keep == 0 or not rows) else slots[shared:]
        cache.view(-1, C)[new] = rand(g, (new.numel(), C))
        rows.append(slots)
    return dict(q=rand(g, (B, H, C)), cache=cache, table=table.to(DEV), lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                rows=rows, scale=192.0 ** -0.5, Lkv=Lkv, shared=torch.tensor([shared], dtype=torch.int32, device=DEV))


def run_cache(c, seqs=None, shared=True, **kw):
    (B, H, C), Lkv = c["q"].shape, c["Lkv"]
    out = torch.full((B, H, Lkv), POISON, dtype=torch.int16, device=DEV).view(torch.bfloat16)
    lse = torch.full((B, H), 123.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    n = binding.attend_cache_workspace_bytes(B, H, Lkv, C - Lkv)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)   # NaN where read before written
    binding.attend_cache(c["q"], c["cache"], c["table"], c["lens"], out, lse, ws, scale=c["scale"], seqs=seqs,
                         shared_len=c["shared"] if shared else None, status=status, **kw)
    return out, lse, int(status.item())


def check_cache(c, out, lse, order=None):
    flat = c["cache"].view(-1, c["cache"].shape[-1])
    for b in range(out.shape[0]):
        rows = flat[c["rows"][b if order is None else order[b]]].double()
        o, z, to, tz = row_attention(c["q"][b].double(), rows, rows[:, :c["Lkv"]], c["scale"])
        check(out[b], o, to, f"out of sequence {b}")
        check(lse[b], z, tz, f"lse of sequence {b}")


@pytest.mark.parametrize("dims", [(16, 512, 64), (128, 512, 64), (130, 512, 64), (5, 256, 32), (2, 64, 16), (33, 512, 0), (1, 16, 16),
                                  (64, 448, 128), (20, 80, 48)])
@pytest.mark.parametrize("page", [16, 48, 64, 128])
def test_cache(dims, page):
    c = cache_case(1, [1, 0, 63, 64, 65, 130, 700], *dims, page)
    out, lse, status = run_cache(c)
    assert status == 0
    check_cache(c, out, lse)


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("shared", [16, 48, 64, 640])
def test_cache_with_a_shared_prefix(H, shared):
    """Sequences that end at the prefix, go beyond it, or (a padded batch) are
    shorter than it; shared or not, the same answer within the tolerance."""
    c = cache_case(2, [shared + n for n in (0, 1, 70, 500)] + [0, shared // 2], H, 512, 64, 16, shared)
    out, lse, status = run_cache(c)
    assert status == 0
    check_cache(c, out, lse)
    check_cache(c, *run_cache(c, shared=False)[:2])


def test_cache_shared_length_inside_a_page_and_beyond():
    """shared_len need not end with a page, and one beyond every sequence shares nothing."""
    c = cache_case(3, [164, 164 + 77, 300], 16, 512, 64, 64, 128)
    for n in (0, 1, 100, 127, 128, 5000, -3):
        c["shared"].fill_(n)
        out, lse, _ = run_cache(c)
        check_cache(c, out, lse)


def test_cache_sequences_a_little_shorter_than_the_shared_prefix():
    """Pages are shared from shared_len tokens on; a shorter sequence has its
    own, however near its length is."""
    for shared, lens in ((208, [258, 200, 207, 400, 208, 193, 130]), (144, [144, 130, 143, 500, 128, 64]), (80, [80, 64, 79, 81, 200])):
        c = cache_case(32, lens, 16, 512, 64, 16, shared)
        out, lse, status = run_cache(c)
        assert status == 0
        check_cache(c, out, lse)


def test_cache_one_long_sequence_among_short_ones():
    c = cache_case(4, [9000, 3, 0, 17], 16, 512, 64, 64)
    out, lse, status = run_cache(c)
    assert status == 0
    check_cache(c, out, lse)
    again, lse2, _ = run_cache(c)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


def test_cache_rows_through_seqs():
    c = cache_case(5, [100, 40, 0, 333, 64], 16, 512, 64, 32)
    order = [3, 0, 3, 2, 4]
    seqs = torch.tensor(order, dtype=torch.int32, device=DEV)
    out, lse, status = run_cache(c, seqs=seqs)
    assert status == 0
    check_cache(c, out, lse, order)
    seqs[1], seqs[2] = -1, 99
    out, lse, status = run_cache(c, seqs=seqs)
    assert status == binding.STATUS_SEQ_RANGE
    assert (out[1:3] == 0).all() and torch.isneginf(lse[1:3]).all()


def test_cache_bad_pages_read_as_zeros():
    c = cache_case(6, [200, 90], 16, 512, 64, 64)
    c["table"][0, 1] = c["cache"].shape[0]
    c["table"][1, 0] = -7
    out, lse, status = run_cache(c)
    assert status == binding.STATUS_PAGE_RANGE
    flat = torch.cat([c["cache"], torch.zeros_like(c["cache"][:1])]).view(-1, 576)
    c["cache"] = flat.view(-1, 64, 576)
    for b, j in ((0, 1), (1, 0)):
        rows = c["rows"][b]
        hit = torch.arange(rows.numel(), device=DEV) // 64 == j
        rows[hit] = (flat.shape[0] - 64) + torch.arange(int(hit.sum()), device=DEV)
    check_cache(c, out, lse)


def test_cache_lengths_outside_the_table():
    c = cache_case(7, [100, 64], 16, 512, 64, 64)
    c["table"] = c["table"][:, :2].contiguous()
    c["lens"][0], c["lens"][1] = -5, 1 << 30
    c["table"][1] = c["table"][0]
    c["cache"].nan_to_num_()
    out, lse, status = run_cache(c)
    assert status == binding.STATUS_SEQ_RANGE
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
    c["rows"][1] = (c["table"][1].long()[:, None] * 64 + torch.arange(64, device=DEV)).reshape(-1)
    check_cache({**c, "q": c["q"][1:], "rows": c["rows"][1:]}, out[1:], lse[1:])


def test_cache_behind_32_bit_offsets():
    """A cache of more than 2^32 bytes and 2^31 elements: pages at its end."""
    pages = (1 << 31) // (64 * 576) + 100
    c = cache_case(8, [130, 64], 16, 512, 64, 64)
    big = torch.zeros((pages, 64, 576), dtype=torch.bfloat16, device=DEV)
    n = c["cache"].shape[0]
    big[-n:] = c["cache"]
    c["table"] = torch.where(c["table"] >= 0, c["table"] + (pages - n), c["table"])
    c["rows"] = [r + (pages - n) * 64 for r in c["rows"]]
    c["cache"] = big
    out, lse, status = run_cache(c)
    assert status == 0
    check_cache(c, out, lse)


@pytest.mark.parametrize("shared", [0, 192])
def test_cache_large_batch(shared):
    """More sequences than a CTA has threads, some empty, some shorter than the prefix."""
    g = torch.Generator().manual_seed(11)
    own = torch.randint(0, 150, (450,), generator=g).tolist()
    lens = [shared + n if i % 7 else n for i, n in enumerate(own)]
    lens[0] = shared + 1
    c = cache_case(11, lens, 4, 512, 64, 64, shared)
    out, lse, status = run_cache(c)
    assert status == 0
    check_cache(c, out, lse)


def test_cache_shared_prefix_seen_first_by_a_later_row():
    """The first sequence is shorter than the prefix; one sequence alone shares nothing."""
    c = cache_case(12, [500, 10, 470, 0], 16, 512, 64, 64, 448)
    for rows in ([1, 0, 2], [1, 3, 0], [3, 1, 1]):
        seqs = torch.tensor(rows, dtype=torch.int32, device=DEV)
        d = {**c, "q": c["q"][:3].contiguous()}
        out, lse, status = run_cache(d, seqs=seqs)
        assert status == 0
        check_cache(d, out, lse, rows)


def test_cache_without_pages():
    c = cache_case(13, [0, 0, 0], 16, 512, 64, 64, spare=0)
    assert c["cache"].shape[0] == 0
    out, lse, status = run_cache(c)
    assert status == 0 and (out == 0).all() and torch.isneginf(lse).all()
    c["lens"][1] = 70   # and no page to hold them: rows of zeros
    c["table"] = torch.zeros((3, 2), dtype=torch.int32, device=DEV)
    out, lse, status = run_cache(c)
    assert status == binding.STATUS_PAGE_RANGE and (out == 0).all()
    assert (lse[1] - math.log(70)).abs().max() <= 1e-5


def test_cache_refuses_a_small_workspace():
    c = cache_case(14, [100, 40], 16, 512, 64, 64)
    n = binding.attend_cache_workspace_bytes(2, 16, 512, 64)
    out, lse = torch.zeros((2, 16, 512), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 16), device=DEV)
    for ws in (torch.empty(n - 1, dtype=torch.uint8, device=DEV), torch.empty(n + 8, dtype=torch.uint8, device=DEV)[8:]):
        with pytest.raises(binding.MlaPrologError):
            binding.attend_cache(c["q"], c["cache"], c["table"], c["lens"], out, lse, ws, scale=1.0)


def test_binding_refusals():
    """Shapes, types and layouts that do not belong together, before any launch."""
    c = prompt_case(15, [20], [20], 2, 2, 64, 64, pad=0)
    out = torch.zeros((20, 2, 64), dtype=torch.bfloat16, device=DEV)
    call = lambda **kw: binding.attend_prompt(*{**dict(q=c["q"], k=c["k"], v=c["v"], cu_q=c["cu_q"], cu_k=c["cu_k"],  # noqa: E731
                                                        out=out), **kw}.values(), scale=1.0)
    call()
    for kw, err in ((dict(q=c["q"].float()), TypeError), (dict(k=c["k"][:, :, :32]), ValueError), (dict(cu_k=c["cu_k"][:1]), ValueError),
                    (dict(cu_q=c["cu_q"].long()), TypeError), (dict(v=c["v"].transpose(0, 1)), ValueError),
                    (dict(out=out.transpose(0, 1)), ValueError), (dict(q=c["q"].cpu()), TypeError),
                    (dict(k=c["k"].cpu()), TypeError)):
        with pytest.raises(err):
            call(**kw)
    with pytest.raises(binding.MlaPrologError):   # 16-byte alignment
        flat = torch.zeros(20 * 2 * 64 + 4, dtype=torch.bfloat16, device=DEV)
        call(out=flat[4:].view(20, 2, 64))


def test_cache_two_graphs_with_their_own_workspaces():
    """Two captured calls replayed at once on two streams, then again with
    other lengths."""
    cs = [cache_case(9, [700, 3, 64], 16, 512, 64, 64), cache_case(10, [5, 1200, 300], 16, 512, 64, 64)]
    outs, graphs, keep = [], [], []
    for c in cs:
        out, lse = (torch.zeros(s, dtype=t, device=DEV) for s, t in (((3, 16, 512), torch.bfloat16), ((3, 16), torch.float32)))
        ws = torch.empty(binding.attend_cache_workspace_bytes(3, 16, 512, 64), dtype=torch.uint8, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            binding.attend_cache(c["q"], c["cache"], c["table"], c["lens"], out, lse, ws, scale=c["scale"])
        outs.append((out, lse)), graphs.append(g), keep.append(ws)
    streams = [torch.cuda.Stream() for _ in cs]
    for turn in range(3):
        if turn == 2:
            for c in cs:
                c["lens"].copy_(torch.tensor([1, 2, 50], dtype=torch.int32))
                c["rows"] = [r[:n] for r, n in zip(c["rows"], (1, 2, 50))]
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for c, (out, lse) in zip(cs, outs):
            check_cache(c, out, lse)


def test_calls_that_feed_one_another():
    """Launches overlap the end of the ones before them: a chain of calls, each
    on what the last one wrote, gives the bits of the same chain with a
    synchronize between any two."""
    H, E, n = 4, 64, 300
    c = prompt_case(30, [n, 17], [n, 17], H, H, 64, E, pad=0)
    cc = cache_case(31, [n, 17], H, E, 0, 16)
    ws = torch.empty(binding.attend_cache_workspace_bytes(2, H, E, 0), dtype=torch.uint8, device=DEV)
    ends = []
    for apart in (False, True):
        a, b = c["v"].clone(), torch.empty_like(c["v"])
        q, o = cc["q"].clone(), torch.empty((2, H, E), dtype=torch.bfloat16, device=DEV)
        torch.cuda.synchronize()
        for _ in range(40):
            binding.attend_prompt(c["q"], c["k"], a, c["cu_q"], c["cu_k"], b, scale=c["scale"])
            if apart:
                torch.cuda.synchronize()
            binding.attend_cache(q, cc["cache"], cc["table"], cc["lens"], o, None, ws, scale=cc["scale"])
            if apart:
                torch.cuda.synchronize()
            a, b, q, o = b, a, o, q
        torch.cuda.synchronize()
        ends.append((a.view(torch.int16).clone(), q.view(torch.int16).clone()))
    assert torch.equal(ends[0][0], ends[1][0]) and torch.equal(ends[0][1], ends[1][1])


def test_prolog_cache_and_attention_together():
    """A prompt and a decoding step, end to end: the pool hands out slots, the
    prolog writes K, V and the latent cache, the prompt attention reads K and
    V; the last token's row, absorbed, reads the same result from the cache."""
    import dataclasses
    from mla_attention_prolog_gb300 import workloads as wl
    from helpers import alloc_outputs, device_inputs
    T, page = 200, 16
    d = dataclasses.replace(wl.WORKLOADS["v2lite_decode"].dims, T=T)
    inp = wl.make_inputs(wl.WORKLOADS["v2lite_decode"], d)
    dev = torch.device(DEV, torch.cuda.current_device())
    x, outs = device_inputs(inp, dev), alloc_outputs(d, dev)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    table, lens, refs = torch.full((4, 20), -1, dtype=torch.int32, device=dev), i32(0, 0, 0, 0), torch.zeros(40, dtype=torch.int32, device=dev)
    pool = binding.PagePool(table, lens, refs, page)
    slots, pos = (torch.zeros(T, dtype=torch.int32, device=dev) for _ in "ab")
    pool.extend(i32(2), i32(T), slots, pos)
    cache = torch.full((40, page, 576), NAN, dtype=torch.bfloat16, device=dev)
    p = binding.MlaProlog.from_dims(d)
    p.run_cached(x["x"], x["gamma"], x["W_a"], x["W_b"], pos, x["cos_sin"], outs["out_k"].t, outs["out_v"].t,
                 outs["out_kpe"].t, None, None, slots, cache.view(-1, 576))
    H, Dn, R, Dv, L = 16, 128, 64, 128, 512
    g = torch.Generator(DEV).manual_seed(11)
    q = rand(g, (T, H, Dn + R))
    out = torch.zeros((T, H, Dv), dtype=torch.bfloat16, device=dev)
    lse = torch.zeros((T, H), device=dev)
    scale = 192.0 ** -0.5
    binding.attend_prompt(q, outs["out_k"].t, outs["out_v"].t, i32(0, T), i32(0, T), out, lse, scale=scale)
    # fork the prompt twice, copy its last page, and decode its last token in all three
    src, dst = i32(-1, -1), i32(-1, -1)
    pool.fork(i32(2, 2), i32(0, 3), src, dst)
    binding.copy_pages(cache, src, dst)
    moved = torch.zeros(40, dtype=torch.int32, device=dev)
    pool.compact(moved)
    binding.copy_pages(cache, None, moved)
    wkvb = x["W_b"].view(H, Dn + Dv, L).double()
    qa = torch.cat([torch.einsum("hd,hdl->hl", q[-1, :, :Dn].double(), wkvb[:, :Dn]), q[-1, :, Dn:].double()], -1)
    qa = qa.to(torch.bfloat16)[None].repeat(3, 1, 1)
    lat = torch.zeros((3, H, L), dtype=torch.bfloat16, device=dev)
    lse3 = torch.zeros((3, H), device=dev)
    ws = torch.empty(binding.attend_cache_workspace_bytes(3, H, L, R), dtype=torch.uint8, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    binding.attend_cache(qa, cache, table, lens, lat, lse3, ws, scale=scale, seqs=i32(0, 2, 3), shared_len=i32(T // page * page),
                         status=status)
    assert int(status.item()) == 0 and p.device_status() == 0
    p.close()
    got = torch.einsum("bhl,hdl->bhd", lat.double(), wkvb[:, Dn:])
    rms = out[-1].double().pow(2).mean().sqrt()
    # BF16 roundings of k, v and q on one side, of the absorbed q and the latent sum on the other: each 2^-8
    # of the score's or result's size at most, on scores of a few units
    assert (got - out[-1].double()).pow(2).mean().sqrt() <= 8 * H8 * rms
    assert (lse3 - lse[-1]).abs().max() <= 32 * H8
    check_cache(dict(q=qa, cache=cache, Lkv=L, scale=scale, rows=[
        (table[s].long()[:, None] * page + torch.arange(page, device=dev)).reshape(-1)[:T] for s in (0, 2, 3)]), lat, lse3)
