"""Host-side checks of the attention and page entry points: arguments that are
refused before any CUDA call (no GPU needed)."""
import ctypes

import pytest

from mla_attention_prolog_gb300 import binding

P16, P4 = ctypes.c_void_p(4096), ctypes.c_void_p(4100)   # never dereferenced on the host
INVALID, DIMS = -1, -2


@pytest.fixture(scope="module")
def L():
    from mla_attention_prolog_gb300 import build
    build.build()
    return binding.lib()


def prompt_dims(**kw):
    base = dict(Tq=8, Tk=8, sequences=1, num_heads=4, kv_heads=2, qk_dim=192, v_dim=128, scale=0.1, flags=1)
    return binding.MlaPrologPromptDims(*{**base, **kw}.values())


def prompt(L, d, **kw):
    base = dict(q=P16, q_scale=None, k=P16, v=P16, cu_q=P4, cu_k=P4, out=P16, lse=P4, status=P4, stream=None)
    return L.mla_prolog_attend_prompt(ctypes.byref(d) if d else None, *{**base, **kw}.values())


@pytest.mark.parametrize("kw,code", [
    (dict(Tq=-1), DIMS), (dict(Tk=-1), DIMS), (dict(sequences=-1), DIMS), (dict(kv_heads=0), DIMS),
    (dict(kv_heads=3), DIMS), (dict(num_heads=0), DIMS), (dict(num_heads=70000, kv_heads=1), DIMS),
    (dict(qk_dim=0), DIMS), (dict(qk_dim=40), DIMS), (dict(qk_dim=272), DIMS), (dict(v_dim=144), DIMS),
    (dict(v_dim=20), DIMS), (dict(scale=0.0), DIMS), (dict(scale=-1.0), DIMS), (dict(scale=float("nan")), DIMS),
    (dict(scale=float("inf")), DIMS), (dict(flags=8), INVALID), (dict(flags=4), INVALID),
    (dict(flags=2), INVALID),   # INT8 q without scales
])
def test_prompt_dims(L, kw, code):
    assert prompt(L, prompt_dims(**kw)) == code


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=P4), dict(k=None), dict(k=P4), dict(v=None), dict(v=P4),
                                dict(out=None), dict(out=P4), dict(cu_q=None), dict(cu_k=None),
                                dict(lse=ctypes.c_void_p(4098)), dict(status=ctypes.c_void_p(4098)), dict(q_scale=P4)])
def test_prompt_pointers(L, kw):
    assert prompt(L, prompt_dims(), **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(Tq=(1 << 30) + 1), dict(Tk=(1 << 30) + 1), dict(scale=2e30), dict(scale=1e-50)])
def test_prompt_dims_behind_32_bits(L, kw):
    assert prompt(L, prompt_dims(**kw)) == DIMS


def test_prompt_nothing_to_do(L):
    assert prompt(L, None) == INVALID
    assert prompt(L, prompt_dims(Tq=0), q=None, out=None) == 0
    assert prompt(L, prompt_dims(sequences=0)) == 0


def cache_dims(**kw):
    base = dict(batch=2, num_heads=16, kv_lora_rank=512, rope_dim=64, page_size=64, table_rows=2, max_pages=8, scale=0.1,
                num_pages=16)
    return binding.MlaPrologCacheDims(*{**base, **kw}.values())


def cache(L, d, **kw):
    base = dict(q=P16, kv_cache=P16, page_table=P4, seq_lens=P4, seqs=None, shared_len=None, out=P16, lse=P4,
                workspace=P16, workspace_bytes=1 << 40, status=P4, stream=None)
    return L.mla_prolog_attend_cache(ctypes.byref(d) if d else None, *{**base, **kw}.values())


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), DIMS), (dict(num_heads=0), DIMS), (dict(batch=1 << 20, num_heads=17), DIMS),
    (dict(kv_lora_rank=0), DIMS), (dict(kv_lora_rank=40), DIMS), (dict(kv_lora_rank=528), DIMS),
    (dict(rope_dim=-16), DIMS), (dict(rope_dim=24), DIMS), (dict(rope_dim=80), DIMS),   # 512 + 80 > 576
    (dict(kv_lora_rank=256, rope_dim=144), DIMS), (dict(page_size=0), DIMS), (dict(page_size=24), DIMS),
    (dict(max_pages=0), DIMS), (dict(max_pages=1 << 25), DIMS), (dict(num_pages=-1), DIMS),
    (dict(num_pages=1 << 26), DIMS), (dict(table_rows=-1), DIMS), (dict(scale=0.0), DIMS),
    (dict(scale=float("nan")), DIMS), (dict(table_rows=1), INVALID),
])
def test_cache_dims(L, kw, code):
    assert cache(L, cache_dims(**kw)) == code


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=P4), dict(kv_cache=None), dict(kv_cache=P4), dict(page_table=None),
                                dict(seq_lens=None), dict(out=None), dict(out=P4), dict(seqs=ctypes.c_void_p(2)),
                                dict(shared_len=ctypes.c_void_p(2)), dict(lse=ctypes.c_void_p(2)),
                                dict(status=ctypes.c_void_p(2))])
def test_cache_pointers(L, kw):
    assert cache(L, cache_dims(), **kw) == INVALID


def test_cache_scale_behind_fp32(L):
    assert cache(L, cache_dims(scale=2e30)) == DIMS


def test_cache_nothing_to_do(L):
    assert cache(L, None) == INVALID
    assert cache(L, cache_dims(batch=0), q=None, out=None, workspace=None) == 0
    n = ctypes.c_size_t(5)
    assert L.mla_prolog_attend_cache_workspace(None, ctypes.byref(n)) == INVALID
    assert L.mla_prolog_attend_cache_workspace(ctypes.byref(cache_dims()), None) == INVALID
    assert L.mla_prolog_attend_cache_workspace(ctypes.byref(cache_dims(kv_lora_rank=8)), ctypes.byref(n)) == DIMS
    assert n.value == 0


def pool(**kw):
    base = dict(sequences=4, max_pages=8, page_size=16, num_pages=32, page_table=P4, seq_lens=P4, refs=P4, status=P4)
    return binding.MlaPrologPool(*{**base, **kw}.values())


@pytest.mark.parametrize("kw,code", [
    (dict(sequences=-1), DIMS), (dict(max_pages=0), DIMS), (dict(page_size=0), DIMS), (dict(num_pages=-1), DIMS),
    (dict(num_pages=1 << 28), DIMS), (dict(max_pages=1 << 28), DIMS), (dict(page_table=None), INVALID),
    (dict(seq_lens=None), INVALID), (dict(refs=None), INVALID), (dict(status=2), INVALID),
])
def test_pool(L, kw, code):
    p = ctypes.byref(pool(**kw))
    assert L.mla_prolog_pages_extend(p, P4, P4, 2, P4, P4, 8, None) == code
    assert L.mla_prolog_pages_fork(p, P4, P4, 2, P4, P4, None) == code
    assert L.mla_prolog_pages_release(p, P4, 2, None) == code
    assert L.mla_prolog_pages_compact(p, P4, None, None) == code


def test_pool_lists(L):
    p = ctypes.byref(pool())
    for n, code in ((-1, INVALID), (1025, DIMS)):
        assert L.mla_prolog_pages_extend(p, P4, P4, n, P4, P4, 8, None) == code
        assert L.mla_prolog_pages_fork(p, P4, P4, n, P4, P4, None) == code
        assert L.mla_prolog_pages_release(p, P4, n, None) == code
    assert L.mla_prolog_pages_extend(p, None, P4, 1, P4, P4, 8, None) == INVALID
    assert L.mla_prolog_pages_extend(p, P4, P4, 1, P4, P4, -1, None) == INVALID
    assert L.mla_prolog_pages_extend(p, P4, P4, 1, ctypes.c_void_p(2), P4, 1, None) == INVALID
    assert L.mla_prolog_pages_fork(p, P4, P4, 1, None, P4, None) == INVALID
    assert L.mla_prolog_pages_compact(p, None, None, None) == INVALID
    assert L.mla_prolog_pages_extend(p, None, None, 0, None, None, 0, None) == 0
    assert L.mla_prolog_pages_fork(p, None, None, 0, None, None, None) == 0
    assert L.mla_prolog_pages_release(p, None, 0, None) == 0
    assert L.mla_prolog_pages_release(None, P4, 1, None) == INVALID


def test_pool_sizes_whose_sums_pass_32_bits(L):
    p = ctypes.byref(pool(max_pages=1 << 27))   # 2^31 tokens in a sequence
    assert L.mla_prolog_pages_release(p, P4, 1, None) == DIMS
    p = ctypes.byref(pool(max_pages=(1 << 26) + 1))
    assert L.mla_prolog_pages_release(p, P4, 1, None) == DIMS
    p = ctypes.byref(pool())
    assert L.mla_prolog_pages_extend(p, P4, P4, 1, P4, P4, (1 << 30) + 1, None) == DIMS
    assert L.mla_prolog_copy_pages(P16, 1, 0, 10, 32, P4, P4, (1 << 30) + 1, None, None) == DIMS


@pytest.mark.parametrize("kw", [dict(layers=-1), dict(layers=70000), dict(page_bytes=0), dict(page_bytes=24),
                                dict(num_pages=-1), dict(n=-1), dict(cache=None), dict(cache=P4), dict(dst=None),
                                dict(src=ctypes.c_void_p(2)), dict(layer_stride=16), dict(layer_stride=10 * 32 + 8),
                                dict(status=ctypes.c_void_p(2)), dict(num_pages=1 << 62)])
def test_copy_pages(L, kw):
    base = dict(cache=P16, layers=2, layer_stride=320, num_pages=10, page_bytes=32, src=P4, dst=P4, n=3, status=None,
                stream=None)
    assert L.mla_prolog_copy_pages(*{**base, **kw}.values()) == INVALID
    assert L.mla_prolog_copy_pages(*{**base, "n": 0}.values()) == 0


def test_status_bits_and_flags_agree_with_the_header():
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mla_prolog.h")).read()
    for name, value in (("MLA_STATUS_SEQ_RANGE", binding.STATUS_SEQ_RANGE), ("MLA_STATUS_PAGE_RANGE", binding.STATUS_PAGE_RANGE),
                        ("MLA_STATUS_POOL_FULL", binding.STATUS_POOL_FULL), ("MLA_PROMPT_CAUSAL", binding.MLA_PROMPT_CAUSAL),
                        ("MLA_PROMPT_Q_INT8", binding.MLA_PROMPT_Q_INT8),
                        ("MLA_PROMPT_Q_SCALE_PER_HEAD", binding.MLA_PROMPT_Q_SCALE_PER_HEAD)):
        m = re.search(r"#define %s\s+(0x[0-9a-fA-F]+)" % name, src)
        assert m and int(m.group(1), 16) == value, name


def test_binding_refuses_cpu_tensors():
    import torch
    t = torch.zeros((2, 2, 16), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        binding.attend_prompt(t, t, t, t, t, t, scale=1.0)
    with pytest.raises(TypeError):
        binding.attend_cache(t, t, t, t, t, t, t, scale=1.0)
    with pytest.raises(TypeError):
        binding.PagePool(t, t, t, 16)
    with pytest.raises(TypeError):
        binding.copy_pages(t, t, t)
