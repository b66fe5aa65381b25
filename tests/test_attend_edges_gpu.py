"""Attention operators on the GPU: calls at the edges of their contracts.
Tolerances as derived in test_attend_gpu.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu

from mla_attention_prolog_gb300 import binding  # noqa: E402
from test_attend_gpu import cache_case, prompt_case, run_cache, run_prompt  # noqa: E402


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
