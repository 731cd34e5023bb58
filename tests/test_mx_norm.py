"""The norm's factor: of a token alone, and the same whatever comes with it."""

import pytest
import torch

import mixture_experts_ffn_infer_gb300 as mx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,n", [(7168, 20000), (1024, 20000), (4128, 8000), (16384, 4000)])
def test_a_token_does_not_depend_on_the_batch(d, n):
    # Up to 304 rows a thread holds one piece of a row, beyond that two (wide rows four, narrow ones a warp's share).
    # bf16 rows: the format in which a last bit of the factor shows most often.
    g = torch.Generator("cuda").manual_seed(d)
    x, r = (torch.randn(n, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    gain = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
    rows, total = mx.mx_add_rmsnorm(x, r, gain, 1e-6, mx.MOE_MX_BF16)
    for a in range(0, n, 304):
        few, part = mx.mx_add_rmsnorm(x[a:a + 304], r[a:a + 304], gain, 1e-6, mx.MOE_MX_BF16)
        assert torch.equal(few.codes, rows.codes[a:a + 304]) and torch.equal(part, total[a:a + 304])
    one, _ = mx.mx_add_rmsnorm(x[:1], r[:1], gain, 1e-6, mx.MOE_MX_BF16)
    assert torch.equal(one.codes, rows.codes[:1])
