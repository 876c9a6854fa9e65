"""Rotary positions and norms of rows at the ends of the numbers' range."""
import pytest
import torch

import lora_co_serving_gb300 as lm
from test_gpu_rotary import BF, F32, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("rot", [64, 32, 0])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_rows_whose_products_with_the_weight_overflow(dtype, rot, interleaved):
    """Such a row's squares are past float32's range as well: it counts as infinitely long, and gives zeros.  An infinite or
    NaN element still gives NaN at its own place and its partner's."""
    x = torch.randn(5, 3 * 64, generator=gen(1)).to(dtype).cuda()
    x[0, :64], x[1, 70], x[2, 3], x[3, 130], x[4, 128:] = 2e38, 3e38, float("inf"), float("nan"), -3e38
    w = torch.full((64,), 4.0, dtype=dtype, device="cuda")
    turns = lm.rotary_turns(rot) if rot else None
    p = torch.arange(5).cuda() if rot else None
    out = lm.rotary_forward(x, p, turns, 2, 1, q_weight=w, k_weight=w, interleaved=interleaved).reshape(5, 3, 64)
    assert (out[0, 0] == 0).all() and (out[1, 1] == 0).all() and (out[4, 2] == 0).all()
    hit = torch.zeros(5, 3, dtype=torch.bool)
    hit[2, 0] = hit[3, 2] = True
    assert torch.equal(out.isfinite().all(-1).cpu(), ~hit)
    assert out[2, 0].isnan().sum() == (2 if rot else 1) and out[3, 2].isnan().all()
    cache = lm.kv_cache(1, 1, 8, 64, torch.float8_e4m3fn)
    slots = torch.arange(5).cuda()
    lm.rotary_forward(x, p, turns, 2, 1, q_weight=w, k_weight=w, interleaved=interleaved, v=x[:, :64], cache=cache, slots=slots)
    k, _ = lm.cache_read(cache, slots)
    assert (k[4] == 0).all() and k[3].isnan().all() and k[:3].isfinite().all()
