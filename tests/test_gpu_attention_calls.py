"""Decode attention called as its documentation allows and as few programs do; against float64, or bit by bit against the same
call in its usual form.  Tolerances: test_gpu_decode.py's."""
import pytest
import torch

import lora_co_serving_gb300 as lm
from test_gpu_decode import Case

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16

# sequences that several CTAs share: joined in one stage; in two; a group of 71 heads, taken in five parts
SPLIT = [([600, 3, 900, 0, 2000], 8, 2, 128), ([20000], 8, 2, 128), ([9000, 1], 71, 1, 64), ([12000], 10, 2, 256),
         ([5000, 800], 32, 2, 128)]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("lengths,hq,hkv,D", SPLIT)
def test_in_place_over_several_ctas(lengths, hq, hkv, D, e4m3):
    """The result in the queries' own rows, where other CTAs still read the queries of the same and of other heads."""
    c = Case(lengths, hq, hkv, D, page=64, e4m3=e4m3)
    q, table, n = c.dev
    ref, lse = c.run()
    c.check(ref, lse)
    wide = torch.full((len(lengths), hq * D + 64), 5.0, dtype=bf16, device="cuda")
    for _ in range(3):
        wide[:, :hq * D] = q
        got, z = lm.decode_attention(wide[:, :hq * D], c.cache, table, n, want_lse=True, out=wide[:, :hq * D])
        assert torch.equal(got, ref) and torch.equal(z, lse) and (wide[:, hq * D:] == 5).all()
