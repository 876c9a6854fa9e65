"""Arguments of the attention side's calls that would give a wrong answer without an error (no GPU is touched)."""
import math

import pytest

import lora_co_serving_gb300 as lm
from test_attention_refusals import FAKE, cache, e4m3, error, lib  # noqa: F401  (lib: a fixture)


def decode(lib, B=2, heads=8, q=FAKE, ld_q=512, c=None, width=4, window=0, scale=0.1, softcap=0.0, out=2 * FAKE, ld_out=512):
    """A call that is refused for its workspace at the latest."""
    return error(lib, lib.lora_decode_attention(B, heads, q, ld_q, cache() if c is None else c, FAKE, width, width, FAKE, window,
                                                scale, softcap, out, ld_out, None, None, 0, None))


@pytest.mark.parametrize("c", [cache(), e4m3()], ids=["bf16", "e4m3"])
def test_decode_in_place_has_one_row_distance(lib, c):
    rc, msg = decode(lib, c=c, out=FAKE, ld_out=520)
    assert lm.ERRORS[rc] == "LORA_ERR_INVALID_ARG" and "in place, ld_out must be ld_q" in msg
    for kw in (dict(out=FAKE), dict(out=FAKE, ld_out=520, B=1), dict(ld_out=520)):
        rc, msg = decode(lib, c=c, **kw)
        assert "in place" not in msg
