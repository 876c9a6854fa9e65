"""The status word of fp8_linear: calls without rows, and calls that ask for it beside others on their stream."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    import lora_co_serving_gb300 as lm
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lm.build()
    lm.library()


def weight():
    import torch
    import lora_co_serving_gb300 as lm
    return lm.fp8_quantize_weight(torch.randn(256, 512, device="cuda"))


def test_a_call_without_rows_has_no_failure():
    """Whatever the workspace held before: nothing ran that could have failed."""
    import torch
    import lora_co_serving_gb300 as lm
    w = weight()
    x = torch.empty(0, 512, dtype=torch.bfloat16, device="cuda")
    for ws in (torch.full((4096,), 255, dtype=torch.uint8, device="cuda"), None):
        assert lm.fp8_linear(x, *w, workspace=ws, check_status=True).shape == (0, 256)
    codes = torch.empty(0, 512, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    y = lm.fp8_linear(codes, *w, x_scales=torch.empty(0, 4, device="cuda"), check_status=True,
                      workspace=torch.full((4096,), 255, dtype=torch.uint8, device="cuda"))
    assert y.shape == (0, 256)


def test_a_checked_call_reads_a_status_of_its_own():
    """Calls of a stream share a status word that nobody reads; one that is read must not be cleared by another call."""
    import torch
    import lora_co_serving_gb300 as lm
    w, x = weight(), torch.randn(3, 512, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = lm.fp8_linear(x, *w, stream=side)
    kept = lm._status_workspaces[(x.device.index, side.cuda_stream)]
    side.synchronize()
    kept.fill_(255)
    torch.cuda.synchronize()
    y = lm.fp8_linear(x, *w, stream=side, check_status=True)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and bool((kept == 255).all())
