"""What the header says of limits and norms that are not finite, and of squares that FP32 does not hold."""
import math

import pytest

torch = pytest.importorskip("torch")

from blockwise_fp8_zero_gb300 import fp8z  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blockwise_fp8_zero_gb300 import build
    build.build()
    return torch.zeros(fp8z.fp8z_grad_norm_workspace(), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_an_infinite_limit_never_clips(ws, bad):
    t = torch.arange(1.0, 101.0, device="cuda")
    t[3] = bad
    before, norm = t.clone(), torch.zeros(2, device="cuda")
    fp8z.fp8z_grad_clip(fp8z.fp8z_encode_tensor_list([t]), math.inf, norm, ws)
    assert norm[1].item() == 1.0 and not math.isfinite(norm[0].item())
    assert torch.equal(t.nan_to_num(nan=-7.0), before.nan_to_num(nan=-7.0))


@pytest.mark.parametrize("size,bits", [(1e-18, 20), (2e19, None), (1e-24, None)])
def test_squares_are_fp32(ws, size, bits):
    t = torch.full((5000,), size, device="cuda")
    norm = torch.zeros(2, device="cuda")
    fp8z.fp8z_grad_norm(fp8z.fp8z_encode_tensor_list([t]), norm, ws)
    want = float(t.double().norm())
    if bits:
        assert abs(norm[0].item() - want) <= 2.0 ** -bits * want
    else:
        assert norm[0].item() == (math.inf if size > 1 else 0.0)
