"""Nothing is written past the rows of dx and dw: rows whose stride is a multiple of 16
bytes but whose end is not lie beside what belongs to somebody else."""
import math

import pytest

torch = pytest.importorskip("torch")

from blockwise_fp8_zero_gb300 import fp8z  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blockwise_fp8_zero_gb300 import build
    build.build()
    fp8z.lib()


@pytest.mark.parametrize("h", [1, 3, 33, 36, 37, 62, 63, 100, 127, 129, 229, 254, 257, 903])
@pytest.mark.parametrize("n,v", [(3, 5), (40, 300), (300, 700)])
@pytest.mark.parametrize("dtype,dw_dtype", [(BF16, F32), (BF16, BF16), (F16, F16)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_row_ends(h, n, v, dtype, dw_dtype, accumulate):
    """The gradient beside a neighbour's columns, equal in every bit to the same gradient in
    tensors of its own, whatever the neighbour's columns hold."""
    g = torch.Generator(device="cuda").manual_seed(h + n)
    x = torch.randn(n, h, generator=g, device="cuda").to(dtype)
    w = (torch.randn(v, h, generator=g, device="cuda") * 2.0 / math.sqrt(h)).to(dtype)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    before = torch.randn(v, h, generator=g, device="cuda").to(dw_dtype)

    def call(dx, dw):
        loss, total = torch.empty(n, device="cuda"), torch.empty(2, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = torch.full((fp8z.fp8z_linear_xent_workspace(x, w, dw=dw),), 255, dtype=torch.uint8, device="cuda")
        fp8z.fp8z_linear_xent_grad(x, w, t, loss, total, dx, dw, ws, accumulate_dw=accumulate, dev_status=status)
        assert status.item() == 0

    dx, dw = torch.empty(n, h, dtype=dtype, device="cuda"), before.clone()
    call(dx, dw)
    for width in {-(-h // 8) * 8, -(-h // 8) * 8 + 8, -(-h // 4) * 4, h + 1}:
        wide_dx = torch.full((n, width), math.nan, dtype=dtype, device="cuda")
        wide_dw = torch.full((v, width), math.nan, dtype=dw_dtype, device="cuda")
        wide_dw[:, :h] = before
        if width > h:
            wide_dw[:, -1] = -3.0
        neighbours = wide_dw[:, h:].clone()
        call(wide_dx[:, :h], wide_dw[:, :h])
        assert torch.equal(wide_dx[:, :h], dx) and torch.equal(wide_dw[:, :h], dw)
        assert bool(wide_dx[:, h:].isnan().all())
        assert torch.equal(wide_dw[:, h:].nan_to_num(nan=7.0), neighbours.nan_to_num(nan=7.0))
