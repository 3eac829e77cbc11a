"""Scales far from 1.  The two scales of a block are multiplied first, in FP32: where that product is a normal
number, results keep test_gpu_matmul's bound; below 2^-126 it is rounded to a multiple of 2^-149, off by half of that
times S, the block's sum of products."""
import pytest
import torch

from blockwise_fp8_zero_gb300 import fp8z

from test_gpu_matmul import BF16, F32, codes, definition, gen, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k", [(5, 300, 640), (60, 520, 1000), (1500, 2304, 384)])
@pytest.mark.parametrize("per_block", [True, False])
@pytest.mark.parametrize("ea,eb", [(120, -130), (-120, 110), (60, 35), (-60, -55), (-70, -60), (-73, -72)])
def test_far_scales(m, n, k, per_block, ea, eb):
    g = gen(m)
    kb = -(-k // 128)
    a, b = codes(g, m, k), codes(g, n, k)
    # 2^ea times 1 to 2: at (60, 35) the results stay below 2^97 * 5 * 2^25
    sa = (1 + torch.rand(m, kb, generator=g, device="cuda")) * 2.0 ** ea
    sb = (1 + torch.rand(-(-n // 128) if per_block else n, kb, generator=g, device="cuda")) * 2.0 ** eb
    for dtype in (F32, BF16):
        out = torch.empty(m, n, dtype=dtype, device="cuda")
        ws = torch.empty(fp8z.fp8z_matmul_workspace(a, b, out), dtype=torch.uint8, device="cuda")
        fp8z.fp8z_matmul(a, sa, b, sb, out, workspace=ws)
        want, size = definition(a, sa, b, sb, per_block)
        # FP32: kb + 35 roundings, each of a unit or of the smallest subnormal number; a half step of the type, or of its smallest one
        bound = (kb + 35) * (2.0 ** -24 * size + 2.0 ** -149)
        if dtype == BF16:
            bound = bound + 2.0 ** -8 * want.abs() * (1 + 1e-3) + 2.0 ** -134
        if ea + eb < -126:
            bound = bound + 2.0 ** -150 * (values(a).abs() @ values(b).abs().t()) * 1.001
        bad = ~((out.double() - want).abs() <= bound)
        assert not bad.any(), (dtype, out[bad][:4], want[bad][:4], int(bad.sum()))
