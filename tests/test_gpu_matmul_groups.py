"""Groups that cut K and are empty behind a ragged end of it: zeros, or an out that stays
as it was, bit for bit.  The groups before them keep test_gpu_matmul's bound."""
import pytest
import torch

from blockwise_fp8_zero_gb300 import fp8z

from test_gpu_matmul import BF16, F32, check, codes, definition, gen, scales

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,accumulate", [(F32, False), (F32, True), (BF16, False)])
@pytest.mark.parametrize("m,n", [(100, 257), (300, 512)])
@pytest.mark.parametrize("cuts", [[500, 500], [0, 384, 500, 500], [0, 500, 500, 500], [500, 500, 500], [0, 200, 200],
                                  [0, 128, 200, 200, 200], [200, 200, 200], [0, 1, 1], [0, 128, 128, 130, 130]])
def test_empty_groups_behind_a_ragged_end(cuts, m, n, dtype, accumulate):
    g = gen(len(cuts) + m)
    e, k = len(cuts) - 1, cuts[-1]
    kb = -(-k // 128)
    a, b = codes(g, m, k), codes(g, n, k)
    sa, sb = scales(g, m, kb) / (448.0 * k ** 0.5), scales(g, n, kb) / 448.0
    start = torch.randn(e, m, n, generator=g, device="cuda").to(dtype)
    for offsets in (torch.tensor(cuts, dtype=t, device="cuda") for t in (torch.int32, torch.int64)):
        out = start.clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = torch.empty(fp8z.fp8z_matmul_workspace(a, b, out, offsets), dtype=torch.uint8, device="cuda")
        fp8z.fp8z_matmul(a, sa, b, sb, out, offsets=offsets, accumulate=accumulate, workspace=ws, dev_status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        for i, (c0, c1) in enumerate(zip(cuts, cuts[1:])):
            if c0 == c1:
                assert torch.equal(out[i], start[i] if accumulate else torch.zeros_like(start[i])), i
            else:
                s = slice(c0 // 128, -(-c1 // 128))
                want, size = definition(a[:, c0:c1], sa[:, s], b[:, c0:c1], sb[:, s], False)
                check(out[i], want, size, c1 - c0, start[i] if accumulate else None)
