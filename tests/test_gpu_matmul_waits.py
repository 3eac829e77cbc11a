"""Products whose waits are made to run out, of every kernel and way of grouping: each says FP8Z_ETIMEOUT, lets its copies and
products land and returns, and the next one has the bits of the one before.

The limit is 1 ns: a wait that finds its barrier incomplete gives up.  Nothing is left unarmed."""
import pytest
import torch

from blockwise_fp8_zero_gb300 import fp8z

from test_gpu_matmul import BF16, F32, codes, gen, scales

pytestmark = pytest.mark.gpu
TRIES = 5


@pytest.mark.parametrize("m,n,k,per_block,dtype,accumulate,cuts", [
    (2048, 2048, 1024, True, BF16, False, None),             # pairs of blocks
    (2048, 2304, 2048, False, F32, True, None),              # a scale for every column, added
    (16, 2048, 4096, True, BF16, False, None),               # few rows, K in parts
    (8, 18432, 1024, True, F32, False, None),                # few rows, K whole
    (64, 2048, 4096, False, F32, True, None),
    (40, 1024, 2048, True, BF16, False, [0, 3, 3, 20, 40]),  # groups of rows
    (4096, 1024, 1024, True, BF16, False, [0, 1000, 1000, 4000, 4096]),
    (512, 1024, 1500, False, F32, False, [0, 384, 1280, 1500, 1500]),    # groups that cut K
    (512, 1024, 2048, False, F32, True, [0, 0, 1024, 1152, 2048]),
])
def test_waits_that_run_out(m, n, k, per_block, dtype, accumulate, cuts):
    g = gen(1)
    kb, nb = -(-k // 128), -(-n // 128)
    bank = len(cuts) - 1 if cuts and per_block else 0
    a, sa = codes(g, m, k), scales(g, m, kb) / 448.0
    b, sb = (codes(g, bank, n, k), scales(g, bank, nb, kb)) if bank else (codes(g, n, k), scales(g, nb if per_block else n, kb))
    start = torch.randn(*((len(cuts) - 1,) if cuts and not bank else ()), m, n, generator=g, device="cuda").to(dtype)
    offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda") if cuts else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(fp8z.fp8z_matmul_workspace(a, b, start, offsets), dtype=torch.uint8, device="cuda")

    def product():
        out = start.clone()
        status.zero_()
        torch.cuda.synchronize()
        fp8z.fp8z_matmul(a, sa, b, sb, out, offsets=offsets, accumulate=accumulate, workspace=ws, dev_status=status)
        torch.cuda.synchronize()
        return out, status.item()
    want, code = product()
    assert code == 0
    gave_up = False
    fp8z.fp8z_set_wait_limit_ns(1)
    try:
        for _ in range(TRIES):
            code = product()[1]
            assert code in (0, fp8z.FP8Z_ETIMEOUT), fp8z.fp8z_status_string(code)
            gave_up |= code == fp8z.FP8Z_ETIMEOUT
    finally:
        fp8z.fp8z_set_wait_limit_ns(0)
    assert gave_up, "no wait ran out"
    got, code = product()
    assert code == 0 and torch.equal(got, want)
