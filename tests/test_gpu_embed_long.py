"""The embedding gradient over lists that one block of the sort takes several tiles of,
and runs of one word over thousands of pieces, against 64 bits: FP32 sums of L terms
within (L + 3) * 2^-24 of the sum of their absolute values, the result's own rounding
on top; where the terms are whole numbers, exactly."""
import pytest

torch = pytest.importorskip("torch")

from blockwise_fp8_zero_gb300 import fp8z  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blockwise_fp8_zero_gb300 import build
    build.build()
    fp8z.lib()


def _grad(ids, d, vocab, **kw):
    n, h = d.shape
    table = torch.full((vocab, h), 7.0, device="cuda")
    ws = torch.full((fp8z.fp8z_embedding_grad_workspace(n, vocab, h),), 255, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp8z.fp8z_embedding_grad(ids, d, table, ws, dev_status=status, **kw)
    assert status.item() == 0
    return table


@pytest.mark.parametrize("tokens", [524288, 524289, 1000003, (1 << 21) + 5])
@pytest.mark.parametrize("vocab", [1, 1000, 70000, 1 << 21])
def test_order_of_a_long_list(tokens, vocab):
    """Whole numbers below 2^24 in every sum: equal, whatever their order, if every token is
    counted once and in its word."""
    g = torch.Generator(device="cuda").manual_seed(tokens + vocab)
    ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    d = torch.randint(-4, 5, (tokens, 8), generator=g, device="cuda").to(torch.bfloat16)
    want = torch.zeros(vocab, 8, dtype=torch.float64, device="cuda").index_add_(0, ids, d.double())
    assert torch.equal(_grad(ids, d, vocab).double(), want)
    # padding and 32-bit ids
    want[0] = 0.0
    assert torch.equal(_grad(ids.int(), d, vocab, padding_idx=0).double(), want)


def test_equal_words_keep_the_list_s_order():
    """FP32 terms of many sizes: sums of the same terms in the order of the tokens, so that
    equal words spread in two ways over a list come out in the same bits."""
    n, vocab = 600000, 5
    g = torch.Generator(device="cuda").manual_seed(3)
    d = torch.randn(n, 8, generator=g, device="cuda") * torch.exp(4 * torch.randn(n, 1, generator=g, device="cuda"))
    ids = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    order = torch.argsort(ids, stable=True)
    assert torch.equal(_grad(ids, d, vocab), _grad(ids[order], d[order], vocab))


@pytest.mark.parametrize("tokens", [262144 + 7, (1 << 21) + 5])
@pytest.mark.parametrize("words", [1, 2, 3, 40])
def test_runs_over_thousands_of_pieces(tokens, words):
    """Whole numbers again, a few words for the whole list, among 1000."""
    g = torch.Generator(device="cuda").manual_seed(tokens + words)
    ids = torch.randint(0, words, (tokens,), generator=g, device="cuda") * 17 + 3
    d = torch.randint(-4, 5, (tokens, 24), generator=g, device="cuda").to(torch.bfloat16)
    want = torch.zeros(1000, 24, dtype=torch.float64, device="cuda").index_add_(0, ids, d.double())
    assert torch.equal(_grad(ids, d, 1000).double(), want)
    # all but a few tokens one word, the others around it
    ids = torch.full((tokens,), 500, device="cuda")
    ids[::100003] = 499
    ids[1::100003] = 501
    want = torch.zeros(1000, 24, dtype=torch.float64, device="cuda").index_add_(0, ids, d.double())
    assert torch.equal(_grad(ids, d, 1000).double(), want)
