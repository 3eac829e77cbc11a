"""The operators on two streams at once, each with its own tensors and workspace, and while
the other stream keeps the GPU busy: the same bits as one after the other."""
import math

import pytest

torch = pytest.importorskip("torch")

from blockwise_fp8_zero_gb300 import fp8z  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from blockwise_fp8_zero_gb300 import build
    build.build()
    fp8z.lib()


class Step:
    """Lookup, loss with gradients, the lookup's gradient into the same table, clipping."""

    def __init__(self, seed, tokens, vocab, hidden):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        self.targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        self.table = (torch.randn(vocab, hidden, generator=g, device="cuda") * 2 / math.sqrt(hidden)).bfloat16()
        self.x = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda")
        self.dx, self.grad = torch.empty_like(self.x), torch.empty(vocab, hidden, device="cuda")
        self.loss, self.total, self.norm = (torch.empty(n, device="cuda") for n in (tokens, 2, 2))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.xent_ws = torch.empty(fp8z.fp8z_linear_xent_workspace(self.x, self.table, dw=self.grad), dtype=torch.uint8, device="cuda")
        self.embed_ws = torch.empty(fp8z.fp8z_embedding_grad_workspace(tokens, vocab, hidden), dtype=torch.uint8, device="cuda")
        self.norm_ws = torch.zeros(fp8z.fp8z_grad_norm_workspace(), dtype=torch.uint8, device="cuda")
        self.list = fp8z.fp8z_encode_tensor_list([self.grad])

    def run(self):
        fp8z.fp8z_embedding(self.ids, self.table, self.x, scale=2.0, dev_status=self.status)
        fp8z.fp8z_linear_xent_grad(self.x, self.table, self.targets, self.loss, self.total, self.dx, self.grad, self.xent_ws,
                                   dev_status=self.status)
        fp8z.fp8z_embedding_grad(self.ids, self.dx, self.grad, self.embed_ws, scale=2.0, accumulate=True, dev_status=self.status)
        fp8z.fp8z_grad_clip(self.list, 0.1, self.norm, self.norm_ws)

    def outputs(self):
        return [t.clone() for t in (self.x, self.dx, self.grad, self.loss, self.total, self.norm, self.status)]


def test_two_streams_at_once():
    steps = [Step(1, 700, 5000, 256), Step(2, 5000, 3001, 200)]
    want = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        want.append(s.outputs())
        assert s.status.item() == 0
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(10):
        for s in steps:
            for t in (s.x, s.dx, s.grad, s.loss, s.total, s.norm):
                t.fill_(math.nan)
        torch.cuda.synchronize()
        for _ in range(3):
            for s, stream in zip(steps, streams):
                with torch.cuda.stream(stream):
                    s.run()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            assert all(torch.equal(a, b) for a, b in zip(s.outputs(), w))
