"""The operators of a layer with FP8 weights together, as they are used: a training block of
them, captured and replayed, on two streams, past 2^31 elements, with offsets that break
their rules and with waits that run out."""
import importlib.util
import os

import pytest
import torch

from blockwise_fp8_zero_gb300 import fp8z

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("fp8_layer", os.path.join(ROOT, "examples", "fp8_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def values(q, s):
    return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)[:, :q.shape[1]]


def weight64(block, i):
    q, s = block.weight(i)
    return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


def test_example_runs(example):
    losses = example.train(steps=5)
    assert len(losses) == 5 and all(map(torch.isfinite, map(torch.tensor, losses)))


def test_example_gradients(example):
    """Each product of the block against 64 bits of the codes it was given: FP32 sums of at most 512 products,
    35 + 4 roundings (2^-24) of the sum of absolute values each."""
    b = example.Block(tokens=256)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(256, b.hidden, generator=g, device="cuda")
    dy = torch.randn(256, b.hidden, generator=g, device="cuda") * 1e-2
    y, (n, h, a) = b.forward(x)
    dx = b.backward(x, dy, (n, h, a))
    u = 40 * 2.0 ** -24
    w1, w2, nv, av = weight64(b, 0), weight64(b, 1), values(*n), values(*a)

    def near(got, p, q, extra=0.0):
        size = p.abs() @ q.abs()
        assert ((got.double() - p @ q).abs() <= u * size + extra).all()
    near(h, nv, w1.t())
    near(y - x, av, w2.t(), 2.0 ** -23 * (x.abs() + y.abs()).double())
    gq = b.quantize(dy)
    dh = b.product(gq, b.weight(1, True), b.inner)
    near(dh, values(*gq), w2)
    ghq = b.quantize(dh * (h > 0))
    near(b.grads[1], values(*b.columns(gq)), values(*b.columns(a)).t())
    near(b.grads[0], values(*b.columns(ghq)), values(*b.columns(n)).t())
    # the column-major copy is the transpose of the weights
    q, s = b.weight(0, True)
    qr, sr = b.weight(0)
    assert torch.equal(q, qr.t()) and torch.equal(s, sr.t())
    # the norm's gradient of dn
    dn = (values(*ghq) @ w1)
    xh = (x.double() - b.mean.double()[:, None]) * b.rstd.double()[:, None]
    gw = dn * b.vectors[0].double()
    want = b.rstd.double()[:, None] * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True)) + dy.double()
    scale = (values(*ghq).abs() @ w1.abs()).max(1, keepdim=True).values * b.rstd.double()[:, None] * 10
    assert ((dx.double() - want).abs() <= u * scale * (1 + xh.abs()) + 2.0 ** -23 * want.abs()).all()
    assert int(b.status.item()) == 0


def test_step_captured_and_replayed(example):
    """A captured step replayed gives what eager steps give, bit for bit; a second graph with buffers of its own beside it."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(512, 256, generator=g, device="cuda")
    t = torch.relu(x)
    hp = fp8z.hparams(lr=1e-3, step=3)
    eager, one, two = (example.Block() for _ in range(3))
    for b in (eager, one, two):
        b.step(x, t, hp)                                       # once eagerly, in each
    torch.cuda.synchronize()
    graphs = []
    for b in (one, two):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            loss = b.step(x, t, hp)
        graphs.append((graph, loss))
    for _ in range(3):
        want = eager.step(x, t, hp)
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for b, (_, loss) in zip((one, two), graphs):
        assert torch.equal(loss, want)
        for k in ("p", "m", "v", "w_row", "w_col", "inv"):
            assert torch.equal(getattr(b, k), getattr(eager, k)), k
        assert all(torch.equal(p, q) for p, q in zip(b.vectors, eager.vectors))


def test_two_streams_at_once(example):
    """Two blocks on two streams, interleaved, give what each gives alone."""
    g = torch.Generator(device="cuda").manual_seed(6)
    xs = [torch.randn(512, 256, generator=g, device="cuda") for _ in range(2)]
    hp = fp8z.hparams(lr=1e-3, step=2)
    alone = []
    for i in range(2):
        b = example.Block(seed=i)
        for _ in range(4):
            b.step(xs[i], xs[i].flip(1), hp)
        alone.append((b.p.clone(), b.vectors[0].clone()))
    blocks, streams = [example.Block(seed=i) for i in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                blocks[i].step(xs[i], xs[i].flip(1), hp)
    torch.cuda.synchronize()
    for b, (p, v) in zip(blocks, alone):
        assert torch.equal(b.p, p) and torch.equal(b.vectors[0], v)


def codes(g, *shape):
    q = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.int32)
    return torch.where((q & 127) == 127, q - 1, q).to(torch.uint8)


@pytest.mark.parametrize("by_k", [False, True])
@pytest.mark.parametrize("bad", [[0, 200, 100, 256], [0, 128, 256, 384], [-1, 0, 128, 256], [0, 1, 128, 256]])
def test_offsets_that_break_their_rules(by_k, bad):
    """Falling, past the end, negative; where they cut K also between blocks: reported, and nothing is written."""
    if not by_k and bad == [0, 1, 128, 256]:
        bad = [300, 300, 300, 300]
    g = torch.Generator(device="cuda").manual_seed(1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    off = torch.tensor(bad, dtype=torch.int64, device="cuda")
    if by_k:
        a, b, out = codes(g, 64, 256), codes(g, 96, 256), torch.full((3, 64, 96), 7.0, device="cuda")
        sa, sb = torch.ones(64, 2, device="cuda"), torch.ones(96, 2, device="cuda")
    else:
        a, b, out = codes(g, 256, 128), codes(g, 3, 96, 128), torch.full((256, 96), 7.0, device="cuda")
        sa, sb = torch.ones(256, 1, device="cuda"), torch.ones(3, 1, 1, device="cuda")
    fp8z.fp8z_matmul(a, sa, b, sb, out, offsets=off, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == fp8z.FP8Z_EINVAL and (out == 7.0).all()


def test_nan_codes_and_scales_reach_their_results_only():
    g = torch.Generator(device="cuda").manual_seed(2)
    for m, n in ((20, 300), (600, 700)):
        a, b = codes(g, m, 384), codes(g, n, 384)
        sa, sb = torch.ones(m, 3, device="cuda"), torch.ones(-(-n // 128), 3, device="cuda")
        a[3, 200], b[5, 7], sa[9, 2], sb[1, 1] = 0x7F, 0xFF, float("nan"), float("inf")
        out = torch.empty(m, n, device="cuda")
        fp8z.fp8z_matmul(a, sa, b, sb, out)
        bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        bad[3], bad[9], bad[:, 5], bad[:, 128:256] = True, True, True, True
        assert out[~bad].isfinite().all() and not out[3].isfinite().any() and not out[9].isfinite().any()
        assert out[:, 5].isnan().all() and not out[:, 128:256].isfinite().any()


def test_past_2_31_elements():
    """70000 x 40000 results, 2.8e9 of them: sampled rows against 64 bits (35 + 1 roundings of the sum of absolute values and
    half a step of BF16)."""
    g = torch.Generator(device="cuda").manual_seed(4)
    m, n, k = 70000, 40000, 128
    a, b = codes(g, m, k), codes(g, n, k)
    sa, sb = torch.rand(m, 1, generator=g, device="cuda") + 0.5, torch.rand(-(-n // 128), 1, generator=g, device="cuda") + 0.5
    out = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    fp8z.fp8z_matmul(a, sa, b, sb, out)
    w = b.view(torch.float8_e4m3fn).double() * sb.double().repeat_interleave(128, 0)[:n]
    for r in (0, 255, 53687, 53688, 69632, m - 1):
        x = a[r].view(torch.float8_e4m3fn).double() * sa[r].double()
        want, size = w @ x, w.abs() @ x.abs()
        assert ((out[r].double() - want).abs() <= 36 * 2.0 ** -24 * size + 2.0 ** -8 * want.abs()).all(), r


def test_waits_that_run_out():
    """With a limit of 1 ns a product may give up: it says so, returns, and the next one is right."""
    g = torch.Generator(device="cuda").manual_seed(7)
    shapes = [(16, 2048, 4096), (2048, 2048, 1024)]
    for m, n, k in shapes:
        a, b = codes(g, m, k), codes(g, n, k)
        sa, sb = torch.ones(m, k // 128, device="cuda"), torch.ones(n // 128, k // 128, device="cuda")
        out, again = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        fp8z.fp8z_matmul(a, sa, b, sb, out, dev_status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        fp8z.fp8z_set_wait_limit_ns(1)
        try:
            fp8z.fp8z_matmul(a, sa, b, sb, again, dev_status=status)
            torch.cuda.synchronize()
        finally:
            fp8z.fp8z_set_wait_limit_ns(0)
        assert status.item() in (fp8z.FP8Z_ETIMEOUT, 0)
        status.zero_()
        fp8z.fp8z_matmul(a, sa, b, sb, again, dev_status=status)
        torch.cuda.synchronize()
        assert status.item() == 0 and torch.equal(out, again)


def test_lists_of_the_other_kind_are_refused():
    t = torch.zeros(8, device="cuda")
    norms = fp8z.fp8z_encode_tensor_list([t])
    steps = fp8z.fp8z_encode_adamw_list([t], [t.clone()], [t.clone()], [t.clone()])
    ws = torch.zeros(fp8z.fp8z_grad_norm_workspace(), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        fp8z.fp8z_adamw(norms, fp8z.hparams())
    with pytest.raises(ValueError):
        fp8z.fp8z_grad_norm(steps, torch.zeros(2, device="cuda"), ws)


def test_binding_refusals():
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device="cuda")
    u8 = torch.uint8
    a, b, sa, sb, out = z(4, 256, d=u8), z(200, 256, d=u8), z(4, 2), z(2, 2), z(4, 200)
    for args, kw in (((a.float(), sa, b, sb, out), {}), ((a, sa, b[:, :128], sb, out), {}), ((a, sa.double(), b, sb, out), {}),
                     ((a, sa[:, :1], b, sb, out), {}), ((a, sa, b, sb[:1], out), {}), ((a, sa, b, sb, out.long()), {}),
                     ((a.t().contiguous().t(), sa, b, sb, out), {}), ((a, sa, b, sb, out), dict(offsets=z(2, d=torch.int32))),
                     ((a, sa, b[None], sb[None], out), {}), ((a, sa, b[None], sb[None], out), dict(offsets=z(3, d=torch.int32))),
                     ((a, sa, b[None], z(1, 200, 2), out), dict(offsets=z(2, d=torch.int32))), ((a.cpu(), sa, b, sb, out), {})):
        with pytest.raises(ValueError):
            fp8z.fp8z_matmul(*args, **kw)
    with pytest.raises(fp8z.Fp8zError):
        fp8z.fp8z_matmul(a, sa, b, sb, out.bfloat16(), accumulate=True)
    x, w = z(4, 256), z(256)
    for call in (lambda: fp8z.fp8z_layer_norm(x, w[:5], None, x, None, None), lambda: fp8z.fp8z_layer_norm(x, w.half(), None, x, None, None),
                 lambda: fp8z.fp8z_layer_norm(x, w, w.half(), x, None, None), lambda: fp8z.fp8z_layer_norm(x, w, None, x.half(), None, None),
                 lambda: fp8z.fp8z_layer_norm(x, w, None, None, None, None, q=z(4, 256, d=u8)),
                 lambda: fp8z.fp8z_layer_norm(x, w, None, None, z(3), None),
                 lambda: fp8z.fp8z_encode_adamw_list([w], [w[:5]], [w], [w]), lambda: fp8z.fp8z_encode_adamw_list([w], [w], [z(256, d=u8)], [z(256, d=u8)]),
                 lambda: fp8z.fp8z_encode_adamw_list([w.half()], [w], [w], [w])):
        with pytest.raises(ValueError):
            call()


def test_one_group_of_columns_has_no_group_stride():
    """Through the C ABI: out_group of a single group is not used, 0 among its values."""
    import ctypes
    g = torch.Generator(device="cuda").manual_seed(8)
    m, n, k = 300, 520, 640
    a, b = codes(g, m, k), codes(g, n, k)
    sa, sb = torch.ones(m, 5, device="cuda"), torch.ones(n, 5, device="cuda")
    off = torch.tensor([0, k], dtype=torch.int32, device="cuda")
    want, out = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
    fp8z.fp8z_matmul(a, sa, b, sb, want[None], offsets=off)
    for step in (0, 3, -16, 2 ** 50):
        out.zero_()
        args = fp8z.fp8z_matmul_args(m=m, n=n, k=k, a_ld=k, b_ld=k, out_ld=n, a_scale_ld=5, b_scale_ld=5, out_group=step, b_scale_rows=1,
                                     out_dtype=fp8z.FP8Z_F32, groups=1, group_by=fp8z.FP8Z_GROUP_K, offsets_dtype=fp8z.FP8Z_I32)
        rc = fp8z.lib().fp8z_matmul(a.data_ptr(), sa.data_ptr(), b.data_ptr(), sb.data_ptr(), ctypes.byref(args), off.data_ptr(),
                                    out.data_ptr(), None, 0, None, torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and torch.equal(out, want), step


def test_adamw_list_refuses_what_overlaps():
    """The same parameter twice, moments that share memory, a copy inside a parameter: a step would race."""
    z = lambda n=300, d=torch.float32: torch.zeros(n, dtype=d, device="cuda")
    p, q, buf = z(), z(), z(600)
    for args, kw in ((([p, p], [z(), z()], [z(), z()], [z(), z()]), {}), (([p], [z()], [q], [q]), {}),
                     (([p], [z()], [buf[:300]], [buf[299:599]]), {}), (([p], [z()], [z()], [p]), {}),
                     (([p, q], [z(), z()], [z(), z()], [z(), z()]), dict(copies=[buf.bfloat16()[:300], q.view(torch.bfloat16)[300:]])),
                     (([p], [z()], [z(d=torch.uint8)], [z(d=torch.uint8)]), dict(exp_avg_scales=[buf[:3]], exp_avg_sq_scales=[buf[2:5]]))):
        with pytest.raises(ValueError):
            fp8z.fp8z_encode_adamw_list(*args, **kw)
    # neighbours, empty tensors and shared gradients are fine
    assert fp8z.fp8z_encode_adamw_list([buf[:300], buf[300:], z(0)], [p, p, z(0)], [z(), z(), z(0)], [z(), z(), z(0)]).chunks == 2
    assert fp8z.fp8z_encode_adamw_list([], [], [], []).chunks == 0
