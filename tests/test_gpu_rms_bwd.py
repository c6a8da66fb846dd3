"""The gradient of the row RMSNorm (rms_norm_backward) on the GPU against the
formula and against differences in 64 bits: row lengths from 1 to beyond what
a block holds, row counts from 0, types, unaligned tensors, extreme values,
aliasing, streams and captured graphs, and a training step of the norms.

Bounds (roundings on the longest path): the row's two sums add at most hidden / 256
values a thread and 10 more; xh has 30, a product 4: K = 128 + hidden / 256 for
dx.  dw adds at most rows / 32 terms of 40 in order and 60 partial sums:
K = 128 + rows / 32."""
import pytest

import rmsnorm_fwd_gb300 as rn

import _rope as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rn.ensure_context(0)
    rn.rmsnorm_get_device_status()
    yield
    torch.cuda.synchronize()
    assert rn.rmsnorm_get_device_status() == rn.OK


def make(dtype, rows, hidden, seed, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = R.DT[dtype]

    def at(shape, scale):
        n = 1
        for s in shape:
            n *= s
        t = torch.empty(n + shift, dtype=dt, device="cuda")[shift:].view(shape)
        return t.copy_(R.rand(g, shape, dt, scale))

    x, dy = at((rows, hidden), 1.5), at((rows, hidden), 0.1)
    return dy, x, at((hidden,), 0.1).add_(1), g


def check(dy, x, w, bias, eps, dx, dw):
    rows, hidden = x.shape
    ref = R.norm_bwd(dy.double(), dy.double().abs(), x, w, bias, eps, 0)
    R.assert_close(dx, ref[0], ref[1], 128 + hidden / 256, "dx")
    if dw is not None:
        assert dw.dtype == torch.float32
        R.assert_close(dw, ref[2], ref[3], 128 + rows / 32, "dw")


SHAPES = [(1, 1), (3, 1), (5, 2), (1, 7), (64, 64), (17, 72), (129, 128), (33, 100), (40, 257),
          (509, 1024), (200, 1000), (77, 2048), (31, 2880), (100, 4096), (3, 4096), (26, 5120),
          (15, 7168), (9, 8192), (21, 8200), (11, 16384), (7, 20000), (4, 32768), (2, 65536),
          (3, 100001), (2500, 96), (700, 255), (700, 331), (9, 9001), (8, 15495), (600, 202), (1200, 640), (4001, 1024),
          (1, 4096), (2, 300000), (1219, 1003), (3001, 247), (2001, 249), (5000, 33), (2000, 1026),
          (610, 4067), (305, 5113), (310, 8177), (160, 8179), (7, 8191), (170, 16369), (160, 16371),
          (154, 16383), (12001, 576), (11000, 723), (10003, 768), (10003, 755)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,hidden", SHAPES)
def test_gradient(rows, hidden, dtype):
    bias = 1.0 if rows % 2 else -0.0
    dy, x, w, _ = make(dtype, rows, hidden, 1)
    kept = dy.clone(), x.clone()
    dx, dw = rn.rms_norm_backward(dy, x, w, 1e-6, bias)
    assert torch.equal(dy, kept[0]) and torch.equal(x, kept[1])
    check(dy, x, w, bias, 1e-6, dx, dw)
    again = rn.rms_norm_backward(dy, x, w, 1e-6, bias)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    # dx alone; over dy; over x
    alone, none = rn.rms_norm_backward(dy, x, w, 1e-6, bias, weight_grad=False)
    assert none is None and torch.equal(alone, dx)
    a = dy.clone()
    out = rn.rms_norm_backward(a, x, w, 1e-6, bias, dx=a)
    assert out[0] is a and torch.equal(a, dx) and torch.equal(out[1], dw)
    b = x.clone()
    out = rn.rms_norm_backward(dy, b, w, 1e-6, bias, dx=b)
    assert torch.equal(b, dx) and torch.equal(out[1], dw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,hidden", [(20, 1024), (9, 4096), (5, 16384), (3, 30000)])
def test_unaligned_tensors(rows, hidden, dtype):
    dy, x, w, _ = make(dtype, rows, hidden, 2, shift=1)
    check(dy, x, w, 0.0, 1e-6, *rn.rms_norm_backward(dy, x, w, 1e-6, 0.0))


@pytest.mark.parametrize("rows,hidden", [(3000, 331), (2000, 1026), (1500, 4067), (400, 12289)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_between_vector_boundaries_keep_to_themselves(dtype, rows, hidden):
    """Rows that share vectors with their neighbours, every other one of NaN, and what lies
    behind the last."""
    dt = R.DT[dtype]
    dy, x, w, g = make(dtype, rows, hidden, 8)
    x[1::2], dy[1::2] = float("nan"), float("inf")
    room = torch.full((rows * hidden + 64,), 7.0, dtype=dt, device="cuda")
    dx = room[:rows * hidden].view(rows, hidden)
    rn.rms_norm_backward(dy, x, w, 1e-6, 0.0, dx=dx)
    assert (room[rows * hidden:] == 7).all() and dx[1::2].isnan().all()
    good = dy[::2].contiguous(), x[::2].contiguous()
    _, dw = rn.rms_norm_backward(*good, w, 1e-6, 0.0)
    check(*good, w, 0.0, 1e-6, dx[::2], dw)
    for over in (x.clone(), dy.clone()):
        a, b = (dy, over) if over[1, 0].isnan() else (over, x)
        rn.rms_norm_backward(a, b, w, 1e-6, 0.0, dx=over, weight_grad=False)
        assert torch.equal(over[::2], dx[::2])


@pytest.mark.parametrize("rows,hidden", [(16384, 1024), (5000, 4096), (30000, 72)])
def test_many_rows(rows, hidden):
    dy, x, w, _ = make("bf16", rows, hidden, 3)
    dx, dw = rn.rms_norm_backward(dy, x, w, 1e-5)
    check(dy, x, w, 0.0, 1e-5, dx, dw)
    assert torch.equal(rn.rms_norm_backward(dy, x, w, 1e-5)[1], dw)


@pytest.mark.parametrize("hidden", [100, 128, 131, 1024, 1027, 4096, 5000, 5120, 16384, 40000])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_extreme_rows(dtype, hidden):
    dy, x, w, _ = make(dtype, 20, hidden, 4)
    dt = R.DT[dtype]
    big, small = ((2.0 ** 100, 2.0 ** -110) if dtype != "f16" else (2.0 ** 11, 2.0 ** -14))
    scale = torch.ones(20, 1, dtype=torch.float64, device="cuda")
    scale[1], scale[2], scale[3], scale[4] = big, small, 0.0, big * 2.0 ** 3
    if dtype != "f16":
        for i, e in enumerate((38, 43, 60, -28, -33, -45, -52, -58, -75)):
            scale[10 + i] = 2.0 ** e
    x = (x.double() * scale).to(dt)
    x[5, 3], x[6, hidden - 1] = float("inf"), float("nan")
    x[7] = torch.finfo(dt).smallest_normal / 4
    for eps in (1e-6, 0.0, 1e-30, 1e-14):
        dx, dw = rn.rms_norm_backward(dy, x, w, eps)
        check(dy, x, w, 0.0, eps, dx, None)
        ref = R.norm_bwd(dy.double(), dy.double().abs(), x, w, 0.0, eps, 0)
        assert torch.equal(dw.isnan(), ref[2].isnan())
    # without the rows that are not numbers, every column's sum
    keep = torch.tensor([0, 1, 2, 4] + list(range(7, 20)), device="cuda")
    dy, x = dy[keep].contiguous(), x[keep].contiguous()
    check(dy, x, w, 0.0, 0.0, *rn.rms_norm_backward(dy, x, w, 0.0))


def test_first_call_of_a_shape_inside_a_capture():
    """What a body looks up at its first launch is looked up in a capture, too."""
    dy, x, w, _ = make("f16", 40, 6136, 12)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, dw = rn.rms_norm_backward(dy, x, w, 1e-6)
    graph.replay()
    torch.cuda.synchronize()
    check(dy, x, w, 0.0, 1e-6, dx, dw)


def test_refusals_of_the_workspace():
    dy, x, w, _ = make("bf16", 8, 4096, 13)
    dx, dw = torch.empty_like(x), torch.empty(4096, device="cuda")
    need = rn.rmsnorm_bwd_workspace(8, 4096, rn.BF16, rn.rmsnorm_device_limits()[0])
    ws = torch.empty(need + 64, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream

    def status(ws_at, n, dw_at=dw.data_ptr()):
        try:
            rn.rmsnorm_bwd(dy.data_ptr(), x.data_ptr(), w.data_ptr(), dx.data_ptr(), dw_at, ws_at, n,
                           8, 4096, 0.0, 1e-6, rn.BF16, s)
        except rn.RmsnormError as e:
            return e.status
        return rn.OK

    p = ws.data_ptr()
    assert status(p, need) == rn.OK and status(p + 16, need) == rn.OK
    assert status(p, need - 1) == rn.ERR_INVALID_ARG and status(0, need) == rn.ERR_INVALID_ARG
    assert status(p + 8, need) == rn.ERR_MISALIGNED
    assert status(dx.data_ptr(), need) == rn.ERR_ALIASING
    assert status(p, need, p + 64) == rn.ERR_ALIASING
    assert status(p, need, w.data_ptr()) == rn.ERR_ALIASING


def test_no_rows():
    w = torch.ones(4096, device="cuda", dtype=torch.bfloat16)
    e = torch.empty(0, 4096, device="cuda", dtype=torch.bfloat16)
    dx, dw = rn.rms_norm_backward(e, e, w, 1e-6)
    assert dx.shape == e.shape and not dw.any()


def test_against_differences():
    """<dx, a> + <dw, b> against the central difference of <dy, y> in 64 bits."""
    dy, x, w, g = make("f32", 7, 200, 5)
    dx, dw = rn.rms_norm_backward(dy, x, w, 1e-6, 1.0)
    a = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
    b = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64)

    def f(h):
        xx = x.double() + h * a
        return (dy.double() * xx * R.factor(xx, 1e-6) * (w.double() + h * b + 1.0)).sum()

    h = 1e-4
    want = ((f(h) - f(-h)) / (2 * h)).item()
    got = ((dx.double() * a).sum() + (dw.double() * b).sum()).item()
    assert abs(got - want) <= 1400 * 128 * R.U + 1e-5  # 1400 fp32 terms of order 1


def test_more_than_4_gib():
    """Rows beyond 2^32 bytes: the last ones against the formula."""
    hidden = 4096
    rows = (1 << 32) // (hidden * 2) + 5
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(rows, hidden, generator=g, device="cuda", dtype=torch.bfloat16)
    dy = torch.zeros_like(x)
    dy[-40:] = R.rand(g, (40, hidden), torch.bfloat16)
    w = torch.ones(hidden, device="cuda", dtype=torch.bfloat16)
    dx, dw = rn.rms_norm_backward(dy, x, w, 1e-6)
    ref = R.norm_bwd(dy[-40:].double(), dy[-40:].double().abs(), x[-40:], w, 0.0, 1e-6, 0)
    R.assert_close(dx[-40:], ref[0], ref[1], 144)
    R.assert_close(dw, ref[2], ref[3], 128 + rows / 32)
    assert not dx[:-40].any()


def test_other_streams_and_graphs():
    sets = [make("bf16", r, 4096, s) for r, s in ((700, 7), (650, 8))]
    want = [rn.rms_norm_backward(dy, x, w, 1e-6) for dy, x, w, _ in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        got = [rn.rms_norm_backward(dy, x, w, 1e-6, stream=s)
               for (dy, x, w, _), s in zip(sets, streams)]
        for s in streams:
            s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    graphs = []
    for dy, x, w, g in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = rn.rms_norm_backward(dy, x, w, 1e-6)
        graphs.append((graph, out))
    for _ in range(2):
        for (dy, x, w, g), (graph, _) in zip(sets, graphs):
            dy.copy_(R.rand(g, dy.shape, dy.dtype))
            graph.replay()
        torch.cuda.synchronize()
        for (dy, x, w, g), (_, out) in zip(sets, graphs):
            got = [t.clone() for t in out]
            want = rn.rms_norm_backward(dy, x, w, 1e-6)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ the operators together

class RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, eps):
        ctx.save_for_backward(x, w)
        ctx.eps = eps
        return rn.rms_norm(x, w, eps)

    @staticmethod
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        dx, dw = rn.rms_norm_backward(dy.contiguous(), x, w, ctx.eps)
        return dx, dw.to(w.dtype), None


class QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, qw, kw, cos_sin, positions, eps):
        ctx.save_for_backward(q, k, qw, kw, cos_sin, positions)
        ctx.eps = eps
        return rn.qk_norm_rope(q, k, qw, kw, cos_sin, positions, eps,
                               q_out=torch.empty(q.shape, dtype=q.dtype, device=q.device),
                               k_out=torch.empty(k.shape, dtype=k.dtype, device=k.device))

    @staticmethod
    def backward(ctx, dq_out, dk_out):
        q, k, qw, kw, cos_sin, positions = ctx.saved_tensors
        dq, dk, dqw, dkw = rn.qk_norm_rope_backward(dq_out, dk_out, q, k, qw, kw, cos_sin,
                                                    positions, ctx.eps)
        return dq, dk, dqw.to(qw.dtype), dkw.to(kw.dtype), None, None, None


def attention(q, k, v):
    """Causal, grouped heads; [T, H, D]."""
    t, hq, d = q.shape
    k, v = (x.repeat_interleave(hq // k.shape[1], 1) for x in (k, v))
    s = torch.einsum("qhd,khd->hqk", q, k) / d ** 0.5
    mask = torch.ones(t, t, dtype=torch.bool, device=q.device).triu(1)
    return torch.einsum("hqk,khd->qhd", s.masked_fill(mask, float("-inf")).softmax(-1), v)


def block(x, wn, wp, qw, kw, cs, pos, norm, rope, hq=4, hk=2, d=64):
    qkv = (norm(x, wn) @ wp).view(x.shape[0], hq + 2 * hk, d)
    q, k = rope(qkv[:, :hq], qkv[:, hq:hq + hk], qw, kw, cs, pos)
    return attention(q, k, qkv[:, hq + hk:]).flatten(1)


def test_training_step_of_a_block():
    """Row norm, projection, head norms with rotation, attention: every
    gradient against automatic differentiation of the definition in 64 bits.
    All in fp32: sums of up to 512 terms through five operations, with
    attention in PyTorch's fp32: 2^-24 * 512 * 8 of each tensor's largest value."""
    T, n, eps = 50, 256, 1e-6
    g = torch.Generator(device="cuda").manual_seed(9)
    mk = lambda *s, scale=1.0, off=0.0: R.rand(g, s, torch.float32, scale) + off
    leaves = [mk(T, n), mk(n, scale=0.1, off=1.0), mk(n, 512, scale=n ** -0.5),
              mk(64, scale=0.1, off=1.0), mk(64, scale=0.1, off=1.0)]
    cs, pos = R.table(64, 64), torch.arange(T, device="cuda")
    up = mk(T, 256)
    mine = [t.clone().requires_grad_() for t in leaves]
    torch.backends.cuda.matmul.allow_tf32 = False
    y = block(*mine, cs, pos, lambda x, w: RmsNorm.apply(x, w, eps),
              lambda q, k, qw, kw, c, p: QkNormRope.apply(q, k, qw, kw, c, p, eps))
    y.backward(up)
    wide = [t.double().requires_grad_() for t in leaves]
    ref = block(*wide, cs.double(), pos,
                lambda x, w: x * R.factor(x, eps) * w,
                lambda q, k, qw, kw, c, p: tuple(
                    R.turn(t * R.factor(t, eps) * w, c[p], False)[0]
                    for t, w in ((q, qw), (k, kw))))
    ref.backward(up.double())
    tol = R.U * 512 * 8
    for a, b in zip([y] + [t.grad for t in mine], [ref] + [t.grad for t in wide]):
        assert (a.double() - b).abs().max() <= tol * b.abs().max()


def test_serving_prompt_then_tokens():
    """A prompt appended in two chunks, then token by token, through a paged
    cache: attention over the pages is attention over the whole sequence."""
    T, hq, hk, d, page = 45, 4, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(10)
    qkv = R.rand(g, (T, hq + 2 * hk, d), torch.float32)
    w = (1 + R.rand(g, d, torch.float64, 0.1)).float()
    cs = R.table(64, d)
    kc, vc = (torch.zeros(8, page, hk, d, device="cuda") for _ in "kv")
    pages = torch.tensor([5, 0, 3], device="cuda")
    pos = torch.arange(T, device="cuda")
    slots = pages[pos // page] * page + pos % page
    q = torch.empty(T, hq, d, device="cuda")
    for a, b in ((0, 30), (30, 41), (41, 42), (42, 43), (43, 44), (44, 45)):
        part = qkv[a:b]
        rn.qk_norm_rope_append(part[:, :hq], part[:, hq:hq + hk], part[:, hq + hk:], w, w, cs,
                               pos[a:b], slots[a:b], kc, vc, 1e-6, q_out=q[a:b])
    got = attention(q, kc.view(-1, hk, d)[slots], vc.view(-1, hk, d)[slots])
    turn = lambda t: R.heads(t, w, 0.0, 1e-6, cs[:T], False)[0]
    want = attention(turn(qkv[:, :hq]), turn(qkv[:, hq:hq + hk]), qkv[:, hq + hk:].double())
    assert (got.double() - want).abs().max() <= R.U * 512 * want.abs().max()


def test_the_readme_examples_run():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "README.md")).read()
    blocks = re.findall(r"```python\n(.*?)```", text, re.S)
    scope = {}
    for b in blocks:
        exec(b, scope)
    torch.cuda.synchronize()
    ref = R.heads(scope["k"], scope["kw"], 0.0, 1e-6, scope["table"], False)
    R.assert_close(scope["k_cache"].view(-1, 8, 128)[64:64 + 4096], *ref, 32)
    b = R.heads_bwd(scope["ko"], scope["k"], scope["kw"], 0.0, 1e-6, scope["table"], False)
    R.assert_close(scope["dk"], b[0], b[1], 128)
    R.assert_close(scope["dkw"], b[2], b[3], 128 + 4096 * 8 / 1000)
