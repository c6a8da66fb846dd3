"""The per-head QK norm with its rotation (qk_norm_rope), its gradient and the
paged-cache form on the GPU, against plain forms in 64 bits: head sizes,
layouts, types, lengths, positions and slots outside their tables, padding,
extreme values, streams and captured graphs.

Bounds (K in _rope.assert_close, roundings on the longest path).  Forward: the
sum of squares adds at most 1024 / 32 values a lane and 5 more, and enters r by
its root (half); division, addition, rsqrt (2 steps), two products, the rotation's
two: below 19 + 10, K = 32.  Gradient: xh has 30, the mean adds at most 64
products a lane and 5 more, with 4 roundings of their own and 30 of xh: K = 128
for dx.  dw: a term has 40, and is added at most N / 1000 times within its warp
(608 blocks of 8 warps) and 60 more up to the total: K = 128 + N / 1000."""
import numpy as np
import pytest

import rmsnorm_fwd_gb300 as rn

import _rope as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
K_FWD, K_DX = 32, 128


@pytest.fixture(scope="module", autouse=True)
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rn.ensure_context(0)
    rn.rmsnorm_get_device_status()
    yield
    torch.cuda.synchronize()
    assert rn.rmsnorm_get_device_status() == rn.OK


def make(dtype, T, hq, hk, D, rd, layout, seed, scale=1.0, context=4096):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = R.DT[dtype]
    c = dict(q=R.lay(R.rand(g, (T, hq, D), dt, scale), layout),
             k=R.lay(R.rand(g, (T, hk, D), dt, 3 * scale), layout),
             v=R.lay(R.rand(g, (T, hk, D), dt), layout),
             qw=(1 + R.rand(g, D, torch.float64, 0.1)).to(dt),
             kw=(1 + R.rand(g, D, torch.float64, 0.1)).to(dt),
             cs=R.table(context, rd) if rd else None,
             pos=torch.randint(0, context, (T,), generator=g, device="cuda"))
    c["rows"] = c["cs"][c["pos"]] if rd else torch.zeros(T, 0, device="cuda")
    return c, g


SHAPES = [
    # T, q_heads, k_heads, head_dim, rotary_dim, layout
    (1, 32, 8, 128, 128, "plain"),
    (7, 32, 8, 128, 128, "wide"),
    (131, 4, 4, 64, 64, "by_head"),
    (33, 16, 8, 256, 64, "plain"),
    (50, 3, 1, 128, 96, "head_major"),
    (65, 12, 12, 96, 96, "wide"),
    (29, 5, 5, 80, 80, "plain"),
    (64, 6, 2, 192, 48, "by_head"),
    (9, 4, 2, 128, 0, "plain"),            # no rotation
    (40, 4, 2, 72, 72, "plain"),           # heads that are no whole pairs of vectors
    (21, 3, 2, 7, 6, "plain"),             # odd head size
    (5, 2, 1, 1, 0, "plain"),              # heads of one element
    (6, 2, 2, 2, 2, "plain"),
    (30, 4, 2, 128, 128, "shifted"),       # unaligned heads
    (12, 2, 1, 512, 512, "plain"),
    (4, 2, 1, 1024, 1024, "plain"),        # the largest head
    (300, 8, 1, 64, 34, "wide"),           # halves that straddle vectors
    (777, 40, 8, 128, 128, "wide"),
    (150, 8, 4, 80, 20, "wide"),           # a small part rotated: 4-byte vectors for halves
    (700, 24, 12, 96, 24, "plain"),        # 8-byte vectors, several heads a lane
    (40, 6, 3, 80, 40, "by_head"),
    (2000, 12, 4, 80, 20, "plain"),
    (13001, 1, 1, 64, 64, "wide"),         # few heads: lane groups with tokens of their own
    (5003, 3, 1, 128, 64, "by_head"),
    (4001, 2, 2, 256, 256, "plain"),
    (9999, 6, 2, 80, 80, "head_major"),
]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,hq,hk,D,rd,layout", SHAPES)
def test_forward(T, hq, hk, D, rd, layout, dtype, inter):
    bias = 1.0 if hq % 2 else 0.0
    c, _ = make(dtype, T, hq, hk, D, rd, layout, 1)
    before = c["q"].clone(), c["k"].clone()
    qo, ko = R.lay(torch.zeros_like(c["q"]), layout), torch.empty_like(before[1])
    out = rn.qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["cs"], c["pos"], 1e-6, bias, inter,
                          q_out=qo, k_out=ko)
    assert out[0] is qo and out[1] is ko
    assert torch.equal(c["q"], before[0]) and torch.equal(c["k"], before[1])
    for got, x, w in ((qo, c["q"], c["qw"]), (ko, c["k"], c["kw"])):
        ref, mag = R.heads(x, w, bias, 1e-6, c["rows"], inter)
        R.assert_close(got, ref, mag, K_FWD, f"{dtype} {layout}")
    # in place: the same bits
    rn.qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["cs"], c["pos"], 1e-6, bias, inter)
    assert torch.equal(c["q"], qo) and torch.equal(c["k"], ko)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_fused_buffer_in_place_leaves_values_alone(dtype):
    T, hq, hk, D = 257, 16, 4, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = R.rand(g, (T, hq + 2 * hk, D), R.DT[dtype])
    before = qkv.clone()
    w = (1 + R.rand(g, D, torch.float64, 0.1)).to(R.DT[dtype])
    pos = torch.arange(T, device="cuda")
    cs = R.table(T, D)
    rn.qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hk], w, w, cs, pos, 1e-5)
    ref, mag = R.heads(before[:, :hq + hk], w, 0.0, 1e-5, cs, False)
    R.assert_close(qkv[:, :hq + hk], ref, mag, K_FWD)
    assert torch.equal(qkv[:, hq + hk:], before[:, hq + hk:])


def test_batched_tokens_and_queries_alone():
    g = torch.Generator(device="cuda").manual_seed(4)
    q = R.rand(g, (3, 11, 4, 64), torch.bfloat16)
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    cs, pos = R.table(11, 64), torch.arange(11, device="cuda").repeat(3)
    qo = torch.empty_like(q)
    out = rn.qk_norm_rope(q, None, w, None, cs, pos, 1e-6, q_out=qo)
    assert out[1] is None
    ref, mag = R.heads(q.view(33, 4, 64), w, 0.0, 1e-6, cs[pos], False)
    R.assert_close(qo.view(33, 4, 64), ref, mag, K_FWD)


def test_no_rotation_is_the_qk_norm():
    c, _ = make("bf16", 40, 8, 2, 128, 0, "plain", 5)
    qo, ko = rn.qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], None, None, 1e-6, 1.0,
                             q_out=torch.empty_like(c["q"]), k_out=torch.empty_like(c["k"]))
    q, k = c["q"].clone(), c["k"].clone()
    rn.qk_norm(q.view(40, -1), k.view(40, -1), c["qw"], c["kw"], 128, 1e-6, 1.0)
    for x, w, a, b in ((c["q"], c["qw"], qo, q), (c["k"], c["kw"], ko, k)):
        ref, mag = R.heads(x, w, 1.0, 1e-6, c["rows"], False)
        R.assert_close(a, ref, mag, K_FWD)
        R.assert_close(b, ref, mag, K_FWD)


# ------------------------------------------------------------------ extreme values

@pytest.mark.parametrize("D", [128, 72, 20, 9, 1024])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_extreme_heads(dtype, D):
    """Heads of magnitudes from 2^-110 to 2^103, zeros, subnormals, with
    infinities and NaN; eps 0, tiny and usual.  The other heads are not touched by
    them."""
    c, g = make(dtype, 24, 4, 2, D, D // 2 * 2, "plain", 6)
    dt = R.DT[dtype]
    big, small = ((2.0 ** 100, 2.0 ** -110) if dtype != "f16" else (2.0 ** 11, 2.0 ** -14))
    scale = torch.ones(24, 4, 1, dtype=torch.float64, device="cuda")
    scale[1], scale[2], scale[3, 1], scale[4] = big, small, 0.0, big * 2.0 ** 3
    if dtype != "f16":
        for i, e in enumerate((38, 43, 60, -28, -33, -45, -52, -58, -75)):
            scale[10 + i] = 2.0 ** e
    c["q"] = (c["q"].double() * scale).to(dt)
    c["q"][5, 0, 3] = float("inf")
    c["q"][6, 1, D - 1] = float("nan")
    c["q"][7, 2, 0] = float("-inf")
    c["q"][8, :, :] = torch.finfo(dt).smallest_normal / 4
    dy_q, dy_k = R.rand(g, (24, 4, D), dt), R.rand(g, (24, 2, D), dt)
    for eps in (1e-6, 0.0, 1e-30, 1e-14):
        qo, ko = rn.qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["cs"], c["pos"], eps,
                                 q_out=torch.empty_like(c["q"]), k_out=torch.empty_like(c["k"]))
        ref, mag = R.heads(c["q"], c["qw"], 0.0, eps, c["rows"], False)
        R.assert_close(qo, ref, mag, K_FWD, f"eps {eps}")
        dq, dk, dqw, dkw = rn.qk_norm_rope_backward(dy_q, dy_k, c["q"], c["k"], c["qw"], c["kw"],
                                                    c["cs"], c["pos"], eps)
        rq = R.heads_bwd(dy_q, c["q"], c["qw"], 0.0, eps, c["rows"], False)
        R.assert_close(dq, rq[0], rq[1], K_DX, f"dq, eps {eps}")
        rk = R.heads_bwd(dy_k, c["k"], c["kw"], 0.0, eps, c["rows"], False)
        R.assert_close(dk, rk[0], rk[1], K_DX, f"dk, eps {eps}")
        assert torch.equal(dqw.isnan(), rq[2].isnan())
        R.assert_close(dkw, rk[2], rk[3], 129)


def test_eps_zero_with_idle_lanes():
    """Head counts that leave lanes of the last warp without a head, eps 0: no
    zero of theirs is divided by the square root of zero."""
    for hq, hk, D in ((3, 1, 128), (5, 2, 64), (1, 1, 80), (3, 1, 72)):
        c, g = make("bf16", 9, hq, hk, D, D, "plain", 8)
        dy_q, dy_k = R.rand(g, (9, hq, D), torch.bfloat16), R.rand(g, (9, hk, D), torch.bfloat16)
        got = rn.qk_norm_rope_backward(dy_q, dy_k, c["q"], c["k"], c["qw"], c["kw"], c["cs"],
                                       c["pos"], 0.0)
        for i, (dy, x, w) in enumerate(((dy_q, c["q"], c["qw"]), (dy_k, c["k"], c["kw"]))):
            ref = R.heads_bwd(dy, x, w, 0.0, 0.0, c["rows"], False)
            R.assert_close(got[i], ref[0], ref[1], K_DX)
            R.assert_close(got[2 + i], ref[2], ref[3], 129)


# ------------------------------------------------------------------ positions outside the table

def test_positions_outside_the_table():
    for D in (128, 72, 7, 600):
        c, g = make("bf16", 40, 4, 2, D, D // 2 * 2, "plain", 7, context=100)
        bad = [0, 3, 17, 39]
        c["pos"][bad] = torch.tensor([-1, 100, 1 << 40, -(1 << 62)], device="cuda")
        fill = R.rand(g, (40, 4, D), torch.bfloat16)
        qo, ko = fill.clone(), fill[:, :2].clone()
        rn.qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["cs"], c["pos"], 1e-6, q_out=qo,
                        k_out=ko)
        assert rn.rmsnorm_get_device_status() == rn.ERR_BAD_INDEX
        assert rn.rmsnorm_get_device_status() == rn.OK
        ok = torch.ones(40, dtype=torch.bool, device="cuda")
        ok[bad] = False
        assert torch.equal(qo[~ok], fill[~ok]) and torch.equal(ko[~ok], fill[~ok][:, :2])
        ref, mag = R.heads(c["q"][ok], c["qw"], 0.0, 1e-6, c["cs"][c["pos"][ok]], False)
        R.assert_close(qo[ok], ref, mag, K_FWD)
        # the gradient: such a token adds nothing
        dy_q, dy_k = R.rand(g, (40, 4, D), torch.bfloat16), R.rand(g, (40, 2, D), torch.bfloat16)
        dq, dk = fill.clone(), fill[:, :2].clone()
        c["q"][3] = float("nan")
        _, _, dqw, dkw = rn.qk_norm_rope_backward(dy_q, dy_k, c["q"], c["k"], c["qw"], c["kw"],
                                                  c["cs"], c["pos"], 1e-6, dq=dq, dk=dk)
        assert rn.rmsnorm_get_device_status() == rn.ERR_BAD_INDEX
        assert torch.equal(dq[~ok], fill[~ok]) and torch.equal(dk[~ok], fill[~ok][:, :2])
        r = R.heads_bwd(dy_q[ok], c["q"][ok], c["qw"], 0.0, 1e-6, c["cs"][c["pos"][ok]], False)
        R.assert_close(dq[ok], r[0], r[1], K_DX)
        R.assert_close(dqw, r[2], r[3], 129)


# ------------------------------------------------------------------ gradient

@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,hq,hk,D,rd,layout", SHAPES)
def test_gradient(T, hq, hk, D, rd, layout, dtype, inter):
    bias = 1.0 if hq % 2 else 0.0
    c, g = make(dtype, T, hq, hk, D, rd, layout, 11)
    dt = R.DT[dtype]
    dy_q, dy_k = R.rand(g, (T, hq, D), dt, 0.1), R.lay(R.rand(g, (T, hk, D), dt, 0.1), layout)
    args = (c["q"], c["k"], c["qw"], c["kw"], c["cs"], c["pos"], 1e-6, bias, inter)
    dq, dk, dqw, dkw = rn.qk_norm_rope_backward(dy_q, dy_k, *args)
    for dx, dw, dy, x, w in ((dq, dqw, dy_q, c["q"], c["qw"]), (dk, dkw, dy_k, c["k"], c["kw"])):
        ref = R.heads_bwd(dy, x, w, bias, 1e-6, c["rows"], inter)
        R.assert_close(dx, ref[0], ref[1], K_DX, "dx")
        assert dw.dtype == torch.float32
        R.assert_close(dw, ref[2], ref[3], 128 + T * x.shape[1] / 1000, "dw")
    # the same inputs give the same bits, into given tensors, without weights' gradients
    again = rn.qk_norm_rope_backward(dy_q, dy_k, *args, dq=R.lay(dq * 0, layout),
                                     dk=torch.empty_like(dk))
    for a, b in zip(again, (dq, dk, dqw, dkw)):
        assert torch.equal(a, b)
    # over the gradients, over the inputs
    over = rn.qk_norm_rope_backward(dy_q, dy_k, *args, dq=dy_q, dk=dy_k, weight_grads=False)
    assert over[0] is dy_q and torch.equal(dy_q, dq) and torch.equal(dy_k, dk)
    assert over[2] is None and over[3] is None


def test_gradient_over_the_inputs():
    for D in (128, 72):
        c, g = make("bf16", 19, 4, 2, D, D, "wide", 12)
        dy_q, dy_k = R.rand(g, (19, 4, D), torch.bfloat16), R.rand(g, (19, 2, D), torch.bfloat16)
        args = (c["q"], c["k"], c["qw"], c["kw"], c["cs"], c["pos"], 1e-6)
        want = rn.qk_norm_rope_backward(dy_q, dy_k, *args)
        got = rn.qk_norm_rope_backward(dy_q, dy_k, *args, dq=c["q"], dk=c["k"])
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_gradient_of_many_tokens():
    """More heads than the grid takes at once; both weights' sums in order."""
    T, hq, hk, D = 5003, 9, 3, 128
    c, g = make("bf16", T, hq, hk, D, D, "wide", 13)
    dy_q, dy_k = R.rand(g, (T, hq, D), torch.bfloat16), R.rand(g, (T, hk, D), torch.bfloat16)
    args = (c["q"], c["k"], c["qw"], c["kw"], c["cs"], c["pos"], 1e-6, 0.0, False)
    got = rn.qk_norm_rope_backward(dy_q, dy_k, *args)
    for i, (dy, x, w) in enumerate(((dy_q, c["q"], c["qw"]), (dy_k, c["k"], c["kw"]))):
        ref = R.heads_bwd(dy, x, w, 0.0, 1e-6, c["rows"], False)
        R.assert_close(got[i], ref[0], ref[1], K_DX)
        R.assert_close(got[2 + i], ref[2], ref[3], 128 + T * x.shape[1] / 1000)
    again = rn.qk_norm_rope_backward(dy_q, dy_k, *args)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_gradient_without_tokens_or_keys():
    w = torch.ones(64, device="cuda")
    e = torch.empty(0, 4, 64, device="cuda")
    pos = torch.empty(0, dtype=torch.int64, device="cuda")
    cs = R.table(4, 64)
    dq, dk, dqw, dkw = rn.qk_norm_rope_backward(e, e, e, e, w, w, cs, pos, 1e-6)
    assert dq.shape == e.shape and not dqw.any() and not dkw.any()
    g = torch.Generator(device="cuda").manual_seed(1)
    q, dy = R.rand(g, (3, 4, 64), torch.float32), R.rand(g, (3, 4, 64), torch.float32)
    pos = torch.arange(3, device="cuda")
    dq, dk, dqw, dkw = rn.qk_norm_rope_backward(dy, None, q, None, w, None, cs, pos, 1e-6)
    ref = R.heads_bwd(dy, q, w, 0.0, 1e-6, cs[pos], False)
    R.assert_close(dq, ref[0], ref[1], K_DX)
    R.assert_close(dqw, ref[2], ref[3], 129)
    assert dk is None and not dkw.any()


@pytest.mark.parametrize("lead", [(0,), (2, 0), (0, 2), (3, 0, 2)])
def test_empty_batches(lead):
    e, w = torch.empty(*lead, 4, 64, device="cuda"), torch.ones(64, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    cs = R.table(4, 64)
    assert rn.qk_norm_rope(e, e, w, w, cs, none, 1e-6)[0] is e
    dq, dk, dqw, _ = rn.qk_norm_rope_backward(e, e, e, e, w, w, cs, none, 1e-6)
    assert dq.shape == e.shape == dk.shape and not dqw.any()
    kc, vc = torch.zeros(2, 1, 16, 4, 64, device="cuda")
    assert rn.qk_norm_rope_append(e, e, e, w, w, cs, none, none, kc, vc, 1e-6) is e
    assert not kc.any() and not vc.any()


@pytest.mark.parametrize("inter", [False, True])
def test_gradient_against_differences(inter):
    """<dx, a> + <dw, b> against the central difference of <dy, y> in 64 bits
    along (a, b): its error is h^2 of the third derivative and 2^-52 / h."""
    c, g = make("f32", 6, 3, 2, 64, 48, "plain", 14)
    dy = R.rand(g, (6, 3, 64), torch.float32)
    dq, _, dqw, _ = rn.qk_norm_rope_backward(dy, R.rand(g, (6, 2, 64), torch.float32), c["q"],
                                             c["k"], c["qw"], c["kw"], c["cs"], c["pos"], 1e-6,
                                             1.0, inter)
    x, w = c["q"].double(), c["qw"].double()
    a = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
    b = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64)
    f = lambda h: (dy.double() * R.heads(x + h * a, w + h * b, 1.0, 1e-6, c["rows"],
                                         inter)[0]).sum()
    h = 1e-4
    want = ((f(h) - f(-h)) / (2 * h)).item()
    got = ((dq.double() * a).sum() + (dqw.double() * b).sum()).item()
    # fp32 gradients: 1152 terms of order 1, each off by a few 2^-24
    assert abs(got - want) <= 1152 * 128 * R.U + 1e-5


# ------------------------------------------------------------------ paged cache

def make_cache(g, dtype, cache, pages, page, hk, D, layout):
    dt = torch.float8_e4m3fn if cache == "e4m3" else R.DT[dtype]
    mk = lambda *s: R.rand(g, s, torch.float32).to(dt)
    if layout == "slots":
        return mk(pages, page, hk, D), mk(pages, page, hk, D)
    if layout == "heads":
        return tuple(mk(pages, hk, page, D).transpose(1, 2) for _ in "kv")
    if layout == "pair":         # [pages, 2, page, heads, D]
        both = mk(pages, 2, page, hk, D)
        return both[:, 0], both[:, 1]
    if layout == "split":        # [pages, page, heads, k | v]
        both = mk(pages, page, hk, 2 * D)
        return both[..., :D], both[..., D:]
    raise ValueError(layout)


def raw(t):
    return t.contiguous().view(torch.uint8)


def check_append(c, g, dtype, cache, page, hk, D, layout, inter, norm=True, bias=0.0, pad=(),
                 scales=(0.25, 0.04)):
    T = c["k"].shape[0]
    pages = T // page + 3
    kc, vc = make_cache(g, dtype, cache, pages, page, hk, D, layout)
    k0, v0 = kc.clone(), vc.clone()
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    live = torch.ones(T, dtype=torch.bool, device="cuda")
    for i, t in enumerate(pad):
        live[t] = False
        slots[t] = -1 - i * (1 << 40)
        c["pos"][t] = -7                      # padding's position is not read
        c["q"][t], c["k"][t], c["v"][t] = (float("nan"),) * 3
    ks, vs = scales if cache == "e4m3" else (1.0, 1.0)
    fill = R.rand(g, c["q"].shape, R.DT[dtype])
    qo = fill.clone()
    kb, vb = c["k"].clone(), c["v"].clone()
    qw, kw = (c["qw"], c["kw"]) if norm else (None, None)
    out = rn.qk_norm_rope_append(c["q"], c["k"], c["v"], qw, kw, c["cs"], c["pos"], slots, kc, vc,
                                 1e-6, bias, inter, ks, vs, q_out=qo)
    assert out is qo
    assert torch.equal(raw(c["k"]), raw(kb)) and torch.equal(raw(c["v"]), raw(vb))
    rows = c["cs"][c["pos"][live]] if c["cs"] is not None else torch.zeros(int(live.sum()), 0,
                                                                          device="cuda")
    ref, mag = R.heads(c["q"][live], qw, bias, 1e-6, rows, inter)
    R.assert_close(qo[live], ref, mag, K_FWD, "q")
    assert torch.equal(qo[~live], fill[~live])
    s = slots[live]
    kr, km = R.heads(c["k"][live], kw, bias, 1e-6, rows, inter)
    vr = c["v"][live].double()
    vm = vr.abs()
    # as bytes where elements are: 8-bit types are not indexed by every version
    at = lambda t: t.contiguous().view(torch.uint8).view(pages * page, -1)
    pick = lambda t, i: at(t)[i].view(t.dtype).view(-1, hk, D)
    if cache == "e4m3":
        f = lambda x, sc: ((x / torch.tensor(sc, dtype=torch.float32).double().item())
                           .clamp(-448, 448))
        kr, km, vr, vm = f(kr, ks), km / ks, f(vr, vs), vm / vs
        R.assert_close(pick(vc, s), vr, vm, 4, "v codes")
    else:
        assert torch.equal(raw(pick(vc, s)), raw(c["v"][live]))
    R.assert_close(pick(kc, s), kr, km, K_FWD + 3, "k")
    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    rest[s] = False
    assert torch.equal(at(kc)[rest], at(k0)[rest]) and torch.equal(at(vc)[rest], at(v0)[rest])


APPEND = [
    # T, q_heads, k_heads, head_dim, rotary_dim, layout of q k v, page, cache layout
    (1, 32, 8, 128, 128, "plain", 16, "slots"),
    (1, 4, 1, 64, 64, "plain", 1, "heads"),
    (37, 32, 8, 128, 128, "wide", 16, "slots"),
    (50, 8, 8, 128, 64, "wide", 17, "heads"),
    (33, 16, 4, 256, 256, "by_head", 64, "pair"),
    (45, 5, 5, 80, 80, "plain", 16, "split"),
    (29, 6, 2, 192, 0, "head_major", 5, "heads"),
    (18, 4, 2, 72, 72, "plain", 16, "slots"),
    (18, 3, 1, 7, 6, "plain", 3, "heads"),
    (23, 4, 2, 128, 128, "shifted", 16, "slots"),
    (11, 2, 2, 512, 128, "plain", 8, "slots"),
    (700, 40, 8, 128, 128, "wide", 16, "slots"),
    (9001, 1, 1, 64, 32, "wide", 16, "heads"),     # lane groups with tokens of their own
    (4003, 3, 1, 128, 128, "by_head", 17, "pair"),
    (5001, 4, 2, 80, 80, "plain", 64, "split"),
]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,hq,hk,D,rd,layout,page,cl", APPEND)
def test_append(T, hq, hk, D, rd, layout, page, cl, dtype, cache, inter):
    c, g = make(dtype, T, hq, hk, D, rd, layout, 21)
    pad = () if T < 4 else (0, T // 2, T - 2, T - 1)
    check_append(c, g, dtype, cache, page, hk, D, cl, inter, bias=1.0 if hq % 2 else 0.0, pad=pad)


@pytest.mark.parametrize("D", [128, 72])
@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_append_rotation_alone(cache, D):
    c, g = make("bf16", 60, 8, 2, D, D, "wide", 22)
    check_append(c, g, "bf16", cache, 16, 2, D, "heads", False, norm=False, pad=(5,))


def test_append_in_place_and_keys_alone():
    c, g = make("bf16", 20, 8, 2, 128, 128, "wide", 23)
    kc, vc = make_cache(g, "bf16", "same", 4, 16, 2, 128, "slots")
    slots = torch.arange(20, device="cuda")
    ref, mag = R.heads(c["q"], c["qw"], 0.0, 1e-6, c["rows"], False)
    out = rn.qk_norm_rope_append(c["q"], c["k"], c["v"], c["qw"], c["kw"], c["cs"], c["pos"],
                                 slots, kc, vc, 1e-6)
    assert out is c["q"]
    R.assert_close(c["q"], ref, mag, K_FWD)
    kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
    assert rn.qk_norm_rope_append(None, c["k"], c["v"], None, c["kw"], c["cs"], c["pos"], slots,
                                  kc2, vc2, 1e-6) is None
    assert torch.equal(kc2.view(-1, 256)[:20], kc.view(-1, 256)[:20])
    assert torch.equal(vc2.view(-1, 256)[:20], vc.view(-1, 256)[:20])


def test_append_saturates_and_keeps_nan():
    c, g = make("bf16", 8, 2, 2, 128, 128, "plain", 24)
    c["v"][0, 0, :6] = torch.tensor([1e6, -1e6, float("inf"), float("-inf"), float("nan"), 0.0],
                                    device="cuda")
    kc, vc = (torch.zeros(1, 8, 2, 128, device="cuda", dtype=torch.uint8) for _ in "kv")
    rn.qk_norm_rope_append(c["q"], c["k"], c["v"], c["qw"], c["kw"], c["cs"], c["pos"],
                           torch.arange(8, device="cuda"), kc, vc, 1e-6, k_scale=1e-3)
    got = vc.view(torch.float8_e4m3fn).float()[0, 0, 0, :6].tolist()
    assert got[:4] == [448.0, -448.0, 448.0, -448.0] and got[4] != got[4] and got[5] == 0.0
    assert kc.view(torch.float8_e4m3fn).float().abs().max() == 448.0


def test_append_to_caches_at_odd_bytes():
    """8-bit caches of which no vector of codes is aligned, and 16-bit ones an
    element off."""
    c, g = make("bf16", 12, 4, 2, 64, 64, "plain", 27)
    slots = torch.randperm(32, generator=g, device="cuda")[:12]
    flat = [torch.zeros(2 * 16 * 2 * 64 + 1, dtype=torch.uint8, device="cuda") for _ in "kv"]
    kc, vc = (f[1:].view(2, 16, 2, 64) for f in flat)
    rn.qk_norm_rope_append(c["q"], c["k"], c["v"], c["qw"], c["kw"], c["cs"], c["pos"], slots, kc,
                           vc, 1e-6, k_scale=0.02, v_scale=0.02)
    kd, vd = (torch.zeros(2, 16, 2, 64, dtype=torch.uint8, device="cuda") for _ in "kv")
    rn.qk_norm_rope_append(None, c["k"], c["v"], None, c["kw"], c["cs"], c["pos"], slots, kd, vd,
                           1e-6, k_scale=0.02, v_scale=0.02)
    ref, mag = R.heads(c["k"], c["kw"], 0.0, 1e-6, c["rows"], False)
    sc = torch.tensor(0.02).double().item()
    for t in (kc, kd):
        codes = t.contiguous().view(32, -1)[slots].view(torch.float8_e4m3fn).view(12, 2, 64)
        R.assert_close(codes, (ref / sc).clamp(-448, 448), mag / sc, K_FWD + 3)
    assert torch.equal(vc.contiguous(), vd)
    flat = [torch.zeros(2 * 16 * 2 * 64 + 1, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    kc, vc = (f[1:].view(2, 16, 2, 64) for f in flat)
    rn.qk_norm_rope_append(None, c["k"], c["v"], None, c["kw"], c["cs"], c["pos"], slots, kc, vc,
                           1e-6)
    R.assert_close(kc.contiguous().view(32, 2, 64)[slots], ref, mag, K_FWD)
    assert torch.equal(vc.contiguous().view(32, 2, 64)[slots], c["v"])


def test_keys_alone_through_the_c_names():
    """No q heads: NULL for q everywhere."""
    c, g = make("bf16", 9, 1, 3, 128, 128, "plain", 28)
    rope = rn.Rope(c["cs"].data_ptr(), c["pos"].data_ptr(), 4096, 128, 0)
    s = torch.cuda.current_stream().cuda_stream
    of = lambda t: rn.Heads(t.data_ptr(), 0, 0)
    ko, dk = torch.empty_like(c["k"]), torch.empty_like(c["k"])
    dy = R.rand(g, c["k"].shape, torch.bfloat16)
    rn.rmsnorm_qk_norm_rope(None, of(c["k"]), None, of(ko), 0, c["kw"].data_ptr(), rope, 9, 0, 3,
                            128, 0.0, 1e-6, rn.BF16, s)
    need = rn.rmsnorm_qk_norm_rope_bwd_workspace(128, rn.rmsnorm_device_limits()[0])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    grads = torch.full((2, 128), 7.0, device="cuda")
    args = (None, of(dy), None, of(c["k"]), None, of(dk), 0, c["kw"].data_ptr(),
            grads[0].data_ptr(), grads[1].data_ptr(), rope, ws.data_ptr())
    rn.rmsnorm_qk_norm_rope_bwd(*args, need, 9, 0, 3, 128, 0.0, 1e-6, rn.BF16, s)
    ref, mag = R.heads(c["k"], c["kw"], 0.0, 1e-6, c["rows"], False)
    R.assert_close(ko, ref, mag, K_FWD)
    b = R.heads_bwd(dy, c["k"], c["kw"], 0.0, 1e-6, c["rows"], False)
    R.assert_close(dk, b[0], b[1], K_DX)
    R.assert_close(grads[1], b[2], b[3], 129)
    assert not grads[0].any()
    # a workspace too small, or not aligned, and outputs inside it
    for bad, status in (((need - 1,), rn.ERR_INVALID_ARG),):
        with pytest.raises(rn.RmsnormError) as e:
            rn.rmsnorm_qk_norm_rope_bwd(*args, *bad, 9, 0, 3, 128, 0.0, 1e-6, rn.BF16, s)
        assert e.value.status == status
    with pytest.raises(rn.RmsnormError) as e:
        rn.rmsnorm_qk_norm_rope_bwd(*args[:-1], ws.data_ptr() + 4, need, 9, 0, 3, 128, 0.0, 1e-6,
                                    rn.BF16, s)
    assert e.value.status == rn.ERR_MISALIGNED
    with pytest.raises(rn.RmsnormError) as e:
        rn.rmsnorm_qk_norm_rope_bwd(*args[:8], ws.data_ptr() + 512, grads[1].data_ptr(), *args[10:],
                                    need, 9, 0, 3, 128, 0.0, 1e-6, rn.BF16, s)
    assert e.value.status == rn.ERR_ALIASING


def test_append_slots_outside_the_cache():
    for D in (128, 72, 7):
        c, g = make("bf16", 30, 4, 2, D, D // 2 * 2, "plain", 25, context=64)
        kc, vc = make_cache(g, "bf16", "same", 3, 16, 2, D, "slots")
        k0, v0 = kc.clone(), vc.clone()
        slots = torch.arange(30, device="cuda") + 9
        slots[4], slots[5], slots[6] = 48, 1 << 50, (1 << 63) - 1
        c["pos"][7] = 64
        fill = R.rand(g, c["q"].shape, torch.bfloat16)
        qo = fill.clone()
        rn.qk_norm_rope_append(c["q"], c["k"], c["v"], c["qw"], c["kw"], c["cs"], c["pos"], slots,
                               kc, vc, 1e-6, q_out=qo)
        assert rn.rmsnorm_get_device_status() == rn.ERR_BAD_INDEX
        bad = torch.tensor([4, 5, 6, 7], device="cuda")
        assert torch.equal(qo[bad], fill[bad])
        at = lambda t: t.view(48, -1)
        for s in (13, 14, 15, 16):                  # the left-out tokens' old places
            assert torch.equal(at(kc)[s], at(k0)[s]) and torch.equal(at(vc)[s], at(v0)[s])
        good = [t for t in range(30) if t not in (4, 5, 6, 7)]
        assert torch.equal(at(vc)[slots[good]], c["v"][good].flatten(1))


def test_bad_and_padded_tokens_between_good_ones():
    """Few heads and many tokens: neighbouring lane groups hold good, padded and
    bad tokens."""
    T = 8000
    c, g = make("bf16", T, 2, 1, 64, 64, "plain", 29, context=64)
    kind = torch.arange(T, device="cuda") % 5           # 1: padding, 2: bad slot, 3: bad position
    slots = torch.randperm(T + 64, generator=g, device="cuda")[:T]
    slots[kind == 1], slots[kind == 2] = -5, T + 64
    c["pos"][kind == 3] = 64
    c["pos"][kind == 1] = 1 << 40
    kc, vc = make_cache(g, "bf16", "same", (T + 64) // 16, 16, 1, 64, "slots")
    k0, v0 = kc.clone(), vc.clone()
    fill = R.rand(g, c["q"].shape, torch.bfloat16)
    qo = fill.clone()
    rn.qk_norm_rope_append(c["q"], c["k"], c["v"], c["qw"], c["kw"], c["cs"], c["pos"], slots, kc,
                           vc, 1e-6, q_out=qo)
    assert rn.rmsnorm_get_device_status() == rn.ERR_BAD_INDEX
    good = (kind == 0) | (kind == 4)
    rows = c["cs"][c["pos"][good]]
    ref, mag = R.heads(c["q"][good], c["qw"], 0.0, 1e-6, rows, False)
    R.assert_close(qo[good], ref, mag, K_FWD)
    assert torch.equal(qo[~good], fill[~good])
    at = lambda t: t.view(T + 64, 1, 64)
    ref, mag = R.heads(c["k"][good], c["kw"], 0.0, 1e-6, rows, False)
    R.assert_close(at(kc)[slots[good]], ref, mag, K_FWD)
    assert torch.equal(at(vc)[slots[good]], c["v"][good])
    rest = torch.ones(T + 64, dtype=torch.bool, device="cuda")
    rest[slots[good]] = False
    assert torch.equal(at(kc)[rest], at(k0)[rest]) and torch.equal(at(vc)[rest], at(v0)[rest])


@pytest.mark.parametrize("T,D", [(8003, 64), (3, 64), (4, 64), (5001, 128), (4001, 192)])
def test_gradient_with_bad_tokens_between_good_ones(T, D):
    """Few heads: neighbouring lane groups hold good and bad tokens, over the inputs."""
    c, g = make("bf16", T, 2, 1, D, D, "plain", 31, context=64)
    ok = torch.arange(T, device="cuda") % 3 != 1
    c["pos"][~ok] = 64
    c["q"][~ok], c["k"][~ok] = float("nan"), float("inf")
    dy_q, dy_k = R.rand(g, (T, 2, D), torch.bfloat16), R.rand(g, (T, 1, D), torch.bfloat16)
    q, k = c["q"].clone(), c["k"].clone()
    dq, dk, dqw, dkw = rn.qk_norm_rope_backward(dy_q, dy_k, q, k, c["qw"], c["kw"], c["cs"],
                                                c["pos"], 1e-6, dq=q, dk=k)
    assert rn.rmsnorm_get_device_status() == rn.ERR_BAD_INDEX
    assert dq.isnan()[~ok].all() and torch.equal(dk[~ok], c["k"][~ok])
    rows = c["cs"][c["pos"][ok]]
    for dx, dw, dy, x, w in ((dq, dqw, dy_q, c["q"], c["qw"]), (dk, dkw, dy_k, c["k"], c["kw"])):
        ref = R.heads_bwd(dy[ok], x[ok], w, 0.0, 1e-6, rows, False)
        R.assert_close(dx[ok], ref[0], ref[1], K_DX, "dx")
        R.assert_close(dw, ref[2], ref[3], 128 + T * x.shape[1] / 1000, "dw")


# ------------------------------------------------------------------ large offsets

def test_offsets_beyond_32_bits():
    """A cache and a fused buffer of more than 2^32 bytes, touched at both ends."""
    D, hk, page = 128, 8, 16
    pages = (1 << 32) // (page * hk * D * 2) + 8           # each of the two caches
    kc = torch.zeros(pages, page, hk, D, device="cuda", dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)
    c, g = make("bf16", 6, 4, hk, D, D, "plain", 26)
    n = pages * page
    slots = torch.tensor([0, 1, n // 2, n - 17, n - 2, n - 1], device="cuda")
    rn.qk_norm_rope_append(c["q"], c["k"], c["v"], c["qw"], c["kw"], c["cs"], c["pos"], slots, kc,
                           vc, 1e-6, q_out=torch.empty_like(c["q"]))
    ref, mag = R.heads(c["k"], c["kw"], 0.0, 1e-6, c["rows"], False)
    R.assert_close(kc.view(n, hk, D)[slots], ref, mag, K_FWD)
    assert torch.equal(vc.view(n, hk, D)[slots], c["v"])
    assert int((vc.view(n, -1)[:, 0] != 0).sum()) <= 6
    del kc, vc
    T = (1 << 32) // (48 * D * 2) + 3
    buf = torch.zeros(T, 48, D, device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(T, device="cuda") % 4096
    small = R.rand(g, (T, 1, D), torch.bfloat16)
    buf[:, 39] = small[:, 0]                                # the last k head
    rn.qk_norm_rope(buf[:, :32], buf[:, 32:40], c["qw"], c["kw"], c["cs"], pos, 1e-6)
    ref, mag = R.heads(small[-64:], c["kw"], 0.0, 1e-6, c["cs"][pos[-64:]], False)
    R.assert_close(buf[-64:, 39:40], ref, mag, K_FWD)


# ------------------------------------------------------------------ streams, graphs, devices

def test_other_streams_and_two_calls_at_once():
    c, g = make("bf16", 3000, 16, 4, 128, 128, "plain", 31)
    d, _ = make("bf16", 2777, 16, 4, 128, 128, "plain", 32)
    dys = [(R.rand(g, x["q"].shape, torch.bfloat16), R.rand(g, x["k"].shape, torch.bfloat16))
           for x in (c, d)]
    args = lambda x: (x["q"], x["k"], x["qw"], x["kw"], x["cs"], x["pos"], 1e-6)
    want = [rn.qk_norm_rope_backward(*dy, *args(x)) for x, dy in zip((c, d), dys)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in "ab"]
    for _ in range(10):
        got = [rn.qk_norm_rope_backward(*dy, *args(x), stream=s)
               for x, dy, s in zip((c, d), dys, streams)]
        for s in streams:
            s.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_inputs_freed_right_after_a_call_on_another_stream():
    """The inputs' memory is not given out again before that stream is done."""
    c, g = make("bf16", 4000, 16, 4, 128, 128, "plain", 33)
    want = rn.qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["cs"], c["pos"], 1e-6,
                           q_out=torch.empty_like(c["q"]), k_out=torch.empty_like(c["k"]))
    s = torch.cuda.Stream()
    for _ in range(5):
        q, k = c["q"].clone(), c["k"].clone()
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000)  # a millisecond: the call below waits behind it
        rn.qk_norm_rope(q, k, c["qw"], c["kw"], c["cs"], c["pos"], 1e-6, q_out=qo, k_out=ko,
                        stream=s)
        del q, k
        torch.full_like(c["q"], 7.0)       # would take their place
        torch.full_like(c["k"], 7.0)
        s.synchronize()
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])


def test_without_dependent_launches():
    """The same bits with programmatic dependent launch off."""
    c, g = make("bf16", 900, 16, 4, 128, 128, "wide", 34)
    dy = R.rand(g, (900, 16, 128), torch.bfloat16), R.rand(g, (900, 4, 128), torch.bfloat16)
    args = (c["q"], c["k"], c["qw"], c["kw"], c["cs"], c["pos"], 1e-6)

    def step():
        qo, ko = rn.qk_norm_rope(*args, q_out=torch.empty(900, 16, 128, device="cuda",
                                                          dtype=torch.bfloat16),
                                 k_out=torch.empty(900, 4, 128, device="cuda",
                                                   dtype=torch.bfloat16))
        return qo, ko, *rn.qk_norm_rope_backward(qo, ko, *args)

    was = rn.rmsnorm_get_pdl()
    try:
        rn.rmsnorm_set_pdl(True)
        a = [step() for _ in range(4)][-1]
        rn.rmsnorm_set_pdl(False)
        b = step()
    finally:
        rn.rmsnorm_set_pdl(was)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_threads_at_once():
    """Two host threads with their own streams and tensors."""
    import threading
    sets = [make("bf16", 700 + 99 * i, 8, 2, 128, 128, "plain", 35 + i) for i in range(2)]
    want, got = [None, None], [None, None]

    def work(i, out, n):
        c, _ = sets[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(n):
                out[i] = rn.qk_norm_rope_backward(c["q"], c["k"], c["q"], c["k"], c["qw"], c["kw"],
                                                  c["cs"], c["pos"], 1e-6)
            torch.cuda.current_stream().synchronize()

    for i in range(2):
        work(i, want, 1)
    threads = [threading.Thread(target=work, args=(i, got, 50)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refusals_of_tensors():
    c, _ = make("bf16", 6, 4, 2, 64, 64, "plain", 37)
    q, k, v, w, cs, pos = c["q"], c["k"], c["v"], c["qw"], c["cs"], c["pos"]
    kc = torch.zeros(2, 4, 2, 64, device="cuda", dtype=torch.bfloat16)
    slots = torch.arange(6, device="cuda")
    ap = lambda **kw: rn.qk_norm_rope_append(**{**dict(
        q=q, k=k, v=v, q_weight=w, k_weight=w, cos_sin=cs, positions=pos, slots=slots, k_cache=kc,
        v_cache=kc.clone(), eps=1e-6, q_out=torch.empty_like(q)), **kw})
    ap()
    for kw in (dict(slots=slots[:5]), dict(slots=slots.cpu()), dict(k_cache=kc[..., :32]),
               dict(v_cache=kc.transpose(0, 1)), dict(positions=pos[:5]), dict(positions=None),
               dict(cos_sin=cs[:, ::2]), dict(v=v[:, :1]), dict(q=q[:5]), dict(k=k[:, :, :32]),
               dict(q_out=q[:5]), dict(q=q.expand(6, 4, 64)[:, :1].expand(6, 4, 64)),
               dict(v_cache=kc.expand(2, 4, 2, 64)[:, :, :1].expand(2, 4, 2, 64)),
               dict(q=None, q_out=q), dict(k=q[0])):
        with pytest.raises(ValueError):
            ap(**kw)
    for kw in (dict(slots=slots.int()), dict(positions=pos.int()), dict(cos_sin=cs.double()),
               dict(q_weight=w.float()), dict(v=v.float()), dict(k_cache=kc.float(),
                                                                 v_cache=kc.float()),
               dict(slots=None)):
        with pytest.raises(TypeError):
            ap(**kw)
    with pytest.raises(rn.RmsnormError) as e:      # one cache for both
        ap(v_cache=kc)
    assert e.value.status == rn.ERR_ALIASING
    with pytest.raises(ValueError):
        rn.qk_norm_rope(q, k, w, w, cs, pos, 1e-6, k_out=k[:5])
    with pytest.raises(ValueError):
        rn.qk_norm_rope(q, None, w, None, cs, pos, 1e-6, k_out=k)
    with pytest.raises(rn.RmsnormError) as e:
        rn.qk_norm_rope(q, k, w, None, cs, pos, 1e-6)
    assert e.value.status == rn.ERR_INVALID_ARG
    with pytest.raises(ValueError):
        rn.qk_norm_rope_backward(q, None, q, k, w, w, cs, pos, 1e-6)
    with pytest.raises(ValueError):
        rn.qk_norm_rope_backward(q[:1, :1].expand(6, 4, 64), k, q, k, w, w, cs, pos, 1e-6)


def test_captured_and_replayed():
    """Forward, gradient and append in one graph; replays follow new inputs,
    positions and slots; a second graph replayed in turn keeps its own results."""
    T, D = 64, 128
    graphs = []
    for seed in (41, 42):
        c, g = make("bf16", T, 8, 2, D, D, "wide", seed)
        kc, vc = make_cache(g, "bf16", "same", 8, 16, 2, D, "heads")
        c.update(kc=kc, vc=vc, slots=torch.arange(T, device="cuda"),
                 qo=torch.empty(T, 8, D, device="cuda", dtype=torch.bfloat16),
                 ko=torch.empty(T, 2, D, device="cuda", dtype=torch.bfloat16))

        def step(c=c):
            rn.qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["cs"], c["pos"], 1e-6,
                            q_out=c["qo"], k_out=c["ko"])
            rn.qk_norm_rope_append(c["q"], c["k"], c["v"], c["qw"], c["kw"], c["cs"], c["pos"],
                                   c["slots"], c["kc"], c["vc"], 1e-6, q_out=c["qo"])
            return rn.qk_norm_rope_backward(c["qo"], c["ko"], c["q"], c["k"], c["qw"], c["kw"],
                                            c["cs"], c["pos"], 1e-6)

        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((c, g, graph, out, step))
    for turn_ in range(3):
        for c, g, graph, out, step in graphs:
            c["q"].copy_(R.rand(g, c["q"].shape, torch.bfloat16))
            c["pos"].copy_(torch.randint(0, 4096, (T,), generator=g, device="cuda"))
            c["slots"].copy_(torch.randperm(128, generator=g, device="cuda")[:T])
            if turn_ == 2:
                c["slots"][T // 2:] = -1
            graph.replay()
        torch.cuda.synchronize()
        for c, g, graph, out, step in graphs:
            got = [t.clone() for t in (*out, c["qo"], c["ko"], c["kc"], c["vc"])]
            want = step()
            for a, b in zip(got, (*want, c["qo"], c["ko"], c["kc"], c["vc"])):
                assert torch.equal(a, b)


# ------------------------------------------------------------------ seeded random cases

def draw(i):
    r = np.random.default_rng(900 + i)
    dtype = ["bf16", "f16", "f32"][r.integers(3)]
    D = int(r.choice([64, 80, 96, 128, 192, 256, 512])) if r.random() < 0.7 else \
        int(r.integers(1, 600))
    rd = int(r.integers(0, D // 2 + 1)) * 2 if r.random() < 0.4 else D // 2 * 2
    if r.random() < 0.3:
        rd = D // 4 // 2 * 2
    hk = int(r.integers(1, 10))
    hq = hk * int(r.integers(1, 6))
    T = int(np.exp(r.uniform(0, np.log(max(2, min(2000, 2 ** 19 // ((hq + hk) * D)))))))
    layout = str(r.choice(["plain", "wide", "by_head", "head_major", "shifted"]))
    return dtype, T, hq, hk, D, rd, layout, bool(r.random() < 0.5), float(r.integers(2)), r


@pytest.mark.parametrize("i", range(120))
def test_random_cases(i):
    dtype, T, hq, hk, D, rd, layout, inter, bias, r = draw(i)
    c, g = make(dtype, T, hq, hk, D, rd, layout, 1000 + i)
    qo, ko = rn.qk_norm_rope(c["q"], c["k"], c["qw"], c["kw"], c["cs"], c["pos"], 1e-6, bias,
                             inter, q_out=torch.empty_like(c["q"].contiguous()),
                             k_out=R.lay(c["k"] * 0, layout))
    dy = [R.rand(g, (T, h, D), R.DT[dtype], 0.2) for h in (hq, hk)]
    grads = rn.qk_norm_rope_backward(*dy, c["q"], c["k"], c["qw"], c["kw"], c["cs"], c["pos"],
                                     1e-6, bias, inter)
    for j, (y, x, w) in enumerate(((qo, c["q"], c["qw"]), (ko, c["k"], c["kw"]))):
        ref, mag = R.heads(x, w, bias, 1e-6, c["rows"], inter)
        R.assert_close(y, ref, mag, K_FWD, "y")
        b = R.heads_bwd(dy[j], x, w, bias, 1e-6, c["rows"], inter)
        R.assert_close(grads[j], b[0], b[1], K_DX, "dx")
        R.assert_close(grads[2 + j], b[2], b[3], 128 + T * x.shape[1] / 1000, "dw")
    pad = sorted(set(int(t) for t in r.integers(0, T, size=T // 5))) if T > 4 else ()
    check_append(c, g, dtype, str(r.choice(["same", "e4m3"])), int(r.choice([1, 3, 16, 64])), hk,
                 D, str(r.choice(["slots", "heads", "pair", "split"])), inter,
                 norm=bool(r.random() < 0.7), bias=bias, pad=pad)
