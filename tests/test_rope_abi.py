"""Argument checks of the rotation, cache and gradient entry points, without a
GPU: pointers are numbers that no check follows."""
import ctypes
import itertools
import random

import pytest

import rmsnorm_fwd_gb300 as rn

import _rope as R

P = 1 << 40                      # pointers, far from one another
STEP = 1 << 36
VALIDATED = (rn.OK, rn.ERR_CUDA, rn.ERR_NOT_INITIALIZED)  # got past argument checks


def ptr(i):
    return P + i * STEP


def rope(**kw):
    d = dict(cos_sin=ptr(20), positions=ptr(21), max_position=4096, rotary_dim=128, interleaved=0)
    d.update(kw)
    return rn.Rope(*d.values())


def H(data, ts=0, hs=0):
    return None if data is None else rn.Heads(data, ts, hs)


def fwd(q=H(ptr(0)), k=H(ptr(1)), qo=None, ko=None, qw=ptr(10), kw=ptr(11), rp=None, T=4, hq=8,
        hk=2, D=128, bias=0.0, eps=1e-6, dtype=rn.BF16):
    return rn._load().rmsnorm_qk_norm_rope(*map(rn._ref, (q, k, qo, ko)), qw, kw,
                                           rn._ref(rp or rope()), T, hq, hk, D, bias, eps, dtype,
                                           None)


SIZES = [
    (dict(dtype=7), rn.ERR_UNSUPPORTED_DTYPE),
    (dict(T=-1), rn.ERR_INVALID_ARG), (dict(hq=-1), rn.ERR_INVALID_ARG),
    (dict(hk=1 << 21), rn.ERR_INVALID_ARG), (dict(D=0), rn.ERR_INVALID_ARG),
    (dict(D=1025), rn.ERR_INVALID_ARG), (dict(eps=-1.0), rn.ERR_INVALID_ARG),
    (dict(eps=float("nan")), rn.ERR_INVALID_ARG), (dict(eps=float("inf")), rn.ERR_INVALID_ARG),
    (dict(bias=float("inf")), rn.ERR_INVALID_ARG), (dict(T=1 << 62), rn.ERR_INVALID_ARG),
    (dict(rp=rope(rotary_dim=130)), rn.ERR_INVALID_ARG),
    (dict(rp=rope(rotary_dim=63)), rn.ERR_INVALID_ARG),
    (dict(rp=rope(rotary_dim=-2)), rn.ERR_INVALID_ARG),
    (dict(rp=rope(interleaved=2)), rn.ERR_INVALID_ARG),
    (dict(rp=rope(max_position=-1)), rn.ERR_INVALID_ARG),
    (dict(rp=rope(cos_sin=None)), rn.ERR_INVALID_ARG),
    (dict(rp=rope(positions=None)), rn.ERR_INVALID_ARG),
    (dict(rp=rope(positions=ptr(21) + 4)), rn.ERR_MISALIGNED),
    (dict(rp=rope(cos_sin=ptr(20) + 2)), rn.ERR_MISALIGNED),
    (dict(q=H(ptr(0) + 1)), rn.ERR_MISALIGNED),
    (dict(qw=ptr(10) + 1), rn.ERR_MISALIGNED), (dict(kw=ptr(11) + 1), rn.ERR_MISALIGNED),
    (dict(kw=ptr(11) + 2, dtype=rn.F32), rn.ERR_MISALIGNED),
    (dict(q=None), rn.ERR_INVALID_ARG), (dict(k=H(0)), rn.ERR_INVALID_ARG),
    (dict(qw=None), rn.ERR_INVALID_ARG), (dict(kw=None), rn.ERR_INVALID_ARG),
    (dict(q=H(ptr(0), -1)), rn.ERR_INVALID_ARG),
    (dict(q=H(ptr(0), 8 * 128 - 1)), rn.ERR_INVALID_ARG),     # tokens share elements
    (dict(q=H(ptr(0), 0, 127)), rn.ERR_INVALID_ARG),          # heads share elements
    (dict(q=H(ptr(0), 128, 511)), rn.ERR_INVALID_ARG),        # head-major, one short
    (dict(q=H(ptr(0), 1 << 60)), rn.ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", SIZES, ids=[str(i) for i in range(len(SIZES))])
def test_sizes_and_pointers(kw, status):
    assert fwd(**kw) == status


@pytest.mark.parametrize("kw", [
    dict(), dict(T=0, q=None, k=None), dict(hq=0, q=None, qw=None), dict(hk=0, k=None, kw=None),
    dict(rp=rope(rotary_dim=0, cos_sin=None, positions=None)), dict(q=H(ptr(0), 128, 512)),
    dict(q=H(ptr(0), 8 * 384, 384)), dict(T=1, q=H(ptr(0), 1, 128)), dict(hq=1, q=H(ptr(0), 128, 1)),
    dict(rp=rope(max_position=0, cos_sin=None)), dict(D=1024, rp=rope(rotary_dim=1024)),
    dict(dtype=rn.F32), dict(dtype=rn.F16, rp=rope(interleaved=1))])
def test_accepted(kw):
    assert fwd(**kw) in VALIDATED


def test_overlaps():
    q, k = ptr(0), ptr(1)
    row = (8 + 2 + 2) * 128
    assert fwd(q=H(q, row), k=H(q + 8 * 256, row)) in VALIDATED          # one fused buffer
    assert fwd(q=H(q, row), k=H(q + 7 * 256, row)) == rn.ERR_ALIASING
    assert fwd(qo=H(q), ko=H(k)) in VALIDATED                            # exactly in place
    assert fwd(qo=H(q + 256)) == rn.ERR_ALIASING                         # one head along
    assert fwd(qo=H(q, 8 * 128 + 128)) == rn.ERR_ALIASING                # other strides
    assert fwd(qo=H(k)) == rn.ERR_ALIASING and fwd(ko=H(q)) == rn.ERR_ALIASING
    assert fwd(qo=H(ptr(2)), ko=H(ptr(2))) == rn.ERR_ALIASING
    # heads side by side, [tokens, heads, q | k | v]
    assert fwd(hk=8, q=H(q, 8 * 384, 384), k=H(q + 256, 8 * 384, 384)) in VALIDATED
    assert fwd(hk=8, q=H(q, 8 * 384, 384), k=H(q + 254, 8 * 384, 384)) == rn.ERR_ALIASING
    for bad in (dict(qw=q + 64), dict(kw=q + 64), dict(kw=k + 2 * 128 * 2 * 4 - 2),
                dict(rp=rope(positions=q + 64)), dict(rp=rope(cos_sin=k - 4096 * 128 * 4 + 4))):
        assert fwd(**bad) == rn.ERR_ALIASING
    assert fwd(kw=k + 2 * 128 * 2 * 4) in VALIDATED                      # right behind k


def test_overlap_rule_against_brute_force():
    """Refused wherever bytes are shared; accepted wherever the two tensors
    have contiguous heads and one token stride, or even head strides, and
    share none."""
    rnd = random.Random(1)
    for _ in range(600):
        D, T = rnd.choice([1, 2, 4]), rnd.randint(1, 4)
        hq, hk = rnd.randint(1, 3), rnd.randint(1, 3)
        if rnd.random() < 0.5:
            ts = (hq + hk) * D + rnd.randint(0, 5)
            a, b = (ts, D), (ts, D)
        else:
            hk, hs = hq, D + rnd.randint(0, 2 * D)
            a = b = (hq * hs, hs)
        off = rnd.randint(-3 * a[0], 3 * a[0])
        cells = lambda o, s, h: {o + t * s[0] + i * s[1] + d
                                 for t, i, d in itertools.product(range(T), range(h), range(D))}
        share = bool(cells(0, a, hq) & cells(off, b, hk))
        rc = fwd(q=H(ptr(0), *a), k=H(ptr(0) + 2 * off, *b), T=T, hq=hq, hk=hk, D=D,
                 rp=rope(rotary_dim=0))
        assert (rc == rn.ERR_ALIASING) == share, (D, T, hq, hk, a, off, rc)


# ------------------------------------------------------------------ gradient of the heads

def bwd(qy=H(ptr(0)), ky=H(ptr(1)), q=H(ptr(2)), k=H(ptr(3)), dq=H(ptr(4)), dk=H(ptr(5)),
        qw=ptr(10), kw=ptr(11), dqw=ptr(12), dkw=ptr(13), rp=None, ws=ptr(14), wb=1 << 30, T=4,
        hq=8, hk=2, D=128, bias=0.0, eps=1e-6, dtype=rn.BF16):
    return rn._load().rmsnorm_qk_norm_rope_bwd(*map(rn._ref, (qy, ky, q, k, dq, dk)), qw, kw, dqw,
                                               dkw, rn._ref(rp or rope()), ws, wb, T, hq, hk, D,
                                               bias, eps, dtype, None)


def test_gradient_arguments():
    for kw, status in SIZES:
        if "q" not in kw and "k" not in kw:
            assert bwd(**kw) == status
    assert bwd() in VALIDATED
    assert bwd(dqw=None, dkw=None, ws=None, wb=0) in VALIDATED
    assert bwd(dqw=None) == rn.ERR_INVALID_ARG
    for name in ("qy", "ky", "q", "k", "dq", "dk"):
        assert bwd(**{name: None}) == rn.ERR_INVALID_ARG
    assert bwd(dq=H(ptr(0))) in VALIDATED and bwd(dq=H(ptr(2))) in VALIDATED
    assert bwd(dq=H(ptr(0) + 2)) == rn.ERR_ALIASING
    assert bwd(dq=H(ptr(1))) == rn.ERR_ALIASING and bwd(dk=H(ptr(2))) == rn.ERR_ALIASING
    assert bwd(dq=H(ptr(4)), dk=H(ptr(4) + 256)) == rn.ERR_ALIASING
    # the checks below need a context, which CPU-only machines do not have
    assert bwd(ws=None) in (rn.ERR_INVALID_ARG,) + VALIDATED


def test_workspace_sizes():
    assert rn.rmsnorm_qk_norm_rope_bwd_workspace(128, 152) >= 152 * 128 * 4
    for D, sms in ((0, 152), (1025, 152), (128, 0)):
        with pytest.raises(rn.RmsnormError):
            rn.rmsnorm_qk_norm_rope_bwd_workspace(D, sms)
    assert rn.rmsnorm_bwd_workspace(0, 4096, rn.BF16, 152) >= 0
    assert rn.rmsnorm_bwd_workspace(16384, 4096, rn.BF16, 152) >= 4096 * 4
    for args in ((-1, 4, rn.BF16, 152), (1, 0, rn.BF16, 152), (1, 4, 9, 152),
                 (1 << 40, 1 << 40, rn.BF16, 152)):
        with pytest.raises(rn.RmsnormError):
            rn.rmsnorm_bwd_workspace(*args)


# ------------------------------------------------------------------ paged cache

def cache(**kw):
    d = dict(k=ptr(15), v=ptr(16), pages=64, page_size=16, page_stride=0, slot_stride=0,
             head_stride=0, e4m3=0, k_scale=1.0, v_scale=1.0)
    d.update(kw)
    return rn.PagedCache(*d.values())


def append(q=H(ptr(0)), k=H(ptr(1)), v=H(ptr(2)), qo=None, qw=ptr(10), kw=ptr(11), rp=None,
           c=None, slots=ptr(17), T=4, hq=8, hk=2, D=128, bias=0.0, eps=1e-6, dtype=rn.BF16):
    return rn._load().rmsnorm_qk_norm_rope_append(*map(rn._ref, (q, k, v, qo)), qw, kw,
                                                  rn._ref(rp or rope()), rn._ref(c or cache()),
                                                  slots, T, hq, hk, D, bias, eps, dtype, None)


def test_status_of_an_index_found_on_the_device():
    assert rn.rmsnorm_status_string(rn.ERR_BAD_INDEX) != "unknown status"


def test_append_arguments():
    for kw, status in SIZES:
        if not ({"q", "k", "qw", "kw"} & set(kw)):
            assert append(**kw) == status
    assert append() in VALIDATED
    assert append(qw=None, kw=None) in VALIDATED                       # rotation alone
    assert append(qw=None) == rn.ERR_INVALID_ARG and append(kw=None) == rn.ERR_INVALID_ARG
    assert append(q=None, hq=0, qw=None) in VALIDATED
    assert append(hk=0) == rn.ERR_INVALID_ARG
    assert append(v=None) == rn.ERR_INVALID_ARG and append(slots=None) == rn.ERR_INVALID_ARG
    assert append(slots=ptr(17) + 4) == rn.ERR_MISALIGNED
    page = 16 * 2 * 128
    for c, status in (
            (cache(pages=-1), rn.ERR_INVALID_ARG), (cache(page_size=0), rn.ERR_INVALID_ARG),
            (cache(k=None), rn.ERR_INVALID_ARG), (cache(v=None), rn.ERR_INVALID_ARG),
            (cache(e4m3=2), rn.ERR_INVALID_ARG), (cache(e4m3=1, k_scale=0.0), rn.ERR_INVALID_ARG),
            (cache(e4m3=1, v_scale=float("nan")), rn.ERR_INVALID_ARG),
            (cache(e4m3=1, v_scale=1e-42), rn.ERR_INVALID_ARG),      # its reciprocal is infinite
            (cache(k=ptr(15) + 1), rn.ERR_MISALIGNED),
            (cache(page_stride=page - 1, slot_stride=256, head_stride=128), rn.ERR_INVALID_ARG),
            (cache(page_stride=page, slot_stride=256, head_stride=127), rn.ERR_INVALID_ARG),
            (cache(page_stride=1 << 58, slot_stride=256, head_stride=128), rn.ERR_INVALID_ARG),
            (cache(v=ptr(15)), rn.ERR_ALIASING), (cache(v=ptr(15) + 256), rn.ERR_ALIASING),
            (cache(k=ptr(0)), rn.ERR_ALIASING), (cache(v=ptr(2) + 512), rn.ERR_ALIASING),
            (cache(k=ptr(10)), rn.ERR_ALIASING), (cache(k=ptr(17)), rn.ERR_ALIASING),
            (cache(k=ptr(21)), rn.ERR_ALIASING), (cache(v=ptr(20)), rn.ERR_ALIASING)):
        assert append(c=c) == status
    for c in (cache(pages=0, k=None, v=None), cache(e4m3=1, k=ptr(15) + 1, v=ptr(16) + 3),
              cache(page_stride=page, slot_stride=128, head_stride=16 * 128),      # head first
              cache(v=ptr(15) + 2 * page, page_stride=2 * page, slot_stride=256, head_stride=128),
              cache(v=ptr(15) + 256, page_stride=2 * page, slot_stride=512, head_stride=256)):
        assert append(c=c) in VALIDATED
    # a cache beside the other, one element too near
    assert append(c=cache(v=ptr(15) + 254, page_stride=2 * page, slot_stride=512,
                          head_stride=256)) == rn.ERR_ALIASING
    assert append(qo=H(ptr(1))) == rn.ERR_ALIASING and append(qo=H(ptr(2))) == rn.ERR_ALIASING
    assert append(qo=H(ptr(17))) == rn.ERR_ALIASING


# ------------------------------------------------------------------ rows

def rows_bwd(dy=ptr(0), x=ptr(1), w=ptr(2), dx=ptr(3), dw=ptr(4), ws=ptr(5), wb=1 << 30, rows=8,
             hidden=4096, bias=0.0, eps=1e-6, dtype=rn.BF16):
    return rn._load().rmsnorm_bwd(dy, x, w, dx, dw, ws, wb, rows, hidden, bias, eps, dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=9), rn.ERR_UNSUPPORTED_DTYPE), (dict(rows=-1), rn.ERR_INVALID_ARG),
    (dict(hidden=0), rn.ERR_INVALID_ARG), (dict(eps=-1.0), rn.ERR_INVALID_ARG),
    (dict(bias=float("nan")), rn.ERR_INVALID_ARG), (dict(w=None), rn.ERR_INVALID_ARG),
    (dict(dy=None), rn.ERR_INVALID_ARG), (dict(x=None), rn.ERR_INVALID_ARG),
    (dict(dx=None), rn.ERR_INVALID_ARG), (dict(rows=1 << 60), rn.ERR_INVALID_ARG),
    (dict(x=ptr(1) + 1), rn.ERR_MISALIGNED), (dict(dw=ptr(4) + 2), rn.ERR_MISALIGNED),
    (dict(dx=ptr(0) + 2), rn.ERR_ALIASING), (dict(dx=ptr(1) + 8192), rn.ERR_ALIASING),
    (dict(dx=ptr(2)), rn.ERR_ALIASING)])
def test_row_gradient_refusals(kw, status):
    assert rows_bwd(**kw) == status


def test_row_gradient_accepted():
    for kw in (dict(), dict(dx=ptr(0)), dict(dx=ptr(1)), dict(dw=None),
               dict(rows=0, dy=None, x=None, dx=None, ws=None, wb=0)):
        assert rows_bwd(**kw) in VALIDATED


# ------------------------------------------------------------------ tensors

def test_tensor_refusals():
    torch = pytest.importorskip("torch")
    q = torch.zeros(3, 4, 64)
    w = torch.ones(64)
    with pytest.raises(ValueError):       # no CPU path
        rn.qk_norm_rope(q, q, w, w, None, None, 1e-6)
    with pytest.raises(ValueError):
        rn.qk_norm_rope_backward(q, q, q, q, w, w, None, None, 1e-6)
    with pytest.raises(ValueError):
        rn.qk_norm_rope_append(q, q, q, w, w, None, None, None, q, q, 1e-6)
    with pytest.raises(ValueError):
        rn.rms_norm_backward(q, q, w, 1e-6)


class Fake:
    """A tensor's layout, as the checks read it."""
    is_cuda, dtype, device = True, "t", "cuda:0"
    dense = False  # what is_contiguous answers; the strides are read where it is false

    def __init__(self, shape, strides):
        self.shape, self._s = tuple(shape), tuple(strides)

    def stride(self):
        return self._s

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def is_contiguous(self):
        return self.dense

    def data_ptr(self):
        return P


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device = "cuda:1"

    with pytest.raises(ValueError):
        rn._there("cuda:0", Stream())


def test_packed_structures_are_the_structures():
    h = rn.Heads.from_buffer_copy(rn._HEADS.pack(1, 2, 3))
    assert (h.data, h.token_stride, h.head_stride) == (1, 2, 3)
    r = rn.Rope.from_buffer_copy(rn._ROPE.pack(1, 2, 3, 4, 5))
    assert [getattr(r, n) for n, _ in r._fields_] == [1, 2, 3, 4, 5]
    c = rn.PagedCache.from_buffer_copy(rn._CACHE.pack(1, 2, 3, 4, 5, 6, 7, 1, 0.5, 0.25))
    assert [getattr(c, n) for n, _ in c._fields_] == [1, 2, 3, 4, 5, 6, 7, 1, 0.5, 0.25]
    for packed, whole in ((rn._HEADS, rn.Heads), (rn._ROPE, rn.Rope), (rn._CACHE, rn.PagedCache)):
        assert packed.size == ctypes.sizeof(whole)


def test_layouts_of_tensors():
    def of(shape, strides):
        packed, tokens = rn._heads(Fake(shape, strides), "q", Fake.dtype, Fake.device)
        return rn.Heads.from_buffer_copy(packed), tokens

    h, n = of((5, 8, 64), (512, 64, 1))
    assert (h.token_stride, h.head_stride, n) == (512, 64, 5)
    h, n = of((2, 5, 8, 64), (5 * 900, 900, 64, 1))
    assert (h.token_stride, h.head_stride, n) == (900, 64, 10)
    h, n = of((2, 1, 5, 8, 64), (4500, 7, 900, 64, 1))
    assert (h.token_stride, n) == (900, 10)
    h, n = of((1, 1, 64), (3, 3, 1))
    assert (h.token_stride, h.head_stride, n) == (0, 0, 1)
    h, n = of((0, 8, 64), (512, 64, 1))
    assert n == 0
    t = Fake((5, 8, 64), (512, 64, 1))
    t.dense = True
    packed, n = rn._heads(t, "q", Fake.dtype, Fake.device)
    h = rn.Heads.from_buffer_copy(packed)
    assert (h.data, h.token_stride, h.head_stride, n) == (P, 0, 0, 5)  # the default strides
    for shape, strides in (((64,), (1,)), ((8, 64), (64, 1)), ((5, 8, 64), (512, 64, 2)),
                           ((2, 5, 8, 64), (4501, 900, 64, 1)), ((5, 8, 64), (0, 64, 1)),
                           ((5, 8, 64), (512, 0, 1)), ((3, 5, 8, 64), (0, 512, 64, 1))):
        with pytest.raises(ValueError):
            of(shape, strides)


def test_plain_gradient_is_the_derivative():
    """The 64-bit gradients that the GPU tests compare with, against central
    differences of the 64-bit forward."""
    torch = pytest.importorskip("torch")
    g = torch.Generator().manual_seed(2)
    cs = R.table(9, 6, device="cpu")
    for inter in (False, True):
        x = torch.randn(9, 2, 8, generator=g, dtype=torch.float64)
        w = torch.randn(8, generator=g, dtype=torch.float64)
        dy = torch.randn(9, 2, 8, generator=g, dtype=torch.float64)
        dx, _, dw, _ = R.heads_bwd(dy, x, w, 1.0, 1e-6, cs, inter)
        f = lambda x, w: (dy * R.heads(x, w, 1.0, 1e-6, cs, inter)[0]).sum()
        h = 1e-5
        for t, grad in ((x, dx), (w, dw)):
            for i in range(0, t.numel(), 7):
                step = torch.zeros_like(t).view(-1)
                step[i] = h
                step = step.view_as(t)
                d = (f(x + step, w) - f(x - step, w)) if t is x else \
                    (f(x, w + step) - f(x, w - step))
                assert abs(d / (2 * h) - grad.reshape(-1)[i]) < 1e-7
