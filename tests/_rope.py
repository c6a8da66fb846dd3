"""Plain 64-bit forms of the rotation, cache and gradient operators, with
first-order error bounds for a computation of them in binary32.

u = 2^-24 bounds the relative error of one fp32 operation.  Each reference
returns, beside its values, the magnitude A that multiplies u: the sum of the
absolute values of the terms added up, so that a result formed with at most K
roundings on any path from an input is off by at most K u A (to first order),
plus half a step of its type where it is rounded to fewer bits."""
import torch

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# half of the smallest subnormal
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150,
        torch.float8_e4m3fn: 2.0 ** -10}


def table(n, rd, base=10000.0, device="cuda"):
    """cos | sin of the first n positions, formed in 64 bits."""
    f = base ** (-torch.arange(rd // 2, dtype=torch.float64, device=device) * 2 / max(rd, 1))
    a = torch.arange(n, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def factor(x, eps):
    """rsqrt(mean x^2 + eps); eps is the fp32 value the kernels are given."""
    e = torch.tensor(eps, dtype=torch.float32).double().item()
    return ((x * x).mean(-1, keepdim=True) + e).rsqrt()


def split(x, rd, inter):
    h = rd // 2
    if inter:
        return x[..., 0:rd:2], x[..., 1:rd:2], x[..., rd:]
    return x[..., :h], x[..., h:rd], x[..., rd:]


def join(a, b, rest, inter):
    p = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([p, rest], -1)


def turn(x, cs, inter, back=False):
    """Rotated [T, H, D] and sum of the terms' absolute values."""
    rd = cs.shape[-1]
    c, s = cs[:, None, :rd // 2], cs[:, None, rd // 2:]
    if back:
        s = -s
    a, b, rest = split(x, rd, inter)
    y = join(a * c - b * s, b * c + a * s, rest, inter)
    m = join((a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs(), rest.abs(), inter)
    return y, m


def heads(x, w, bias, eps, cs, inter):
    """Norm (w None: none) and rotation of x [T, H, D] in 64 bits: (y, A)."""
    u = x.double()
    if w is not None:
        u = u * factor(u, eps) * (w.double() + bias)
    return turn(u, cs.double(), inter)


def norm_bwd(du, du_mag, x, w, bias, eps, over):
    """(dx, A, dw, A) of the norm's gradient in 64 bits."""
    x, g = x.double(), w.double() + bias
    r = factor(x, eps)
    xh = x * r
    n = x.shape[-1]
    m = (du * g * xh).sum(-1, keepdim=True) / n
    am = (du_mag * g.abs() * xh.abs()).sum(-1, keepdim=True) / n
    dx = r * (du * g - xh * m)
    return (dx, r * (du_mag * g.abs() + xh.abs() * am), (du * xh).sum(over),
            (du_mag * xh.abs()).sum(over))


def heads_bwd(dy, x, w, bias, eps, cs, inter):
    du, mag = turn(dy.double(), cs.double(), inter, back=True)
    return norm_bwd(du, mag, x, w, bias, eps, (0, 1))


def assert_close(got, ref, mag, K, what=""):
    """|got - ref| <= K u A, and half a step of got's type: NaN and infinities
    have to be the reference's (a finite reference may round to infinity only
    beyond the type's range)."""
    dt = got.dtype
    g = got.double()
    if dt != torch.float8_e4m3fn:
        top = torch.finfo(dt).max * (1 + torch.finfo(dt).eps / 4)
        ref = torch.where(ref.abs() >= top, ref.sign() * float("inf"), ref)
    nan = ref.isnan()
    assert torch.equal(nan, g.isnan()), f"{what}: NaN pattern differs"
    inf = ref.isinf()
    assert torch.equal(g[inf], ref[inf]), f"{what}: infinities differ"
    fin = ~(nan | inf)
    own = K * U * mag[fin]
    half = (0.0 if dt == torch.float32 else torch.finfo(dt).eps / 2)
    tol = own + half * (ref[fin].abs() + own) + TINY[dt]
    d = (g[fin] - ref[fin]).abs()
    bad = d > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{(d / tol).max().item():.3g} of the bound")


def rand(gen, shape, dt, scale=1.0, device="cuda"):
    return (torch.randn(shape, generator=gen, device=device, dtype=torch.float64)
            * scale).to(dt)


def lay(values, layout):
    """A tensor of the same values [T, H, D] in the named layout."""
    t, h, d = values.shape
    kw = dict(dtype=values.dtype, device=values.device)
    if layout == "plain":
        out = torch.empty(t, h, d, **kw)
    elif layout == "wide":       # a slice of a wider row, as of a fused QKV buffer
        out = torch.empty(t, h + 3, d, **kw)[:, 2:2 + h]
    elif layout == "by_head":    # a head's q, k and v side by side
        out = torch.empty(t, h, 3, d, **kw)[:, :, 1]
    elif layout == "head_major":
        out = torch.empty(h, t, d, **kw).transpose(0, 1)
    elif layout == "shifted":    # one element off every vector boundary
        out = torch.empty(t * h * d + 1, **kw)[1:].view(t, h, d)
    else:
        raise ValueError(layout)
    out.copy_(values)
    return out
