"""What the norms' rotation, cache and gradient operators are measured on.

Four operators: the per-head QK norm with the position rotation in the same
pass (``rope``), its gradient (``rope_bwd``), the same pass with keys and
values appended to a paged cache (``append``), and the gradient of the row
RMSNorm (``rms_bwd``).  ``run`` computes them from elementary torch operations
in 32 bits, rounded once at the end, or, where ``own`` is true, through the
package's public calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def _rope(name, op, dtype, tokens, q_heads, k_heads, head_dim, rotary_dim, interleaved, fused,
          seqs, bias=0.0):
    return dict(name=name, op=op, dtype=dtype, tokens=tokens, q_heads=q_heads, k_heads=k_heads,
                head_dim=head_dim, rotary_dim=rotary_dim, interleaved=interleaved, fused=fused,
                seqs=seqs, bias=bias)


def _append(name, dtype, tokens, q_heads, k_heads, head_dim, rotary_dim, interleaved, seqs, page,
            heads_first, cache, padded, norm=True, bias=0.0):
    return dict(_rope(name, "append", dtype, tokens, q_heads, k_heads, head_dim, rotary_dim,
                      interleaved, True, seqs, bias),
                page=page, heads_first=heads_first, cache=cache, padded=padded, norm=norm)


def _rms(name, dtype, rows, hidden, bias=0.0):
    return dict(name=name, op="rms_bwd", dtype=dtype, rows=rows, hidden=hidden, bias=bias)


def listed():
    return [
        # one decoded token of a model with grouped queries: latency
        _rope("rope_bf16_1tok_32q8k_128", "rope", "bf16", 1, 32, 8, 128, 128, False, True, 1),
        # a training or prefill batch of packed sequences, the QKV projection's own output
        _rope("rope_bf16_16384tok_32q8k_128", "rope", "bf16", 16384, 32, 8, 128, 128, False, True,
              4),
        # wide heads, a part of each rotated in neighbouring pairs, a ragged number of tokens,
        # weights held as an offset from one
        _rope("rope_f16_5003tok_16q8k_256_part", "rope", "f16", 5003, 16, 8, 256, 64, True, False,
              3, 1.0),
        # gradients of a short training batch
        _rope("rope_bwd_bf16_500tok_16q4k_64", "rope_bwd", "bf16", 500, 16, 4, 64, 64, False,
              False, 2),
        # gradients of the large training batch
        _rope("rope_bwd_bf16_16384tok_32q8k_128", "rope_bwd", "bf16", 16384, 32, 8, 128, 128,
              False, True, 4),
        # single precision, an unusual head size, an odd number of tokens
        _rope("rope_bwd_f32_4097tok_12q12k_96", "rope_bwd", "f32", 4097, 12, 12, 96, 96, True,
              False, 1),
        # one step of a serving batch: a token of each of 32 sequences
        _append("append_bf16_32tok_32q8k_128", "bf16", 32, 32, 8, 128, 128, False, 32, 16, False,
                "same", 0),
        # prompts' chunks into a cache laid out head by head
        _append("append_bf16_16384tok_32q8k_128", "bf16", 16384, 32, 8, 128, 128, False, 9, 64,
                True, "same", 0),
        # an 8-bit cache, a captured batch's padding behind the last sequence
        _append("append_f16_e4m3_3000tok_64q4k_128", "f16", 3000, 64, 4, 128, 64, False, 7, 16,
                False, "e4m3", 317),
        # gradients of the embedding model's rows at a small batch
        _rms("rms_bwd_bf16_509x1024", "bf16", 509, 1024),
        # the block norm of the large training batch
        _rms("rms_bwd_bf16_16384x4096", "bf16", 16384, 4096),
        # a row length that is no power of two, weights held as an offset from one
        _rms("rms_bwd_f16_9001x2880", "f16", 9001, 2880, 1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# Elements of one tensor that a drawn case goes up to.
MOST_HEADS = 16384 * 40 * 128
MOST_ROWS = 16384 * 4096


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "rms_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    size = 2 if dtype == "f32" else 1
    bias = rng.choice([0.0, 0.0, 1.0])
    if op == "rms_bwd":
        hidden = _log(rng, 64, 16384)
        if rng.random() < 0.75:  # most models' rows are whole vectors
            hidden = max(64, hidden // 64 * 64)
        rows = _log(rng, 1, max(2, min(65536, MOST_ROWS // size // hidden)))
        return {k: v for k, v in _rms("", dtype, rows, hidden, bias).items() if k != "name"}
    head_dim = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
    k_heads = rng.choice([1, 2, 4, 5, 8, 12, 16])
    q_heads = k_heads * rng.choice([1, 2, 3, 4, 8])
    rotary_dim = head_dim // rng.choice([1, 1, 1, 2, 4]) // 2 * 2
    limit = MOST_HEADS // size // ((q_heads + 2 * k_heads) * head_dim)
    tokens = _log(rng, 1, max(2, min(16384, limit)))
    interleaved, fused = rng.random() < 0.4, rng.random() < 0.6
    seqs = _log(rng, 1, min(tokens, 64))
    if op == "append":
        cache = rng.choice(["same", "same", "e4m3"])
        padded = rng.randrange(tokens // 2) if tokens > 4 and rng.random() < 0.4 else 0
        c = _append("", dtype, tokens, q_heads, k_heads, head_dim, rotary_dim, interleaved, seqs,
                    rng.choice([1, 16, 16, 17, 64, 128]), rng.random() < 0.5, cache, padded,
                    rng.random() < 0.75, bias)
        c["fused"] = fused
    else:
        c = _rope("", op, dtype, tokens, q_heads, k_heads, head_dim, rotary_dim, interleaved,
                  fused, seqs, bias)
    return {k: v for k, v in c.items() if k != "name"}


def _lengths(c):
    """Tokens of each sequence: they differ by one at most."""
    live = c["tokens"] - c.get("padded", 0)
    seqs = min(c["seqs"], live)
    return [live // seqs + (i < live % seqs) for i in range(seqs)]


def _cache_slots(c):
    """Slots of the cache: every sequence's pages, and as many again."""
    return 2 * sum(-(-n // c["page"]) + 1 for n in _lengths(c)) * c["page"]


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _weight(gen, n, bias, dt):
    return (1.0 - bias + 0.1 * _randn(gen, n)).to(dt)


def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] == "rms_bwd":
        # activations with rows of differing size, gradients as small as a mean loss leaves them
        x = (_randn(gen, c["rows"], c["hidden"]) * torch.exp(_randn(gen, c["rows"], 1))).to(dt)
        dy = (_randn(gen, c["rows"], c["hidden"]) * 2.0 ** -6).to(dt)
        return dict(case=c, x=x, dy=dy, w=_weight(gen, c["hidden"], c["bias"], dt))
    t, hq, hk, d, rd = (c[k] for k in ("tokens", "q_heads", "k_heads", "head_dim", "rotary_dim"))
    # the angles' table that a model keeps: cos of half the rotated size, then sin
    lengths = _lengths(c)
    context = 32768
    angle = (torch.arange(context, device="cuda", dtype=torch.float64)[:, None]
             * 10000.0 ** (-torch.arange(rd // 2, device="cuda", dtype=torch.float64) * 2 / rd))
    table = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    if c["fused"]:  # the QKV projection's output
        qkv = _randn(gen, t, hq + 2 * hk, d).to(dt)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    else:
        q, k, v = (_randn(gen, t, h, d).to(dt) for h in (hq, hk, hk))
    s = dict(case=c, q=q, k=k, v=v, table=table, qw=_weight(gen, d, c["bias"], dt),
             kw=_weight(gen, d, c["bias"], dt))
    # training starts each sequence at 0; serving goes on behind what is cached
    starts = torch.randint(0, context - max(lengths), (len(lengths),), generator=gen,
                           device="cuda") * (c["op"] == "append")
    n = torch.tensor(lengths, device="cuda")
    which = torch.repeat_interleave(torch.arange(len(lengths), device="cuda"), n)
    within = torch.arange(int(n.sum()), device="cuda") - (n.cumsum(0) - n)[which]
    positions = starts[which] + within
    pad = c.get("padded", 0)
    s["positions"] = torch.cat([positions, positions.new_zeros(pad)])
    if c["op"] == "rope_bwd":
        s["dq_out"], s["dk_out"] = ((_randn(gen, t, h, d) * 2.0 ** -6).to(dt) for h in (hq, hk))
    else:
        s["q_out"] = torch.empty(t, hq, d, device="cuda", dtype=dt)
        s["k_out"] = torch.empty(t, hk, d, device="cuda", dtype=dt)
    if c["op"] == "append":
        # every sequence's pages lie anywhere in the cache; its first token may come to stand
        # inside a page
        page, slots = c["page"], _cache_slots(c)
        most = -(-max(lengths) // page) + 1
        pages = torch.randperm(slots // page, generator=gen, device="cuda")
        first = torch.cumsum(torch.tensor([0] + [-(-m // page) + 1 for m in lengths[:-1]],
                                          device="cuda"), 0)
        index = torch.randint(0, page, (len(lengths),), generator=gen,
                              device="cuda")[which] + within
        assert most * page > int(index.max())
        slot = pages[first[which] + index // page] * page + index % page
        s["slots"] = torch.cat([slot, slot.new_full((pad,), -1)])
        ct = torch.float8_e4m3fn if c["cache"] == "e4m3" else dt
        shape = (slots // page, hk, page, d) if c["heads_first"] else (slots // page, page, hk, d)
        for name in ("k_cache", "v_cache"):
            full = _randn(gen, *shape).to(ct)
            s[name] = full.transpose(1, 2) if c["heads_first"] else full
        s["q_out"].copy_(_randn(gen, t, hq, d))  # what padding rows keep
        # per-tensor scales of the 8-bit cache
        s["k_scale"], s["v_scale"] = (0.03125, 0.0173) if c["cache"] == "e4m3" else (1.0, 1.0)
    return s


# ---- plain forms: 32 bits, one rounding


def _factor(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _rotate(u, cos, sin, interleaved):
    """u [tokens, heads, head_dim] with the first 2 * cos.shape[-1] elements rotated."""
    half = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = u[..., 0:2 * half:2], u[..., 1:2 * half:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = u[..., :half], u[..., half:2 * half]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, u[..., 2 * half:]], -1)


def _angles(s):
    row = s["table"][s["positions"]]
    half = row.shape[-1] // 2
    return row[:, :half], row[:, half:]


def _plain_heads(x, w, s):
    u = x.float()
    if w is not None:
        u = u * _factor(u) * (w.float() + s["case"]["bias"])
    return _rotate(u, *_angles(s), s["case"]["interleaved"])


def _plain_heads_bwd(dy, x, w, s):
    cos, sin = _angles(s)
    du = _rotate(dy.float(), cos, -sin, s["case"]["interleaved"])
    return _plain_norm_bwd(du, x, w, s["case"]["bias"], (0, 1))


def _plain_norm_bwd(du, x, w, bias, over):
    xf = x.float()
    r = _factor(xf)
    xh = xf * r
    dxh = du * (w.float() + bias)
    dx = r * (dxh - xh * (dxh * xh).mean(-1, keepdim=True))
    return dx.to(x.dtype), (du * xh).sum(over)


def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _plain_append(s):
    c = s["case"]
    live = c["tokens"] - c["padded"]
    norm = c["norm"]
    y = _plain_heads(s["q"], s["qw"] if norm else None, s)
    s["q_out"][:live] = y[:live].to(s["q_out"].dtype)
    kv = (_plain_heads(s["k"], s["kw"] if norm else None, s), s["v"].float())
    slots = s["slots"][:live]
    for name, values, scale in (("k_cache", kv[0], s["k_scale"]), ("v_cache", kv[1], s["v_scale"])):
        cache = s[name]
        if c["cache"] == "e4m3":  # as bytes: indexing by them writes any 8-bit type
            cache, values = cache.view(torch.uint8), _e4m3(values / scale).view(torch.uint8)
        cache[slots // c["page"], slots % c["page"]] = values[:live].to(cache.dtype)
    return s["q_out"], s["k_cache"], s["v_cache"]


def run(state):
    s, c = state, state["case"]
    if own:
        import rmsnorm_fwd_gb300 as rn
        if c["op"] == "rms_bwd":
            return rn.rms_norm_backward(s["dy"], s["x"], s["w"], EPS, weight_bias=c["bias"])
        if c["op"] == "rope":
            return rn.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["table"], s["positions"],
                                   EPS, weight_bias=c["bias"], interleaved=c["interleaved"],
                                   q_out=s["q_out"], k_out=s["k_out"])
        if c["op"] == "rope_bwd":
            return rn.qk_norm_rope_backward(s["dq_out"], s["dk_out"], s["q"], s["k"], s["qw"],
                                            s["kw"], s["table"], s["positions"], EPS,
                                            weight_bias=c["bias"], interleaved=c["interleaved"])
        q_out = rn.qk_norm_rope_append(s["q"], s["k"], s["v"], s["qw"] if c["norm"] else None,
                                       s["kw"] if c["norm"] else None, s["table"],
                                       s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                                       EPS, weight_bias=c["bias"], interleaved=c["interleaved"],
                                       k_scale=s["k_scale"], v_scale=s["v_scale"],
                                       q_out=s["q_out"])
        return q_out, s["k_cache"], s["v_cache"]
    if c["op"] == "rms_bwd":
        return _plain_norm_bwd(s["dy"].float(), s["x"], s["w"], c["bias"], (0,))
    dt = DTYPES[c["dtype"]]
    if c["op"] == "rope":
        return _plain_heads(s["q"], s["qw"], s).to(dt), _plain_heads(s["k"], s["kw"], s).to(dt)
    if c["op"] == "rope_bwd":
        dq, dqw = _plain_heads_bwd(s["dq_out"], s["q"], s["qw"], s)
        dk, dkw = _plain_heads_bwd(s["dk_out"], s["k"], s["kw"], s)
        return dq, dk, dqw, dkw
    return _plain_append(s)


def work(case):
    c = case
    b = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rms_bwd":
        n = c["rows"] * c["hidden"]
        return {"bytes": 3 * n * b + c["hidden"] * (b + 4), "flops": 12 * n}
    t = c["tokens"] - c.get("padded", 0)
    d, rd = c["head_dim"], c["rotary_dim"]
    q, k = t * c["q_heads"] * d, t * c["k_heads"] * d
    rows = t if c["op"] == "append" else max(_lengths(c))  # of the table
    small = 8 * c["tokens"] + 4 * rows * rd + 2 * d * b
    if c["op"] == "rope":
        return {"bytes": 2 * (q + k) * b + small, "flops": 9 * (q + k)}
    if c["op"] == "rope_bwd":
        return {"bytes": 3 * (q + k) * b + small + 8 * d, "flops": 16 * (q + k)}
    cb = 1 if c["cache"] == "e4m3" else b
    return {"bytes": 2 * q * b + 2 * k * (b + cb) + small + 8 * c["tokens"],
            "flops": 9 * (q + k) + k}


# ---- the definition in 64 bits: the rotation as a product of complex numbers, gradients as
# derivatives of the definition


def _exact_heads(x, g, s):
    c = s["case"]
    if g is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * g
    rd = c["rotary_dim"]
    row = s["table"].double().index_select(0, s["positions"]).unsqueeze(1)
    turn = torch.complex(row[..., :rd // 2], row[..., rd // 2:])
    head, rest = x.split([rd, x.shape[-1] - rd], -1)
    pairs = head.unflatten(-1, (rd // 2, 2) if c["interleaved"] else (2, rd // 2))
    along = -1 if c["interleaved"] else -2
    z = torch.complex(pairs.select(along, 0), pairs.select(along, 1)) * turn
    return torch.cat([torch.stack([z.real, z.imag], along).flatten(-2), rest], -1)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "rms_bwd":
        x = s["x"].double().requires_grad_()
        w = s["w"].double().requires_grad_()
        y = x * (w + c["bias"]) / (x.pow(2).sum(-1, keepdim=True) / c["hidden"] + EPS).sqrt()
        return torch.autograd.grad(y, (x, w), s["dy"].double())
    if c["op"] == "rope_bwd":
        leaves = [s[n].double().requires_grad_() for n in ("q", "k", "qw", "kw")]
        q, k, qw, kw = leaves
        ys = (_exact_heads(q, qw + c["bias"], s), _exact_heads(k, kw + c["bias"], s))
        return torch.autograd.grad(ys, leaves, (s["dq_out"].double(), s["dk_out"].double()))
    norm = c.get("norm", True)
    gq, gk = ((s[n].double() + c["bias"]) if norm else None for n in ("qw", "kw"))
    q, k = _exact_heads(s["q"].double(), gq, s), _exact_heads(s["k"].double(), gk, s)
    if c["op"] == "rope":
        return q, k
    q_out = torch.where((s["slots"] < 0)[:, None, None], s["q_out"].double(), q)
    filled = []
    live = s["slots"] >= 0
    for cache, values, scale in ((s["k_cache"], k, s["k_scale"]),
                                 (s["v_cache"], s["v"].double(), s["v_scale"])):
        wide = cache.double()  # keeps the cache's order of dimensions
        if c["cache"] == "e4m3":
            values = (values / scale).clamp(-448.0, 448.0)
        pages = torch.div(s["slots"][live], c["page"], rounding_mode="floor")
        wide.index_put_((pages, s["slots"][live] - pages * c["page"]), values[live])
        filled.append(wide)
    return q_out, filled[0], filled[1]
