"""The 8-bit linear layer and the gated norms around a transformer block: cases, plain forms and exact results.

Four operators, each in every direction it has:

* ``linear``       y = Q(x) Q(W)^T + b, Q the 8-bit format with one scale for each block of 128
* ``linear_grad``  dx = Q(dy) Q(W), dW = Qt(dy)^T Qt(x), db = the sum of dy's rows (Qt: blocks of 128 rows)
* ``norm``         h = alpha x + gate * post(y), n = pre(h) (1 + scale) + shift, over ragged sequences
* ``norm_grad``    the gradients of all inputs of ``norm``

and ``chain``: a norm whose result leaves in the 8-bit format and enters the linear layer as it is.

The 8-bit format: a block of 128 consecutive elements along the contracted axis shares the scale S, the
smallest power of two (at least 2^-126) with max|v| / S <= 448; an element is E4M3(v / S), round to nearest
even.  A weight's blocks are 128 x 128.  Codes: one byte for each element, rows padded with zeros to whole
blocks.  Scales: the byte exponent + 127, in groups of four consecutive blocks, [groups][rows][4], padded
with 127.

``own`` chooses between the plain forms here (elementary torch operations) and the library's kernels.
"""

import torch

own = False

BLOCK = 128
EPS = 1e-6


def listed():
    return [
        # one new token through an up projection of the action expert: a serving step, launch latency and the weight's bytes
        dict(name="linear_one_token", op="linear", M=1, K=1024, N=4096, dtype="bf16", bias=True),
        # the action expert's down projection on its 256 action tokens: one denoising step
        dict(name="linear_action", op="linear", M=256, K=4096, N=1024, dtype="bf16", bias=True),
        # sizes that fill no tile or block, float32 activations and results: calibration runs on ragged batches
        dict(name="linear_ragged_f32", op="linear", M=777, K=1000, N=2056, dtype="f32", bias=False),
        # a wide up projection over a whole prompt or video prefill: bound by the matrix units
        dict(name="linear_prefill", op="linear", M=4096, K=4096, N=14336, dtype="bf16", bias=True),
        # gradients of a small square projection on the 256 action tokens
        dict(name="grad_action", op="linear_grad", M=256, K=1024, N=1024, dtype="bf16", bias=True),
        # gradients at a training batch's size
        dict(name="grad_batch", op="linear_grad", M=8192, K=4096, N=4096, dtype="bf16", bias=True),
        # one token between two blocks: a serving step, launch latency
        dict(name="norm_one_token", op="norm", M=1, C=1024, dtype="bf16", post="rms", pre="rms", mod=False, affine=True, seqs=1, pad=0),
        # a modulated layer norm over eight packed sequences with padding behind the last
        dict(name="norm_packed", op="norm", M=16384, C=4096, dtype="bf16", post="rms", pre="layer", mod=True, affine=True, seqs=8, pad=96),
        # float32 stream, an odd width that no vector load fits
        dict(name="norm_grad_ragged_f32", op="norm_grad", M=1000, C=1001, dtype="f32", post="layer", pre="layer", mod=True, affine=True, seqs=5, pad=7),
        # the gradients of the packed case: a training batch
        dict(name="norm_grad_packed", op="norm_grad", M=16384, C=4096, dtype="bf16", post="rms", pre="rms", mod=True, affine=True, seqs=8, pad=96),
        # four new tokens from one block's end into the next block's up projection: serving
        dict(name="chain_few_tokens", op="chain", M=4, C=1024, N=4096, dtype="bf16", post="rms", pre="rms", mod=False, affine=True, seqs=1, pad=0),
        # the same over a prefill
        dict(name="chain_prefill", op="chain", M=2048, C=4096, N=4096, dtype="bf16", post="none", pre="layer", mod=True, affine=False, seqs=2, pad=0),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm; two in three of them odd or ragged."""
    v = lo * (hi / lo) ** rng.random()
    v = int(v)
    kind = rng.randrange(3)
    if kind == 0 and v > 128:
        v = (v + 127) // 128 * 128
    elif kind == 1:
        v |= 1
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "norm", "norm_grad", "chain"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "linear":
        return dict(op=op, M=_spread(rng, 1, 4096), K=_spread(rng, 64, 4096), N=_spread(rng, 64, 14336), dtype=dtype, bias=rng.random() < 0.5)
    if op == "linear_grad":
        return dict(op=op, M=_spread(rng, 1, 8192), K=_spread(rng, 64, 4096), N=_spread(rng, 64, 4096), dtype=dtype, bias=rng.random() < 0.5)
    seqs = rng.choice([1, 2, 5, 16])
    case = dict(op=op, M=_spread(rng, 1, 2048 if op == "chain" else 16384), C=_spread(rng, 64, 4096), dtype=dtype, post=rng.choice(["none", "rms", "layer"]),
                pre=rng.choice(["rms", "layer"]), mod=rng.random() < 0.5, affine=rng.random() < 0.7, seqs=seqs, pad=0)
    if op == "chain":
        case.update(N=_spread(rng, 64, 4096), dtype="bf16")
    elif case["M"] > 1:
        case["pad"] = rng.randrange(0, min(100, case["M"]))
    return case


# ------------------------------------------------------------------ the inputs


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _power(k):
    """2^k as float32, exactly, for whole k in -126..127."""
    return ((k + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The exponent of the smallest power of two S >= 2^-126 with amax / S <= 448."""
    m, e = torch.frexp(amax)
    e = torch.clamp(torch.where(m <= 0.875, e - 9, e - 8), min=-126)
    return torch.where(amax == 0, -126, e).to(torch.int32)


def _pad(v, rows, cols):
    """v with zeros behind it, up to whole multiples of rows and cols."""
    return torch.nn.functional.pad(v, (0, -v.shape[1] % cols, 0, -v.shape[0] % rows))


def _weight(w):
    """A weight in the 8-bit format, blocks of 128 x 128: codes and scales along its rows, and of its transpose."""
    n, k = w.shape
    p = _pad(w, BLOCK, BLOCK)
    b = p.view(p.shape[0] // BLOCK, BLOCK, p.shape[1] // BLOCK, BLOCK)
    e = _exponent(b.abs().amax(dim=(1, 3)))
    q = (b * _power(-e)[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(p.shape)

    def scales(e, rows):
        s = (e + 127).to(torch.uint8).repeat_interleave(BLOCK, 0)[:rows]
        s = torch.nn.functional.pad(s, (0, -s.shape[1] % 4), value=127)
        return s.view(rows, -1, 4).transpose(0, 1).contiguous()

    return dict(codes=q[:n].contiguous(), scales=scales(e, n), codes_t=q.t()[:k].contiguous(), scales_t=scales(e.t(), k))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = _type(case)

    def normal(*size):
        return torch.randn(size, generator=g, device="cuda")

    def activations(rows, cols):
        # a few channels carry values many times larger, as activations in front of a projection do
        spread = torch.where(torch.rand((cols,), generator=g, device="cuda") < 0.01, 12.0, 1.0)
        return (normal(rows, cols) * spread).to(t)

    M, state = case["M"], dict(case)
    if case["op"] in ("linear", "linear_grad"):
        K, N = case["K"], case["N"]
        state.update(_weight(normal(N, K) / K ** 0.5), x=activations(M, K), b=normal(N) if case["bias"] else None)
        if case["op"] == "linear_grad":
            state["dy"] = (normal(M, N) * 1e-3 * torch.exp(normal(M, 1))).to(t)
        return state
    C, G = case["C"], case["seqs"]
    state.update(x=activations(M, C), y=(normal(M, C) * 3).to(t), alpha=0.9)
    state["post_weight"] = 1 + 0.1 * normal(C) if case["post"] != "none" else None
    state["weight"] = 1 + 0.1 * normal(C) if case["affine"] else None
    state["bias"] = 0.1 * normal(C) if case["affine"] and case["pre"] == "layer" else None
    # one table for each sequence, as a conditioning network gives it: gate, scale and shift side by side
    table = 0.3 * normal(G, 3, C)
    state["gate"] = table[:, 0]
    state["scale"], state["shift"] = (table[:, 1], table[:, 2]) if case["mod"] else (None, None)
    # the sequences' first rows, and the end of the last; some sequences may be empty
    cuts = torch.randint(0, M - case["pad"] + 1, (G - 1,), generator=g, device="cuda").sort().values
    ends = torch.tensor([0, M - case["pad"]], device="cuda")
    state["offsets"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32) if G > 1 or case["pad"] else None
    if case["op"] == "norm":
        state.update(h_out=torch.zeros_like(state["x"]), n_out=torch.zeros_like(state["x"]))
    elif case["op"] == "norm_grad":
        state["h"] = (normal(M, C) * 2 + 0.3).to(t)
        state.update(dh=(normal(M, C) * 1e-2).to(t), dn=(normal(M, C) * 1e-2).to(t), dx_out=torch.zeros_like(state["x"]), dy_out=torch.zeros_like(state["x"]))
    else:
        state.update(_weight(normal(case["N"], C) / C ** 0.5), b=normal(case["N"]))
    return state


# ------------------------------------------------------------ the plain forms


def _rounded(v):
    """float32 rows as the values their 8-bit form stands for, blocks along the row."""
    p = _pad(v, 1, BLOCK)
    b = p.view(p.shape[0], -1, BLOCK)
    e = _exponent(b.abs().amax(dim=2, keepdim=True))
    return ((b * _power(-e)).to(torch.float8_e4m3fn).float() * _power(e)).view(p.shape)[:, :v.shape[1]]


def _values(codes, scales, cols):
    """The values of a weight in the 8-bit format."""
    e = scales.transpose(0, 1).reshape(codes.shape[0], -1)[:, :codes.shape[1] // BLOCK].to(torch.int32) - 127
    v = codes.view(torch.float8_e4m3fn).float().view(codes.shape[0], -1, BLOCK) * _power(e)[:, :, None]
    return v.view(codes.shape)[:, :cols]


def _linear(x, s, K):
    y = _rounded(x.float()) @ _values(s["codes"], s["scales"], K).t()
    return y if s["b"] is None else y + s["b"]


def _rows(s, M):
    """[G, M] of 0 and 1: which rows are whose.  A row behind the last sequence is nobody's."""
    if s["offsets"] is None:
        return torch.ones((1, M), device="cuda")
    row, o = torch.arange(M, device="cuda"), s["offsets"]
    return ((row >= o[:-1, None]) & (row < o[1:, None])).float()


def _statistics(v, kind):
    """(normed rows, 1 / their deviation)"""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * r, r


def _norm(s):
    x, y = s["x"].float(), s["y"].float()
    rows = _rows(s, s["M"])
    if s["post"] != "none":
        y = _statistics(y, s["post"])[0] * s["post_weight"]
    # the stream is kept in its own type, and the next norm reads it so
    h = (s["alpha"] * x + (rows.t() @ s["gate"]) * y).to(s["x"].dtype)
    n = _statistics(h.float(), s["pre"])[0]
    if s["weight"] is not None:
        n = n * s["weight"]
    if s["bias"] is not None:
        n = n + s["bias"]
    if s["scale"] is not None:
        n = n * (1 + rows.t() @ s["scale"]) + rows.t() @ s["shift"]
    valid = rows.sum(0)[:, None] > 0
    return h.where(valid, h * 0), n.where(valid, n * 0)


def _norm_grad(s):
    y, h, dh, dn = s["y"].float(), s["h"].float(), s["dh"].float(), s["dn"].float()
    rows = _rows(s, s["M"])
    valid = rows.sum(0)[:, None] > 0
    out = {}

    def back(g, v, r, kind):
        g = g - v * (g * v).mean(1, keepdim=True) if kind == "rms" else g - g.mean(1, keepdim=True) - v * (g * v).mean(1, keepdim=True)
        return g * r

    v, r = _statistics(h, s["pre"])
    w = torch.ones_like(h[0]) if s["weight"] is None else s["weight"]
    m = torch.ones_like(h) if s["scale"] is None else 1 + rows.t() @ s["scale"]
    if s["scale"] is not None:
        out["scale"] = rows @ (dn * (v * w if s["bias"] is None else v * w + s["bias"]))
        out["shift"] = rows @ dn
    if s["weight"] is not None:
        out["weight"] = (rows @ (dn * m * v)).sum(0)
    if s["bias"] is not None:
        out["bias"] = (rows @ (dn * m)).sum(0)
    dh = dh + back(dn * m * w, v, r, s["pre"])
    out["dx"] = (s["alpha"] * dh).where(valid, dh * 0).to(s["h"].dtype)
    g = rows.t() @ s["gate"]
    if s["post"] == "none":
        out["gate"] = rows @ (dh * y)
        dy = dh * g
    else:
        v, r = _statistics(y, s["post"])
        out["gate"] = rows @ (dh * v * s["post_weight"])
        out["post_weight"] = (rows @ (dh * g * v)).sum(0)
        dy = back(dh * g * s["post_weight"], v, r, s["post"])
    out["dy"] = dy.where(valid, dy * 0).to(s["h"].dtype)
    return out


def _plain(s):
    if s["op"] == "linear":
        return _linear(s["x"], s, s["K"]).to(s["x"].dtype)
    if s["op"] == "linear_grad":
        x, dy = s["x"].float(), s["dy"].float()
        dx = _rounded(dy) @ _values(s["codes"], s["scales"], s["K"])
        dw = _rounded(dy.t().contiguous()) @ _rounded(x.t().contiguous()).t()
        return dict(dx=dx.to(s["x"].dtype), dw=dw, db=None if s["b"] is None else dy.sum(0))
    if s["op"] == "norm_grad":
        return _norm_grad(s)
    h, n = _norm(s)
    if s["op"] == "norm":
        return dict(h=h, n=n.to(s["x"].dtype))
    return dict(h=h, y=_linear(n, s, s["C"]).to(s["x"].dtype))


# --------------------------------------------------------- the library's calls


def _own(s):
    from wam_asp_w4a4_amd.fp8 import Fp8Layer
    from wam_asp_w4a4_amd.norm import gated_norm, gated_norm_backward

    if s["op"] in ("linear", "linear_grad", "chain"):
        layer = Fp8Layer(s["N"], s["C"] if s["op"] == "chain" else s["K"], s["codes"], s["scales"], s["codes_t"], s["scales_t"], s["b"])
    if s["op"] == "linear":
        return layer.forward(s["x"], s["dtype"])
    if s["op"] == "linear_grad":
        dx, dw, db = layer.backward(s["dy"], s["x"])
        return dict(dx=dx, dw=dw, db=db)
    spec = dict(alpha=s["alpha"], post=s["post"], post_weight=s["post_weight"], gate=s["gate"], pre=s["pre"], weight=s["weight"], bias=s["bias"],
                scale=s["scale"], shift=s["shift"], offsets=s["offsets"], eps=EPS)
    if s["op"] == "norm":
        h, n = gated_norm(s["x"], s["y"], h=s["h_out"], n=s["n_out"], **spec)
        return dict(h=h, n=n)
    if s["op"] == "norm_grad":
        g = gated_norm_backward(s["dh"], s["dn"], s["h"], s["y"], dx=s["dx_out"], dy=s["dy_out"], **spec)
        return {k: v for k, v in g._asdict().items() if v is not None}
    h, n = gated_norm(s["x"], s["y"], out="fp8", **spec)
    return dict(h=h, y=layer.forward(n, s["dtype"]))


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    M = case["M"] - case.get("pad", 0)
    if case["op"] in ("linear", "linear_grad"):
        K, N = case["K"], case["N"]
        weight = N * K + N * K // BLOCK
        if case["op"] == "linear":
            return dict(bytes=weight + e * M * (K + N) + 4 * N * case["bias"], flops=2 * M * N * K)
        return dict(bytes=weight + e * M * (2 * K + N) + 4 * N * K + 4 * N, flops=4 * M * N * K)
    C, G = case["C"], case["seqs"]
    tables = 4 * C * ((case["post"] != "none") + case["affine"] * (2 if case["pre"] == "layer" else 1) + G * (3 if case["mod"] else 1))
    if case["op"] == "norm":
        return dict(bytes=4 * e * M * C + tables, flops=20 * M * C)
    if case["op"] == "norm_grad":
        return dict(bytes=6 * e * M * C + 2 * tables, flops=40 * M * C)
    N = case["N"]
    return dict(bytes=3 * e * M * C + e * M * N + tables + N * C + N * C // BLOCK + 4 * N, flops=2 * M * N * C + 20 * M * C)


# ------------------------------------------------------ the results in 64 bits


def _e4m3(v):
    """v on the E4M3 grid: four significant bits down to 2^-6, steps of 2^-9 below."""
    top = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20)))
    step = torch.exp2(top.clamp(min=-6.0) - 3)
    return torch.round(v / step) * step


def _held(v):
    """64-bit rows as their 8-bit form holds them.  The scale's exponent comes from comparisons, not from a logarithm's last bits."""
    rows, cols = v.shape
    out = torch.zeros((rows, (cols + 127) // 128, 128), dtype=torch.float64, device=v.device)
    out.view(rows, -1)[:, :cols] = v
    top = out.abs().max(2, keepdim=True).values
    k = torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -140)))
    k = k + (top > 448 * torch.exp2(k)).double()
    k = k - (top <= 448 * torch.exp2(k - 1)).double()
    unit = torch.exp2(k.clamp(min=-126.0))
    return (_e4m3(out / unit) * unit).view(rows, -1)[:, :cols]


def _weight64(s, cols):
    code = s["codes"].to(torch.int64)
    exponent, fraction = (code >> 3) & 15, (code & 7).double()
    value = torch.where(exponent == 0, fraction * 2.0 ** -9, (8 + fraction) * torch.exp2(exponent.double() - 10))
    value = torch.where(code >= 128, -value, value)
    scale = torch.exp2(s["scales"].permute(1, 0, 2).flatten(1).double() - 127)[:, :code.shape[1] // 128]
    return (value * scale.repeat_interleave(128, dim=1))[:, :cols]


def _normed64(v, kind):
    centre = v.mean(1, keepdim=True) if kind == "layer" else 0.0
    return (v - centre) / torch.sqrt(((v - centre) ** 2).mean(1, keepdim=True) + EPS)


def _stream64(s, x, y, gate, post_weight):
    """(alpha x + gate * post(y)), the rows of one sequence"""
    if s["post"] != "none":
        y = _normed64(y, s["post"]) * post_weight
    return s["alpha"] * x + gate * y


def _pre64(s, h, weight, bias, scale, shift):
    n = _normed64(h, s["pre"])
    n = n if weight is None else n * weight
    n = n if bias is None else n + bias
    return n if scale is None else n * (1 + scale) + shift


def exact(case, seed):
    s = prepare(case, seed)

    def wide(v):
        return None if v is None else v.double()

    if case["op"] == "linear":
        y = _held(s["x"].double()) @ _weight64(s, case["K"]).t()
        return y if s["b"] is None else y + s["b"].double()
    if case["op"] == "linear_grad":
        dy = s["dy"].double()
        return dict(dx=_held(dy) @ _weight64(s, case["K"]), dw=_held(dy.t()) @ _held(s["x"].double().t()).t(), db=None if s["b"] is None else dy.sum(0))
    o = [0, case["M"]] if s["offsets"] is None else s["offsets"].tolist()
    x, y = s["x"].double(), s["y"].double()
    if case["op"] == "norm_grad":
        h, dh, dn = s["h"].double(), s["dh"].double(), s["dn"].double()
        names = [k for k in ("post_weight", "weight", "bias") if s[k] is not None]
        shared = {k: s[k].double().requires_grad_() for k in names}
        out = dict(dx=torch.zeros_like(h), dy=torch.zeros_like(h), gate=torch.zeros_like(s["gate"]).double())
        out.update({k: torch.zeros_like(v) for k, v in shared.items()})
        tables = ["gate"] if s["scale"] is None else ["gate", "scale", "shift"]
        out.update({k: torch.zeros_like(s[k]).double() for k in tables})
        for g in range(case["seqs"]):
            at = slice(o[g], o[g + 1])
            if o[g] == o[g + 1]:
                continue
            # the gradients of <n, dn> + <h, dh> by differentiating the definition
            stream, branch = h[at].clone().requires_grad_(), y[at].clone().requires_grad_()
            mine = {k: s[k][g].double().requires_grad_() for k in tables}
            n = _pre64(s, stream, shared.get("weight"), shared.get("bias"), mine.get("scale"), mine.get("shift"))
            found = dict(zip(["h"] + names + tables, torch.autograd.grad((n * dn[at]).sum(), [stream] + list(shared.values()) + list(mine.values()), allow_unused=True)))
            total = found["h"] + dh[at]
            h2 = _stream64(s, 0.0, branch, mine["gate"], shared.get("post_weight"))
            second = dict(zip(["y"] + names + tables, torch.autograd.grad((h2 * total).sum(), [branch] + list(shared.values()) + list(mine.values()), allow_unused=True)))
            out["dx"][at], out["dy"][at] = s["alpha"] * total, second["y"]
            for f in (found, second):
                for k in names:
                    out[k] += 0 if f[k] is None else f[k]
                for k in tables:
                    out[k][g] += 0 if f[k] is None else f[k]
        return out
    h, n = torch.zeros_like(x), torch.zeros_like(x)
    for g in range(case["seqs"]):
        at = slice(o[g], o[g + 1])
        if o[g] < o[g + 1]:
            h[at] = _stream64(s, x[at], y[at], s["gate"][g].double(), wide(s["post_weight"])).to(s["x"].dtype).double()
            n[at] = _pre64(s, h[at], wide(s["weight"]), wide(s["bias"]), None if s["scale"] is None else s["scale"][g].double(),
                           None if s["shift"] is None else s["shift"][g].double())
    if case["op"] == "norm":
        return dict(h=h, n=n)
    return dict(h=h, y=_held(n) @ _weight64(s, case["C"]).t() + s["b"].double())
