"""The attention of a transformer block: cases, plain forms and exact results.

Three operators, in a block's order:

* ``heads``   the norm of each head of the queries and keys, and their position rotation
              (``heads_grad``: its gradients)
* ``attend``  o = softmax(scale q k^T) v of packed sequences whose queries and keys differ in number, with
              shared heads and masked keys (``attend_grad``: its gradients)
* ``cache``   the same over keys and values held in 4 bits: E2M1 elements, an E4M3 scale for each 16 of a head
              (``store``: new tokens into such a cache, and the cache's values)

The 4-bit format: S = E4M3(max|v| / 6) over 16 consecutive elements, round to nearest even, at most 448; an element
is E2M1(|v| / S), ties to the even code, with v's sign.  Two codes a byte, the even element in the low half.

``own`` chooses between the plain forms here (elementary torch operations) and the library's kernels.
"""

import random

import torch

own = False

EPS = 1e-6
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MASKED = 0.25  # share of the keys that a mask leaves out


def listed():
    return [
        # one new token: a serving step, launch latency
        dict(name="heads_one_token", op="heads", T=1, Hq=16, Hk=16, D=64, rot=64, pairs=True, norm="rms", dtype="bf16", pad=0),
        # a prefill with shared key heads, padding tokens at its end
        dict(name="heads_prefill", op="heads", T=16384, Hq=32, Hk=8, D=128, rot=128, pairs=True, norm="rms", dtype="bf16", pad=100),
        # float32, odd counts, heads rotated in part: calibration
        dict(name="heads_grad_ragged_f32", op="heads_grad", T=1001, Hq=6, Hk=2, D=80, rot=40, pairs=False, norm="layer", dtype="f32", pad=13),
        # a training batch
        dict(name="heads_grad_batch", op="heads_grad", T=8192, Hq=32, Hk=8, D=128, rot=128, pairs=False, norm="rms", dtype="bf16", pad=0),
        # the action expert's 256 tokens over an encoder's 512 states: one denoising step
        dict(name="attend_action", op="attend", Tq=256, Tk=512, Hq=16, Hk=16, D=64, dtype="bf16", seqs=1, pad=0, mask=False),
        # float32, a head size and lengths that fill no tile, masked keys, padding rows: calibration on ragged batches
        dict(name="attend_ragged_f32", op="attend", Tq=777, Tk=1234, Hq=8, Hk=2, D=80, dtype="f32", seqs=5, pad=9, mask=True),
        # a whole video's tokens: bound by the matrix units
        dict(name="attend_prefill", op="attend", Tq=8192, Tk=8192, Hq=16, Hk=16, D=128, dtype="bf16", seqs=1, pad=0, mask=False),
        # gradients of the action expert's step
        dict(name="attend_grad_action", op="attend_grad", Tq=256, Tk=512, Hq=16, Hk=16, D=64, dtype="bf16", seqs=1, pad=0, mask=False),
        # gradients at a training batch's size: packed sequences, shared heads, padded encoder states
        dict(name="attend_grad_batch", op="attend_grad", Tq=8192, Tk=8192, Hq=16, Hk=4, D=128, dtype="bf16", seqs=4, pad=50, mask=True),
        # eight requests' prompts enter the cache, which is read back
        dict(name="store_prompts", op="store", T=6000, rows=8192, Hk=8, D=128, dtype="bf16", seqs=8),
        # one new token of each of eight requests over their caches: bound by the cache's bytes
        dict(name="cache_one_token", op="cache", Tq=8, Tk=131072, Hq=32, Hk=8, D=128, dtype="bf16", seqs=8, pad=0, mask=False),
        # the action expert's tokens over the video's cached ones: one denoising step
        dict(name="cache_action", op="cache", Tq=256, Tk=4096, Hq=16, Hk=16, D=64, dtype="bf16", seqs=1, pad=0, mask=False),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm; a third of them odd, a third multiples of 64."""
    v = int(lo * (hi / lo) ** rng.random())
    kind = rng.randrange(3)
    if kind == 0 and v > 64:
        v = v // 64 * 64
    elif kind == 1:
        v |= 1
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["heads", "heads_grad", "attend", "attend", "attend_grad", "cache", "store"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hq, Hk = rng.choice([(1, 1), (8, 8), (16, 16), (8, 2), (32, 8), (12, 4), (8, 1), (6, 2)])
    if op in ("heads", "heads_grad"):
        T, D = _spread(rng, 1, 8192), rng.choice([32, 64, 72, 80, 96, 128, 128])
        return dict(op=op, T=T, Hq=Hq, Hk=Hk, D=D, rot=rng.choice([D, D, D // 2]), pairs=rng.random() < 0.5, norm=rng.choice(["rms", "rms", "layer", "none"]),
                    dtype=dtype, pad=rng.randrange(0, min(T, 50)) if rng.random() < 0.5 else 0)
    if op == "store":
        T = _spread(rng, 1, 6000)
        return dict(op=op, T=T, rows=T + rng.randrange(0, 2000), Hk=Hk, D=rng.choice([32, 64, 80, 96, 128]), dtype=dtype, seqs=rng.choice([1, 2, 8]))
    Tq, Tk, D = _spread(rng, 1, 8192), _spread(rng, 1, 8192), rng.choice([32, 64, 64, 80, 96, 128, 128])
    # at most the work of the largest listed ones of the type
    while Tq * Tk * Hq * D > (2 ** 37 if dtype == "bf16" else 2 ** 33) // (2 if op == "attend_grad" else 1):
        Tq, Tk = (Tq // 2 + 1, Tk) if Tq > Tk else (Tq, Tk // 2 + 1)
    return dict(op=op, Tq=Tq, Tk=Tk, Hq=Hq, Hk=Hk, D=D, dtype=dtype, seqs=rng.choice([1, 1, 2, 5]), pad=rng.randrange(0, min(Tq, 20)) if rng.random() < 0.3 else 0,
                mask=rng.random() < 0.4)


# ------------------------------------------------------------------ the inputs


def _cuts(total, parts):
    """The first rows of `parts` sequences that share `total` rows, and the end of the last.  Of several, some may be empty."""
    if total == parts:
        return list(range(parts + 1))
    rng = random.Random(31 * total + parts)
    return [0] + sorted(rng.randrange(total + 1) for _ in range(parts - 1)) + [total]


def _pairs(case):
    """How many pairs of a query and a key there are."""
    q, k = _cuts(case["Tq"] - case["pad"], case["seqs"]), _cuts(case["Tk"], case["seqs"])
    return sum((q[g + 1] - q[g]) * (k[g + 1] - k[g]) for g in range(case["seqs"]))


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _quantised(v):
    """float32 (..., D) in 4 bits: codes (..., D / 2), scales (..., D / 16), bytes."""
    b = v.unflatten(-1, (-1, 16))
    scale = (b.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
    s, a = scale.float(), b.abs()
    # each step of the grid: a tie goes to the even code; the borders times the scale are exact
    code = (a > 0.25 * s).int() + (a >= 0.75 * s) + (a > 1.25 * s) + (a >= 1.75 * s) + (a > 2.5 * s) + (a >= 3.5 * s) + (a > 5 * s)
    code = torch.where(s > 0, code, 0) + 8 * torch.signbit(b).int()
    code = code.flatten(-2).unflatten(-1, (-1, 2))
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8), scale.view(torch.uint8).squeeze(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t, op, state = _type(case), case["op"], dict(case)

    def normal(*size):
        return torch.randn(size, generator=g, device="cuda")

    if op in ("heads", "heads_grad"):
        T, Hq, Hk, D, rot = (case[n] for n in ("T", "Hq", "Hk", "D", "rot"))
        # queries, keys and values as one projection leaves them
        qkv = ((normal(T, Hq + 2 * Hk, D) + 0.1) * 2).to(t)
        state.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk])
        state["q_weight"], state["k_weight"] = (None, None) if case["norm"] == "none" else (1 + 0.1 * normal(D), 1 + 0.1 * normal(D))
        # positions within longer texts; padding tokens have none
        angle = torch.arange(2 * T + 64, device="cuda").double()[:, None] * torch.exp2(torch.arange(rot // 2, device="cuda").double() * (-26.0 / rot))
        state.update(cos=torch.cos(angle).float(), sin=torch.sin(angle).float())
        first = int(torch.randint(0, T + 64, (1,), generator=g, device="cuda"))
        state["positions"] = torch.arange(first, first + T, dtype=torch.int32, device="cuda")
        state["positions"][T - case["pad"]:] = -1
        if op == "heads_grad":
            state.update(dq=(normal(T, Hq, D) * 1e-2).to(t), dk=(normal(T, Hk, D) * 1e-2).to(t))
        return state

    G = case["seqs"]
    if op == "store":
        T, rows, Hk, D = (case[n] for n in ("T", "rows", "Hk", "D"))
        kv = normal(T, 2, Hk, D).to(t)
        state.update(k=kv[:, 0], v=kv[:, 1])
        held = [_quantised(normal(rows, Hk, D)) for _ in range(2)]
        state.update(k_codes=held[0][0], k_scales=held[0][1], v_codes=held[1][0], v_scales=held[1][1])
        # each request's rows of the cache, how many of them it has used, and its new tokens: what does not fit is dropped
        slabs, new = _cuts(rows, G), _cuts(T, G)
        used = [(slabs[i + 1] - slabs[i]) // 8 for i in range(G)]
        state.update(slabs=slabs, new=new, used=used, offsets=torch.tensor(new, dtype=torch.int32, device="cuda"),
                     kv_offsets=torch.tensor(slabs, dtype=torch.int32, device="cuda"), kv_lengths=torch.tensor(used, dtype=torch.int32, device="cuda"))
        return state

    Tq, Tk, Hq, Hk, D = (case[n] for n in ("Tq", "Tk", "Hq", "Hk", "D"))
    state["q"] = (normal(Tq, Hq, D) * 1.5).to(t)
    if op == "cache":
        k, v = _quantised(normal(Tk, Hk, D)), _quantised(normal(Tk, Hk, D))
        state.update(k_codes=k[0], k_scales=k[1], v_codes=v[0], v_scales=v[1])
    else:
        kv = normal(Tk, 2, Hk, D).to(t)
        state.update(k=kv[:, 0], v=kv[:, 1])
    packed = G > 1 or case["pad"] > 0
    state["q_cuts"], state["k_cuts"] = _cuts(Tq - case["pad"], G), _cuts(Tk, G)
    for name, cuts in (("q_offsets", "q_cuts"), ("kv_offsets", "k_cuts")):
        state[name] = torch.tensor(state[cuts], dtype=torch.int32, device="cuda") if packed else None
    state["mask"] = torch.rand((Tk,), generator=g, device="cuda") >= MASKED if case["mask"] else None
    if op == "attend_grad":
        state["do"] = normal(Tq, Hq, D).to(t)
        # what the forward pass left
        o, state["lse"] = _attend(state, state["k"].float(), state["v"].float())
        state["o"] = o.to(t)
    return state


# ------------------------------------------------------------ the plain forms


def _normed(x, kind):
    """(normed heads, 1 / their deviation)"""
    if kind == "none":
        return x, None
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _turned(x, c, s, rot, pairs):
    """The first `rot` elements of each head as pairs, turned by the angles of c and s."""
    y = x.clone()
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, a * s + b * c
    return y


def _heads(s):
    live = (s["positions"] >= 0)[:, None, None]
    at = s["positions"].clamp(min=0).long()
    c, d = s["cos"][at][:, None], s["sin"][at][:, None]
    out = {}
    for n in "qk":
        x, w = s[n].float(), s[n + "_weight"]
        y = _normed(x, s["norm"])[0]
        y = _turned(y if w is None else y * w, c, d, s["rot"], s["pairs"])
        out[n] = torch.where(live, y, 0.0).to(s[n].dtype)
    return out


def _heads_grad(s):
    live = (s["positions"] >= 0)[:, None, None]
    at = s["positions"].clamp(min=0).long()
    c, d = s["cos"][at][:, None], s["sin"][at][:, None]
    out = {}
    for n in "qk":
        x, w, dy = s[n].float(), s[n + "_weight"], torch.where(live, s["d" + n].float(), 0.0)
        g = _turned(dy, c, -d, s["rot"], s["pairs"])
        v, r = _normed(x, s["norm"])
        if w is not None:
            out[n + "_weight"] = (g * v).sum((0, 1))
            g = g * w
        if r is not None:
            g = r * (g - v * (g * v).mean(-1, keepdim=True) - (g.mean(-1, keepdim=True) if s["norm"] == "layer" else 0.0))
        out["d" + n] = torch.where(live, g, 0.0).to(s[n].dtype)
    return out


def _values(codes, scales):
    """float32 (..., D) of a cache's bytes."""
    table = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _scores(s, g, q, k):
    """Sequence g's rows of q, rows of k, and scale q k^T of them, (Hk, shared heads * queries, keys), and which keys count."""
    a, b = slice(s["q_cuts"][g], s["q_cuts"][g + 1]), slice(s["k_cuts"][g], s["k_cuts"][g + 1])
    score = torch.bmm(_by_head(q[a], s["Hk"]), k[b].permute(1, 2, 0).contiguous()) * s["D"] ** -0.5
    live = None if s["mask"] is None else s["mask"][b]
    return a, b, score, live


def _by_head(x, heads):
    """(T, H, D) as (heads, H / heads * T, D)"""
    return x.unflatten(1, (heads, -1)).permute(1, 2, 0, 3).flatten(1, 2).contiguous()


def _by_token(x, tokens):
    """Back: (heads, n * T, D) as (T, heads * n, D)"""
    return x.unflatten(1, (-1, max(tokens, 1))).permute(2, 0, 1, 3).flatten(1, 2)


def _attend(s, k, v):
    q = s["q"].float()
    o, lse = torch.zeros_like(q), torch.full(q.shape[:2], -torch.inf, device=q.device)
    for g in range(s["seqs"]):
        a, b, score, live = _scores(s, g, q, k)
        n = a.stop - a.start
        if n == 0 or b.stop == b.start:
            continue
        if live is not None:
            score = score.masked_fill(~live, -torch.inf)
        top = score.amax(-1, keepdim=True).clamp(min=-1e30)  # a row without a key has no weights, not NaN
        p = torch.exp(score - top)
        total = p.sum(-1, keepdim=True)
        y = torch.bmm(p, v[b].transpose(0, 1).contiguous()) / torch.where(total > 0, total, 1.0)
        o[a] = _by_token(y, n)
        lse[a] = _by_token(torch.where(total > 0, top + torch.log(total), -torch.inf), n)[..., 0]
    return o, lse


def _attend_grad(s):
    q, k, v, o, do = (s[n].float() for n in ("q", "k", "v", "o", "do"))
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for g in range(s["seqs"]):
        a, b, score, live = _scores(s, g, q, k)
        n = a.stop - a.start
        if n == 0 or b.stop == b.start:
            continue
        lse = _by_head(s["lse"][a][..., None], s["Hk"])
        p = torch.exp(score - lse.clamp(min=-1e30))
        p = p if live is None else p.masked_fill(~live, 0.0)
        y, dy = _by_head(o[a], s["Hk"]), _by_head(do[a], s["Hk"])
        ds = torch.bmm(dy, v[b].permute(1, 2, 0).contiguous())
        ds = p * (ds - (y * dy).sum(-1, keepdim=True)) * s["D"] ** -0.5
        dq[a] = _by_token(torch.bmm(ds, k[b].transpose(0, 1).contiguous()), n)
        dk[b] = torch.bmm(ds.transpose(1, 2).contiguous(), _by_head(q[a], s["Hk"])).transpose(0, 1)
        dv[b] = torch.bmm(p.transpose(1, 2).contiguous(), dy).transpose(0, 1)
    return dict(dq=dq.to(s["q"].dtype), dk=dk.to(s["q"].dtype), dv=dv.to(s["q"].dtype))


def _store(s):
    out = {}
    for n in "kv":
        held = _values(s[n + "_codes"], s[n + "_scales"])
        new = _values(*_quantised(s[n].float()))
        for g in range(s["seqs"]):
            to = s["slabs"][g] + s["used"][g]
            count = min(s["new"][g + 1] - s["new"][g], s["slabs"][g + 1] - to)
            held[to:to + count] = new[s["new"][g]:s["new"][g] + count]
        out[n] = held.to(torch.bfloat16)
    return out


def _plain(s):
    if s["op"] == "heads":
        return _heads(s)
    if s["op"] == "heads_grad":
        return _heads_grad(s)
    if s["op"] == "attend":
        return _attend(s, s["k"].float(), s["v"].float())[0].to(s["q"].dtype)
    if s["op"] == "attend_grad":
        return _attend_grad(s)
    if s["op"] == "cache":
        return _attend(s, _values(s["k_codes"], s["k_scales"]), _values(s["v_codes"], s["v_scales"]))[0].to(s["q"].dtype)
    return _store(s)


# --------------------------------------------------------- the library's calls


def _own(s):
    from wam_asp_w4a4_amd.attention import Nvfp4Cache, attention, attention_backward
    from wam_asp_w4a4_amd.heads import head_norm, head_norm_backward

    if s["op"] in ("heads", "heads_grad"):
        spec = dict(norm=s["norm"], q_weight=s["q_weight"], k_weight=s["k_weight"], cos=s["cos"], sin=s["sin"], positions=s["positions"],
                    layout="pairs" if s["pairs"] else "halves", eps=EPS)
        if s["op"] == "heads":
            q, k = head_norm(s["q"], s["k"], **spec)
            return dict(q=q, k=k)
        g = head_norm_backward(s["dq"], s["dk"], s["q"], s["k"], **spec)
        return {n: v for n, v in g._asdict().items() if v is not None}
    if s["op"] in ("cache", "store"):
        cache = Nvfp4Cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
        if s["op"] == "store":
            cache.store(s["k"], s["v"], offsets=s["offsets"], kv_offsets=s["kv_offsets"], kv_lengths=s["kv_lengths"])
            k, v = cache.dequantize("bf16")
            return dict(k=k, v=v)
    spec = dict(q_offsets=s["q_offsets"], kv_offsets=s["kv_offsets"], key_mask=s["mask"])
    if s["op"] == "cache":
        return attention(s["q"], cache, **spec)[0]
    if s["op"] == "attend":
        return attention(s["q"], s["k"], s["v"], **spec)[0]
    g = attention_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], **spec)
    return dict(dq=g.dq, dk=g.dk, dv=g.dv)


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, D, Hk = case["op"], case["D"], case["Hk"]
    if op in ("heads", "heads_grad"):
        values = (case["T"] - case["pad"]) * (case["Hq"] + Hk) * D
        return dict(bytes=(2 if op == "heads" else 3) * e * values + 4 * case["T"] * case["rot"], flops=(10 if op == "heads" else 20) * values)
    if op == "store":
        # read, held, read back
        return dict(bytes=2 * case["T"] * Hk * D * (e + 9 / 16) + 2 * case["rows"] * Hk * D * (2 + 9 / 16), flops=20 * case["T"] * Hk * D)
    share = 1 - MASKED if case["mask"] else 1
    queries, keys = e * (case["Tq"] - case["pad"]) * case["Hq"] * D, 2 * share * case["Tk"] * Hk * D
    flops = D * case["Hq"] * _pairs(case) * share
    if op == "attend_grad":
        return dict(bytes=4 * queries + 2 * e * keys, flops=10 * flops)
    return dict(bytes=2 * queries + (9 / 16 if op == "cache" else e) * keys, flops=4 * flops)


# ------------------------------------------------------ the results in 64 bits


def _sequence(cuts, total):
    """Which sequence each of `total` rows belongs to, -1 for none."""
    rows = torch.full((total,), -1, dtype=torch.int64, device="cuda")
    for g in range(len(cuts) - 1):
        rows[cuts[g]:cuts[g + 1]] = g
    return rows


def _rotated64(x, s, at):
    rot, turn = s["rot"], torch.complex(s["cos"].double()[at], s["sin"].double()[at])[:, None]
    head, rest = x[..., :rot], x[..., rot:]
    head = head.unflatten(-1, (-1, 2)) if s["pairs"] else head.unflatten(-1, (2, -1)).transpose(-1, -2)
    head = torch.view_as_real(torch.complex(head[..., 0], head[..., 1]) * turn)
    head = head.flatten(-2) if s["pairs"] else head.transpose(-1, -2).flatten(-2)
    return torch.cat([head, rest], -1)


def _heads64(s, x, w, at):
    if s["norm"] == "layer":
        x = x - x.sum(-1, keepdim=True) / s["D"]
    if s["norm"] != "none":
        x = x * ((x ** 2).sum(-1, keepdim=True) / s["D"] + EPS) ** -0.5 * w
    return _rotated64(x, s, at)


def _attend64(q, k, v, allowed, scale):
    """One head's rows."""
    score = (q @ k.t() * scale).masked_fill(~allowed, -torch.inf)
    some = allowed.any(1)
    weights = torch.zeros_like(score)
    weights[some] = torch.softmax(score[some], 1)
    return weights @ v


def _cache64(codes, scales):
    """A cache's values by the formats' fields: a sign, two exponent bits, a fraction bit; and four bits and three."""
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int64)
    e, m = (code >> 1) & 3, (code & 1).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1)) * (1 - 2 * (code >> 3))
    b = scales.to(torch.int64)
    e, m = b >> 3, (b & 7).double()
    return v * torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10)).repeat_interleave(16, -1)


def _held64(v):
    """v as 4 bits hold it, by distances: the nearest of the format's values, of two equally near the one with the even code."""
    def nearest(a, grid):
        """Indices; a and grid in 64 bits, the distances exact."""
        i = torch.searchsorted(grid, a).clamp(1, len(grid) - 1)
        low, high = a - grid[i - 1], grid[i] - a
        return torch.where((low < high) | ((low == high) & (i % 2 == 1)), i - 1, i)

    b = v.unflatten(-1, (-1, 16))
    codes = torch.arange(127, device=v.device)
    scales = _cache64(torch.zeros((127, 8), dtype=torch.uint8, device=v.device) + 0x22, codes.to(torch.uint8)[:, None])[:, 0]
    s = scales[nearest(b.abs().amax(-1) / 6, scales)][..., None]
    grid = torch.tensor(GRID, dtype=torch.float64, device=v.device)
    code = nearest(b.abs() / s.clamp(min=1e-30), grid)
    return (torch.where(s > 0, grid[code], 0.0) * s * torch.sign(b)).flatten(-2)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("heads", "heads_grad"):
        live, out = s["positions"] >= 0, {}
        at = s["positions"][live].long()
        for n in "qk":
            x = s[n][live].double().requires_grad_(op == "heads_grad")
            w = None if s[n + "_weight"] is None else s[n + "_weight"].double().requires_grad_(op == "heads_grad")
            y = _heads64(s, x, w, at)
            full = torch.zeros(s[n].shape, dtype=torch.float64, device="cuda")
            if op == "heads":
                full[live] = y
                out[n] = full
                continue
            found = torch.autograd.grad((y * s["d" + n][live]).sum(), [x] if w is None else [x, w])
            full[live] = found[0]
            if w is not None:
                out[n + "_weight"] = found[1]
            out["d" + n] = full
        return out
    if op == "store":
        out = {}
        for n in "kv":
            out[n] = _cache64(s[n + "_codes"], s[n + "_scales"])
            new = _held64(s[n].double())
            for g in range(case["seqs"]):
                for i in range(s["new"][g + 1] - s["new"][g]):
                    to = s["slabs"][g] + s["used"][g] + i
                    if to < s["slabs"][g + 1]:
                        out[n][to] = new[s["new"][g] + i]
        return out
    if case["Tq"] * case["Tk"] * case["Hq"] > 2 ** 31:
        return None
    if op == "cache":
        k, v = _cache64(s["k_codes"], s["k_scales"]), _cache64(s["v_codes"], s["v_scales"])
    else:
        k, v = s["k"].double(), s["v"].double()
    allowed = _sequence(s["q_cuts"], case["Tq"])[:, None] == _sequence(s["k_cuts"], case["Tk"])[None, :]
    if s["mask"] is not None:
        allowed &= s["mask"]
    q, group = s["q"].double(), case["Hq"] // case["Hk"]
    grad = op == "attend_grad"
    out = [torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)]
    for h in range(case["Hq"]):
        own_q, own_k, own_v = (t.contiguous().requires_grad_(grad) for t in (q[:, h], k[:, h // group], v[:, h // group]))
        o = _attend64(own_q, own_k, own_v, allowed, case["D"] ** -0.5)
        if not grad:
            out[0][:, h] = o
            continue
        found = torch.autograd.grad((o * s["do"][:, h]).sum(), [own_q, own_k, own_v])
        out[0][:, h] = found[0]
        out[1][:, h // group] += found[1]
        out[2][:, h // group] += found[2]
    return dict(dq=out[0], dk=out[1], dv=out[2]) if grad else out[0]
