"""Cases and plain forms of the serving operators around a recurrent layer: a normalisation with 8-bit
output, the 8-bit matrix product of the projections, and linear attention with one decay per head
(chunked for prompts, recurrent for single tokens).

With `own` false, run() computes the operators by elementary torch operations in 32 bits; with `own`
true it calls libkda through the package's binding.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0        # largest e4m3 value
AMAX_FLOOR = 1e-30     # a block of zeros gets the scale AMAX_FLOOR / FP8_MAX
BLOCK = 128            # values (rows x values of a weight) that share a scale
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the norm in front of a projection for one generated token: latency
        {"name": "norm token", "op": "norm", "rows": 1, "dim": 4096, "dtype": "bf16", "residual": True},
        # ... for a prompt of 8192 tokens: bandwidth
        {"name": "norm prompt", "op": "norm", "rows": 8192, "dim": 4096, "dtype": "bf16", "residual": True},
        # a 32-bit residual stream, rows that are no multiple of anything, a last block of 80 values, no residual
        {"name": "norm ragged fp32", "op": "norm", "rows": 1237, "dim": 2000, "dtype": "fp32", "residual": False},
        # output projection (32 heads of 128 values) of one token
        {"name": "matmul token", "op": "matmul", "m": 1, "n": 4096, "k": 4096, "out": "bf16"},
        # q, k and v projection of a decode batch
        {"name": "matmul batch", "op": "matmul", "m": 64, "n": 12288, "k": 4096, "out": "bf16"},
        # a short prompt, with blocks that end inside a tile on every side
        {"name": "matmul ragged", "op": "matmul", "m": 1000, "n": 4200, "k": 2000, "out": "bf16"},
        # q, k and v projection of a prompt
        {"name": "matmul prompt", "op": "matmul", "m": 8192, "n": 12288, "k": 4096, "out": "bf16"},
        # a short prompt in 32 bits with heads of 64
        {"name": "linear short fp32", "op": "chunk", "b": 1, "t": 256, "least": 256, "h": 2, "dk": 64, "dv": 64, "dtype": "fp32",
         "decay": "token", "h0": False, "packed": False},
        # one prompt, its q, k and v being parts of one projection's rows
        {"name": "linear prompt", "op": "chunk", "b": 1, "t": 8192, "least": 8192, "h": 32, "dk": 128, "dv": 128, "dtype": "bf16",
         "decay": "token", "h0": False, "packed": True},
        # eight prompts that go on from earlier states, one constant decay per head
        {"name": "linear batch", "op": "chunk", "b": 8, "t": 8192, "least": 512, "h": 32, "dk": 128, "dv": 128, "dtype": "bf16",
         "decay": "head", "h0": True, "packed": True},
        # one generated token of one request
        {"name": "linear token", "op": "step", "n": 1, "h": 32, "dk": 128, "dv": 128, "dtype": "bf16", "decay": "token", "slots": 4},
        # one generated token of each of 256 requests
        {"name": "linear tokens", "op": "step", "n": 256, "h": 32, "dk": 128, "dv": 128, "dtype": "bf16", "decay": "head",
         "slots": 512},
    ]


def _log(rng, low, high, step=1):
    """step * a number of [low, high], even in its logarithm; round sizes (multiples of 1024) are for the listed cases."""
    n = step * int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return n - step if n % 1024 == 0 else n


def draw(rng):
    op = rng.choice(["norm", "matmul", "chunk", "step"])
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 8192), "dim": _log(rng, 4, 256, 16), "dtype": rng.choice(["bf16", "bf16", "fp32"]),
                "residual": rng.random() < 0.7}
    if op == "matmul":
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 16, 12288), "k": _log(rng, 4, 256, 16), "out": "bf16"}
    dk, dv, decay = rng.choice([64, 128, 128]), rng.choice([64, 128, 128]), rng.choice(["token", "head"])
    if op == "step":
        n = _log(rng, 1, 256)
        return {"op": op, "n": n, "h": _log(rng, 1, 32), "dk": dk, "dv": dv, "dtype": rng.choice(["bf16", "bf16", "fp32"]),
                "decay": decay, "slots": n + rng.randrange(n + 3)}
    wide = rng.random() < 0.25
    t, b = _log(rng, 1, 1024 if wide else 8192), _log(rng, 1, 8)
    return {"op": op, "b": b, "t": t, "least": max(1, t // rng.randrange(1, 17)), "h": _log(rng, 1, 32), "dk": dk, "dv": dv,
            "dtype": "fp32" if wide else "bf16", "decay": decay, "h0": rng.random() < 0.5, "packed": rng.random() < 0.5}


def _lengths(case):
    """Sequence lengths of a packed batch: the longest first, the others spread evenly (in the logarithm) down to the least."""
    b, t, least = case["b"], case["t"], case["least"]
    return [max(1, int(round(t * (least / t) ** (i / max(1, b - 1))))) for i in range(b)]


def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "norm":
        r, d, e = case["rows"], case["dim"], size[case["dtype"]]
        moved = r * d * (e * (3 if case["residual"] else 1) + 1) + 4 * r * -(-d // BLOCK) + 4 * d
        return {"bytes": moved, "flops": 6 * r * d}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // BLOCK)
        return {"bytes": m * k + n * k + m * n * size[case["out"]] + 4 * m * kb + 4 * -(-n // BLOCK) * kb, "flops": 2 * m * n * k}
    h, dk, dv, e = case["h"], case["dk"], case["dv"], size[case["dtype"]]
    if case["op"] == "step":
        n = case["n"]
        g = 4 * h * (n if case["decay"] == "token" else 1)
        return {"bytes": n * h * (8 * dk * dv + e * (2 * dk + 2 * dv)) + g + 4 * n, "flops": 5 * n * h * dk * dv}
    t, b = sum(_lengths(case)), case["b"]
    g = 4 * h * (t if case["decay"] == "token" else 1)
    states = 4 * b * h * dk * dv * (2 if case["h0"] else 1)
    return {"bytes": t * h * e * (2 * dk + 2 * dv) + g + states, "flops": 5 * t * h * dk * dv}


# ------------------------------------------------------------------------------------------- inputs
def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _decay(case, gen, rows):
    """Log decays: one constant for each head (a geometric ladder of slopes), or one for each token and head around the head's rate."""
    h = case["h"]
    if case["decay"] == "head":
        return -torch.pow(2.0, -8.0 * torch.arange(1, h + 1, device="cuda", dtype=torch.float32) / h)
    rate = torch.exp(torch.empty(h, device="cuda").uniform_(math.log(1e-3), math.log(0.3), generator=gen))
    return (-rate * torch.nn.functional.softplus(_randn(gen, rows, h))).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"op": case["op"]}
    if case["op"] == "norm":
        dt, r, d = TYPES[case["dtype"]], case["rows"], case["dim"]
        s["x"] = _randn(gen, r, d, dtype=dt)
        s["residual"] = _randn(gen, r, d, dtype=dt) if case["residual"] else None
        s["weight"] = 1.0 + 0.1 * _randn(gen, d)
        return s
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // BLOCK)
        a, a_scale = _quantise(_randn(gen, m, k))
        s["a"], s["a_scale"] = a, a_scale
        # a weight with an own scale for each 128 x 128 block, as a checkpoint stores it
        s["b"] = (_randn(gen, n, k) * (FP8_MAX / 4.5)).clamp(-FP8_MAX, FP8_MAX).to(FP8)
        s["b_scale"] = (4.5 / FP8_MAX) * k ** -0.5 * torch.exp(0.3 * _randn(gen, -(-n // BLOCK), kb))
        s["out"] = TYPES[case["out"]]
        return s
    h, dk, dv, dt = case["h"], case["dk"], case["dv"], TYPES[case["dtype"]]
    s["scale"] = dk ** -0.5
    if case["op"] == "step":
        n = case["n"]
        s["q"], s["k"], s["v"] = (_randn(gen, n, h, d, dtype=dt) for d in (dk, dk, dv))
        s["g"] = _decay(case, gen, n)
        s["pool"] = _randn(gen, case["slots"], h, dk, dv)
        s["slot"] = torch.randperm(case["slots"], generator=gen, device="cuda")[:n].to(torch.int32)
        return s
    lengths = _lengths(case)
    t = sum(lengths)
    if case["packed"]:  # q, k and v of a token side by side in one row
        row = _randn(gen, t, h * (2 * dk + dv), dtype=dt)
        s["q"], s["k"] = (row[:, i * h * dk:(i + 1) * h * dk].view(t, h, dk) for i in (0, 1))
        s["v"] = row[:, 2 * h * dk:].view(t, h, dv)
    else:
        s["q"], s["k"], s["v"] = (_randn(gen, t, h, d, dtype=dt) for d in (dk, dk, dv))
    s["g"] = _decay(case, gen, t)
    s["h0"] = _randn(gen, case["b"], h, dk, dv) if case["h0"] else None
    s["cu"] = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")
    s["longest"] = max(lengths)
    return s


# ------------------------------------------------------------------------------------------- one pass
def run(s):
    if own:
        import gated_delta_rule_08_gb300 as kda
        if s["op"] == "norm":
            return kda.kda_rmsnorm_quant(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        if s["op"] == "matmul":
            return kda.kda_matmul_fp8(s["a"], s["a_scale"], s["b"], s["b_scale"], out_dtype=s["out"])
        if s["op"] == "step":
            return kda.kda_linear_decode_step(s["q"], s["k"], s["v"], s["g"], s["pool"], s["slot"], scale=s["scale"]), s["pool"]
        return kda.kda_linear_chunk_fwd(s["q"], s["k"], s["v"], s["g"], h0=s["h0"], cu_seqlens=s["cu"], scale=s["scale"])
    return {"norm": _plain_norm, "matmul": _plain_matmul, "step": _plain_step, "chunk": _plain_chunk}[s["op"]](s)


def _quantise(y):
    """Rows of y (32 bits) as e4m3 values with one scale, the largest magnitude over 448, for each 128 of them."""
    r, d = y.shape
    wide = torch.nn.functional.pad(y, (0, -d % BLOCK)).view(r, -1, BLOCK)
    scale = wide.abs().amax(2).clamp_min(AMAX_FLOOR) / FP8_MAX
    return (wide / scale[..., None]).clamp(-FP8_MAX, FP8_MAX).view(r, -1)[:, :d].to(FP8).contiguous(), scale


def _plain_norm(s):
    z = s["x"].float()
    if s["residual"] is not None:
        z = z + s["residual"].float()
    y = z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS) * s["weight"]
    q, scale = _quantise(y)
    return q, scale, (z.to(s["x"].dtype) if s["residual"] is not None else None)


def _plain_matmul(s):
    (m, k), n = s["a"].shape, s["b"].shape[0]
    a = s["a"].float() * s["a_scale"].repeat_interleave(BLOCK, 1)[:, :k]
    b = s["b"].float() * s["b_scale"].repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return (a @ b.T).to(s["out"])


def _plain_step(s):
    slot = s["slot"].long()
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    state = torch.exp(s["g"].expand(q.shape[0], -1))[..., None, None] * s["pool"][slot] + k[..., :, None] * v[..., None, :]
    s["pool"][slot] = state
    return (s["scale"] * (q[..., None] * state).sum(2)).to(s["q"].dtype), s["pool"]


def _plain_chunk(s, C=64):
    """Per chunk of C tokens, with G the running sum of the log decays in the chunk and S the state before it:
    o_i = e^{G_i} S^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j; the chunks' own states are joined by one
    product over the chunks.  The sequences lie padded to one length (tokens of zeros with no decay)."""
    (t, h, dk), dv, b = s["q"].shape, s["v"].shape[2], s["cu"].numel() - 1
    n = -(-s["longest"] // C)
    token = torch.arange(t, device="cuda")
    seq = torch.searchsorted(s["cu"][1:].contiguous(), token, right=True)
    pos = token - s["cu"][seq]

    def padded(x):
        wide = torch.zeros(b, n * C, *x.shape[1:], dtype=x.dtype, device="cuda")
        wide[seq, pos] = x
        return wide.view(b, n, C, *x.shape[1:]).transpose(2, 3)  # [b, n, h, C, ...]

    q, k, v = padded(s["q"].float()), padded(s["k"].float()), padded(s["v"].float())
    g = padded(s["g"].double().expand(t, -1)[..., None])[..., 0].cumsum(3)
    causal = torch.ones(C, C, dtype=torch.bool, device="cuda").tril()
    weight = torch.exp((g[..., :, None] - g[..., None, :]).masked_fill_(~causal, -math.inf)).float()
    inside = ((q @ k.transpose(3, 4)) * weight) @ v
    states = (k * torch.exp(g[..., -1:] - g).float()[..., None]).transpose(3, 4) @ v          # [b, n, h, dk, dv]
    total = g[..., -1].cumsum(1).transpose(1, 2)                                              # [b, h, n], ends of the chunks
    starts = torch.nn.functional.pad(total, (1, 0))                                           # ... and their starts: [b, h, n + 1]
    before = torch.ones(n + 1, n, dtype=torch.bool, device="cuda").tril(-1)
    join = torch.exp((starts[..., :, None] - total[..., None, :]).masked_fill_(~before, -math.inf)).float()
    at = join @ states.transpose(1, 2).reshape(b, h, n, dk * dv)
    if s["h0"] is not None:
        at = at + torch.exp(starts).float()[..., None] * s["h0"].reshape(b, h, 1, dk * dv)
    at = at.view(b, h, n + 1, dk, dv)
    out = inside + torch.exp(g).float()[..., None] * (q @ at[:, :, :n].transpose(1, 2))
    out = (s["scale"] * out).transpose(2, 3).reshape(b, n * C, h, dv)[seq, pos].to(s["q"].dtype)
    return out, at[:, :, n].contiguous()


# ------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        z = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        y = z / torch.sqrt((z * z).sum(1, keepdim=True) / z.shape[1] + EPS) * s["weight"].double()
        scale = torch.stack([p.abs().max(1).values for p in y.split(BLOCK, 1)], 1).clamp(min=AMAX_FLOOR) / FP8_MAX
        each = torch.arange(y.shape[1], device="cuda") // BLOCK
        return y / scale[:, each], scale, (z if s["residual"] is not None else None)
    if case["op"] == "matmul":
        k, n = case["k"], case["n"]
        kb, nb = torch.arange(k, device="cuda") // BLOCK, torch.arange(n, device="cuda") // BLOCK
        return torch.matmul(s["a"].double() * s["a_scale"].double()[:, kb], (s["b"].double() * s["b_scale"].double()[nb][:, kb]).T)
    if case["op"] == "step":
        state = s["pool"].double()
        out = torch.empty(case["n"], case["h"], case["dv"], dtype=torch.float64, device="cuda")
        for i, at in enumerate(s["slot"].tolist()):
            decay = s["g"][i] if s["g"].dim() == 2 else s["g"]
            state[at] = torch.exp(decay.double())[:, None, None] * state[at] + torch.einsum("hk,hv->hkv", s["k"][i].double(), s["v"][i].double())
            out[i] = s["scale"] * torch.einsum("hkv,hk->hv", state[at], s["q"][i].double())
        return out, state
    # token by token, all sequences of the batch that are still running at once (they lie longest first)
    lengths, cu = _lengths(case), s["cu"].long()
    h, dk, dv = case["h"], case["dk"], case["dv"]
    state = s["h0"].double() if s["h0"] is not None else torch.zeros(case["b"], h, dk, dv, dtype=torch.float64, device="cuda")
    q, k, v, decay = s["q"].double(), s["k"].double(), s["v"].double(), torch.exp(s["g"].double()).expand(s["q"].shape[0], -1)
    out = torch.empty(sum(lengths), h, dv, dtype=torch.float64, device="cuda")
    for i in range(max(lengths)):
        live = sum(n > i for n in lengths)
        at = cu[:live] + i
        now = state[:live]
        now.mul_(decay[at][..., None, None]).addcmul_(k[at][..., None], v[at][..., None, :])
        out[at] = s["scale"] * torch.matmul(q[at][..., None, :], now)[..., 0, :]
    return out, state

