"""Cases and plain forms of the operators of an attention layer over a paged cache, as models put one between their
recurrent layers: the batch's block tables and slots, rotary positions with the cache's write, attention with a sliding
window and sinks (prompts and single tokens), and attention of trees of drafted tokens.

With `own` false, run() computes the operators by elementary torch operations in 32 bits; with `own`
true it calls libkda through the package's binding.
"""
import math

import torch

own = False

THETA = 10000.0  # base of the rotary frequencies
BF16 = torch.bfloat16


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one more token for each of 256 requests that are being answered: latency
        {"name": "tables tokens", "op": "tables", "n": 256, "kind": "tokens", "most": 8192, "new": 1, "block": 16},
        # a step with prompts of up to 2048 tokens, single tokens, and requests that end or take back drafted tokens
        {"name": "tables mixed", "op": "tables", "n": 1000, "kind": "mixed", "most": 16000, "new": 2048, "block": 64},
        # one generated token
        {"name": "rotary token", "op": "rope", "t": 1, "h": 32, "hk": 8, "d": 128, "rot": 128, "axes": 1, "far": 8192,
         "pairs": "halves", "dtype": "bf16", "packed": True, "block": 16},
        # 32-bit rows with pairs side by side, half of each head rotated, positions far beyond 32-bit angles
        {"name": "rotary far fp32", "op": "rope", "t": 1237, "h": 12, "hk": 4, "d": 64, "rot": 32, "axes": 1, "far": 1 << 30,
         "pairs": "adjacent", "dtype": "fp32", "packed": False, "block": 32},
        # a video's tokens (time, height and width), parts of one projection's rows
        {"name": "rotary video", "op": "rope", "t": 16384, "h": 32, "hk": 8, "d": 128, "rot": 128, "axes": 3, "far": 8192,
         "pairs": "halves", "dtype": "bf16", "packed": True, "block": 64},
        # one prompt in a layer with a window
        {"name": "window prompt", "op": "prompt", "n": 1, "new": 8192, "least": 8192, "cached": 0, "h": 32, "hk": 8, "d": 128,
         "window": 1024, "sinks": 4, "block": 64},
        # parts of five prompts that go on from what is cached, five heads to a key, small heads and blocks
        {"name": "window parts", "op": "prompt", "n": 5, "new": 2000, "least": 3, "cached": 9000, "h": 20, "hk": 4, "d": 64,
         "window": 4096, "sinks": 0, "block": 16},
        # one long prompt in a layer without a window
        {"name": "whole prompt", "op": "prompt", "n": 1, "new": 16384, "least": 16384, "cached": 0, "h": 32, "hk": 8, "d": 128,
         "window": 0, "sinks": 0, "block": 128},
        # one generated token of one request, all of its cache
        {"name": "attention token", "op": "token", "n": 1, "longest": 8000, "least": 8000, "h": 32, "hk": 8, "d": 128, "window": 0,
         "sinks": 0, "block": 64},
        # one generated token of each of 256 requests in a layer with a window
        {"name": "attention tokens", "op": "token", "n": 256, "longest": 16000, "least": 20, "h": 32, "hk": 8, "d": 128,
         "window": 1024, "sinks": 4, "block": 16},
        # twelve drafted tokens of one request
        {"name": "tree", "op": "tree", "n": 1, "drafted": 12, "longest": 4000, "least": 4000, "h": 32, "hk": 8, "d": 128,
         "window": 0, "sinks": 0, "block": 16},
        # trees of 64 drafted tokens of 32 requests
        {"name": "tree batch", "op": "tree", "n": 32, "drafted": 64, "longest": 16000, "least": 500, "h": 32, "hk": 8, "d": 128,
         "window": 0, "sinks": 0, "block": 64},
    ]


def _log(rng, low, high):
    """A number of [low, high], even in its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "prompt", "token", "tree"])
    block = rng.choice([16, 32, 64, 128])
    if op == "tables":
        kind = rng.choice(["tokens", "mixed"])
        return {"op": op, "n": _log(rng, 1, 1000), "kind": kind, "most": _log(rng, 100, 16000),
                "new": _log(rng, 1, 2048) if kind == "mixed" else _log(rng, 1, 8), "block": block}
    hk, d = _log(rng, 1, 8), rng.choice([64, 128, 128])
    h = hk * rng.choice([1, 2, 3, 4, 4, 5, 8])
    if h > 32:
        h = hk * 4
    if op == "rope":
        rot = rng.choice([d, d, d // 2])
        return {"op": op, "t": _log(rng, 1, 16384), "h": h, "hk": hk, "d": d, "rot": rot, "axes": rng.choice([1, 3]),
                "far": _log(rng, 1000, 1 << 30), "pairs": rng.choice(["halves", "adjacent"]),
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "packed": rng.random() < 0.5, "block": block}
    window = rng.choice([0, _log(rng, 16, 4096), _log(rng, 16, 4096)])
    case = {"op": op, "n": 1, "h": h, "hk": hk, "d": d, "window": window, "sinks": rng.choice([0, 4, _log(rng, 1, 100)]), "block": block}
    if op == "prompt":
        case["n"] = _log(rng, 1, 8)
        case["new"] = _log(rng, 16, 8192 // case["n"])
        case["least"] = max(1, case["new"] // rng.randrange(1, 20))
        case["cached"] = rng.choice([0, _log(rng, 10, 8192)])
        return case
    case["n"] = _log(rng, 1, 256 if op == "token" else 32)
    case["longest"] = min(_log(rng, 100, 16000), 1000000 // case["n"])
    case["least"] = max(1, case["longest"] // rng.randrange(1, 40))
    if op == "tree":
        case["drafted"] = _log(rng, 2, 64)
    return case


def _spread(n, most, least):
    """n numbers from the most down to the least, even in their logarithm."""
    return [max(1, int(round(most * (least / most) ** (i / max(1, n - 1))))) for i in range(n)]


def _batch(case):
    """Tokens in the cache before the call and new tokens, of each request."""
    n = case["n"]
    if case["op"] == "prompt":
        new = _spread(n, case["new"], case["least"])
        return ([case["cached"] // (i + 1) for i in range(n)] if case["cached"] else [0] * n), new
    before = _spread(n, case["longest"], case["least"])
    before = before[::2] + before[1::2][::-1]  # in no order of their length
    if case["op"] == "token":
        return [b - 1 for b in before], [1] * n
    return before, [max(1, case["drafted"] - i % 4) for i in range(n)]


def _tables_batch(case):
    """Lengths and counts of a tables case, and the blocks that its requests hold and take."""
    n, most, new = case["n"], case["most"], case["new"]
    lengths = [most * (i + 1) // n * 7 % (most + 1) for i in range(n)]
    if case["kind"] == "tokens":
        counts = [1 + i % new for i in range(n)]
    else:
        counts = [max(1, new >> (i % 11)) if i % 10 == 0 else 1 if i % 10 < 7 else -lengths[i] if i % 10 == 7 else
                  -min(lengths[i], i % 23) for i in range(n)]
        for i in range(0, n, 10):
            lengths[i] = 0 if i % 20 == 0 else lengths[i]
    return lengths, counts


def _blocks(tokens, block):
    return -(-tokens // block)


def _pairs_seen(case):
    """Pairs of a token and a key it sees, and keys that some token of its request sees, over all requests."""
    pairs = keys = 0
    window, sinks = case["window"], case["sinks"]
    for before, new in zip(*_batch(case)):
        if case["op"] == "tree":
            w = window or before
            first = max(0, before + 1 - w) if window else 0
            keys += min(before, before - first + min(sinks, first)) + new
            pairs += new * (min(before, before - first + min(sinks, first))) + new * 6
            continue
        full = before + new
        for at in range(0, new, max(1, new // 64)):  # sums over a sample of the tokens
            p = before + at
            first = max(0, p + 1 - window) if window else 0
            pairs += (p + 1 - first + min(sinks, first)) * min(max(1, new // 64), new - at)
        first = max(0, before + 1 - window) if window else 0
        keys += full - first + min(sinks, first)
    return pairs, keys


def work(case):
    op = case["op"]
    if op == "tables":
        lengths, counts = _tables_batch(case)
        tokens = sum(c for c in counts if c > 0)
        moved = sum(abs(_blocks(a + c, case["block"]) - _blocks(a, case["block"])) for a, c in zip(lengths, counts))
        return {"bytes": 8 * tokens + 16 * case["n"] + 8 * moved, "flops": 0}
    h, hk, d = case["h"], case["hk"], case["d"]
    if op == "rope":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["t"] * ((h + 2 * hk) * d * (size + 2) + 4 * case["axes"] + 4), "flops": case["t"] * (h + hk) * case["rot"] * 3}
    pairs, keys = _pairs_seen(case)
    tokens = sum(_batch(case)[1])
    return {"bytes": 4 * keys * hk * d + 4 * tokens * h * d, "flops": 4 * pairs * h * d}


# ------------------------------------------------------------------------------------------- inputs
def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(new):
    return _ints([sum(new[:i]) for i in range(len(new) + 1)])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, block = case["op"], case["block"]
    s = {"op": op, "block": block}
    if op == "tables":
        lengths, counts = _tables_batch(case)
        held = [_blocks(a, block) for a in lengths]
        taken = sum(max(0, _blocks(a + c, block) - b) for a, c, b in zip(lengths, counts, held))
        blocks = sum(held) + taken + 50
        width = max(_blocks(a + max(c, 0), block) for a, c in zip(lengths, counts)) + 2
        order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((case["n"], width), -1, dtype=torch.int32, device="cuda")
        mine = torch.arange(width, device="cuda")[None] < _ints(held)[:, None]
        table[mine] = order[:sum(held)]
        head, free = int(seed) * 7919 % blocks, blocks - sum(held)
        ring = torch.full((blocks,), -1, dtype=torch.int32, device="cuda")
        ring[(head + torch.arange(free, device="cuda")) % blocks] = order[sum(held):]
        s.update(counts=_ints(counts), lengths=_ints(lengths), table=table, ring=ring, free=_ints([head, free]),
                 tokens=sum(c for c in counts if c > 0))
        return s
    h, hk, d = case["h"], case["hk"], case["d"]
    if op == "rope":
        t, dt = case["t"], BF16 if case["dtype"] == "bf16" else torch.float32
        if case["packed"]:  # q, k and v of a token side by side in one row
            row = _randn(gen, t, (h + 2 * hk) * d, dtype=dt).view(t, h + 2 * hk, d)
            s["q"], s["k"], s["v"] = row[:, :h], row[:, h:h + hk], row[:, h + hk:]
        else:
            s["q"], s["k"], s["v"] = (_randn(gen, t, n, d, dtype=dt) for n in (h, hk, hk))
        pairs, axes = case["rot"] // 2, case["axes"]
        s["freq"] = THETA ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)
        s["axis"] = (torch.arange(pairs, device="cuda") * axes // pairs).to(torch.int32)
        s["pos"] = torch.randint(0, case["far"], (axes, t), generator=gen, device="cuda", dtype=torch.int32)
        blocks = _blocks(t, block) + 3
        s["slot"] = torch.randperm(blocks * block, generator=gen, device="cuda")[:t].to(torch.int32)
        s["k_cache"], s["v_cache"] = (_randn(gen, blocks, block, hk, d, dtype=BF16) for _ in range(2))
        s["adjacent"] = case["pairs"] == "adjacent"
        return s
    before, new = _batch(case)
    held = [_blocks(b + n, block) for b, n in zip(before, new)]
    blocks, width = sum(held) + 5, max(held) + 1
    table = torch.zeros(case["n"], width, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None] < _ints(held)[:, None]] = \
        torch.randperm(blocks, generator=gen, device="cuda")[:sum(held)].to(torch.int32)
    s.update(table=table, before=before, new=new, lengths=_ints([b + n for b, n in zip(before, new)]), cu=_offsets(new),
             window=case["window"], sinks=case["sinks"], scale=d ** -0.5)
    s["k_cache"], s["v_cache"] = (_randn(gen, blocks, block, hk, d, dtype=BF16) for _ in range(2))
    s["q"] = _randn(gen, sum(new), h, d, dtype=BF16)
    if op == "tree":
        # every drafted token follows one of the two to three before it, the first ones the request's last token
        masks = []
        for i, n in enumerate(new):
            seen = []
            for j in range(n):
                parent = j - 1 - (j * 5 + i + int(seed)) % 3
                seen.append((seen[parent] if parent >= 0 else 0) | 1 << j)
            masks += [m - (1 << 64) if m >> 63 else m for m in seen]
        s["mask"] = torch.tensor(masks, dtype=torch.int64, device="cuda")[:, None].contiguous()
    return s


# ------------------------------------------------------------------------------------------- one pass
def run(s):
    if own:
        import gated_delta_rule_08_gb300 as kda
        if s["op"] == "tables":
            slot, pos, cu, lengths, free = kda.kda_block_tables(s["counts"], s["lengths"], s["table"], s["ring"], s["free"],
                                                                block_size=s["block"], max_tokens=s["tokens"])
            return slot, pos, cu, lengths, free, s["table"], s["ring"]
        if s["op"] == "rope":
            q = kda.kda_rope_append(s["q"], s["k"], s["v"], s["freq"], s["pos"], s["slot"], s["k_cache"], s["v_cache"],
                                    axis=s["axis"], interleaved=s["adjacent"])
            return q, s["k_cache"], s["v_cache"]
        if s["op"] == "prompt":
            return kda.kda_window_attention_fwd(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["cu"],
                                                window=s["window"], sinks=s["sinks"], scale=s["scale"])
        if s["op"] == "token":
            return kda.kda_window_attention_decode_step(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"],
                                                        window=s["window"], sinks=s["sinks"], scale=s["scale"])
        return kda.kda_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["cu"], s["mask"],
                                      window=s["window"], sinks=s["sinks"], scale=s["scale"])
    return {"tables": _plain_tables, "rope": _plain_rope, "prompt": _plain_prompt, "token": _plain_few, "tree": _plain_few}[s["op"]](s)


def _plain_tables(s):
    block, ring, table = s["block"], s["ring"], s["table"]
    lengths, counts = s["lengths"].long(), s["counts"].long()
    size, (head, free) = ring.shape[0], s["free"].long()
    held, after = -(-lengths // block), -(-(lengths + counts) // block)
    at = torch.arange(table.shape[1], device="cuda")[None]
    gone = (at >= after[:, None]) & (at < held[:, None])
    taken = (at >= held[:, None]) & (at < after[:, None])
    ring[(head + free + torch.arange(gone.sum(), device="cuda")) % size] = table[gone]
    table[taken] = ring[(head + torch.arange(taken.sum(), device="cuda")) % size]
    new = counts.clamp_min(0)
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    whose = torch.repeat_interleave(new, output_size=s["tokens"])
    pos = torch.arange(s["tokens"], device="cuda") - cu[whose] + lengths[whose]
    slot = table[whose, pos // block] * block + pos % block
    state = torch.stack([(head + taken.sum()) % size, free - taken.sum() + gone.sum()])
    return slot.int(), pos.int(), cu.int(), (lengths + counts).int(), state.int(), table, ring


def _plain_rope(s):
    pairs = s["freq"].shape[0]
    angle = s["pos"].double()[s["axis"].long()].T * s["freq"]  # [t, pairs], in 64 bits: positions are far
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def rotate(x):
        x, rest = x[..., :2 * pairs].float(), x[..., 2 * pairs:].float()
        if s["adjacent"]:
            a, b = x[..., 0::2], x[..., 1::2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :pairs], x[..., pairs:]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y, rest], -1).to(BF16)

    slot = s["slot"].long()
    s["k_cache"].view(-1, *s["k_cache"].shape[2:])[slot] = rotate(s["k"])
    s["v_cache"].view(-1, *s["v_cache"].shape[2:])[slot] = s["v"].to(BF16)
    return rotate(s["q"]), s["k_cache"], s["v_cache"]


def _softmax_product(scores, seen, v):
    """softmax over the last axis of what is seen, times v; nothing seen gives zeros."""
    scores = scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores.sub_(torch.where(top == -math.inf, 0.0, top)))
    return (p @ v) / p.sum(-1, keepdim=True).clamp_min(1e-30)


def _plain_prompt(s, rows=1024):
    """Request by request, `rows` tokens at a time with the keys that some of them see."""
    h, (hk, d) = s["q"].shape[1], s["k_cache"].shape[2:]
    block, out, t = s["block"], torch.empty_like(s["q"]), 0
    for i, (before, new) in enumerate(zip(s["before"], s["new"])):
        flat = (s["table"][i].long()[:, None] * block + torch.arange(block, device="cuda")).flatten()[:before + new]
        k, v = (c.view(-1, hk, d)[flat].float().transpose(0, 1) for c in (s["k_cache"], s["v_cache"]))
        for r in range(0, new, rows):
            m = min(rows, new - r)
            pos = before + r + torch.arange(m, device="cuda")[:, None]
            first = max(0, before + r + 1 - s["window"]) if s["window"] else 0
            key = torch.arange(first, before + r + m, device="cuda")
            if first:
                key = torch.cat([torch.arange(min(s["sinks"], first), device="cuda"), key])
            seen = key <= pos
            if s["window"]:
                seen = seen & ((key > pos - s["window"]) | (key < s["sinks"]))
            q = s["q"][t + r:t + r + m].float().view(m, hk, h // hk, d).permute(1, 2, 0, 3).reshape(hk, -1, d)
            scores = (q @ k[:, key].transpose(1, 2)).mul_(s["scale"]).view(hk, h // hk, m, -1)
            o = _softmax_product(scores, seen, v[:, None, key])
            out[t + r:t + r + m] = o.permute(2, 0, 1, 3).reshape(m, h, d).to(BF16)
        t += new
    return out


def _plain_few(s):
    """All requests at once, padded: single tokens, or trees."""
    n, h, (hk, d) = len(s["new"]), s["q"].shape[1], s["k_cache"].shape[2:]
    block, window, sinks, most = s["block"], s["window"], s["sinks"], max(s["new"])
    before = s["lengths"].long() - (s["cu"][1:] - s["cu"][:-1]).long()
    long, low = max(s["before"]), min(s["before"])
    # a window's keys: the sinks, then as many before the new tokens as the window has; else all keys
    if window and sinks + window + most < long:
        first = (before + 1 - window).clamp_min(0)
        ahead = torch.arange(min(sinks, long), device="cuda").expand(n, -1)
        ahead = torch.where(ahead < torch.minimum(first, before)[:, None], ahead, -1)
        key = torch.cat([ahead, first[:, None] + torch.arange(window + most, device="cuda")], 1)
    else:
        key = torch.arange(long + most, device="cuda").expand(n, -1)
    key = torch.where(key < s["lengths"][:, None], key, -1)
    flat = s["table"].long().gather(1, (key.clamp_min(0) // block)) * block + key.clamp_min(0) % block
    k, v = (c.view(-1, hk, d)[flat].float().transpose(1, 2) for c in (s["k_cache"], s["v_cache"]))  # [n, hk, keys, d]
    step = torch.arange(most, device="cuda")
    live = step < (s["cu"][1:] - s["cu"][:-1])[:, None]                                           # [n, most]
    token = (s["cu"][:-1, None] + step).clamp_max(s["q"].shape[0] - 1).long()
    if s["op"] == "tree":
        bit = (s["mask"][token, 0][:, :, None] >> torch.arange(64, device="cuda")) & 1            # [n, most, 64]
        depth = before[:, None] + bit.sum(2) - 1
        drafted = (key - before[:, None])[:, None]                                                # [n, 1, keys]
        tree = bit.gather(2, drafted.clamp(0, 63).expand(-1, most, -1)).bool() & (drafted >= 0)
    else:
        depth, tree = before[:, None] + step, None
    seen = (key[:, None] >= 0) & (key[:, None] < before[:, None, None] if tree is not None else key[:, None] <= depth[..., None])
    if window:
        seen = seen & ((key[:, None] > depth[..., None] - window) | (key[:, None] < sinks))
    if tree is not None:
        seen = seen | (tree & (key[:, None] >= 0))
    q = s["q"][token].float().view(n, most, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, d)
    scores = (q @ k.transpose(2, 3)).mul_(s["scale"]).view(n, hk, h // hk, most, -1)
    o = _softmax_product(scores, seen[:, None, None], v[:, :, None])
    return o.permute(0, 3, 1, 2, 4).reshape(n, most, h, d)[live].to(BF16)


# ------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, block = case["op"], case["block"]
    if op == "tables":
        return None  # whole numbers
    h, hk, d = case["h"], case["hk"], case["d"]
    if op == "rope":
        half, out = case["rot"] // 2, []
        turn = torch.outer(torch.ones(case["t"], device="cuda", dtype=torch.float64), s["freq"])
        for i, a in enumerate(s["axis"].tolist()):
            turn[:, i] *= s["pos"][a].double()
        unit = torch.polar(torch.ones_like(turn), turn)[:, None]
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            even, odd = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if s["adjacent"] else (slice(0, half), slice(half, 2 * half))
            z = torch.complex(y[..., even].contiguous(), y[..., odd].contiguous()) * unit
            y[..., even], y[..., odd] = z.real, z.imag
            out.append(y)
        caches = [s["k_cache"].double(), s["v_cache"].double()]
        for c, x in zip(caches, (out[1], s["v"].double())):
            c.view(-1, hk, d).index_copy_(0, s["slot"].long(), x)
        return out[0], caches[0], caches[1]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    t = 0
    for i, (before, new) in enumerate(zip(s["before"], s["new"])):
        length = before + new
        pages = s["table"][i, :_blocks(length, block)].long()
        k, v = (c[pages].flatten(0, 1)[:length].double() for c in (s["k_cache"], s["v_cache"]))
        for r in range(0, new, 512):
            m = min(512, new - r)
            row, col = torch.arange(r, r + m, device="cuda")[:, None], torch.arange(length, device="cuda")[None]
            if op == "tree":
                own_bits = s["mask"][t + r:t + r + m]
                place = before - 1 + sum(((own_bits >> j) & 1) for j in range(64))
                drafted = ((own_bits >> (col - before).clamp(0, 63)) & 1).bool() & (col >= before)
                seen = (col < before) & ((col > place - case["window"]) | (col < case["sinks"]) | (case["window"] == 0)) | drafted
            else:
                seen = (col <= before + row) & ((col > before + row - case["window"]) | (col < case["sinks"]) | (case["window"] == 0))
            keep = seen.any(0).nonzero()[:, 0]  # keys that one of these tokens sees
            for head in range(h):
                z = s["q"][t + r:t + r + m, head].double() @ k[keep, head * hk // h].T * s["scale"]
                z = torch.where(seen[:, keep], z, -math.inf)
                out[t + r:t + r + m, head] = torch.softmax(z, 1) @ v[keep, head * hk // h]
        t += new
    return out
