"""Inputs and error bounds for the tests of the operators around a recurrent layer."""
from __future__ import annotations

import numpy as np
import torch

#: half a step of rounding to a type, relative to the value
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float32)}
E4M3_HALF, E4M3_TINY = 2.0 ** -4, 2.0 ** -10  # relative, and half the spacing of the subnormal numbers
F32 = 2.0 ** -24


def gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=g.device).to(dtype)


def f64(t):
    return t.detach().to(torch.float32).cpu().double().numpy() if t.dtype != torch.float64 else t.detach().cpu().numpy()


def within(got, want, bound, what):
    """|got - want| <= bound everywhere, NaN nowhere."""
    got, off = f64(got), None
    off = np.abs(got - want)
    bad = ~(off <= bound)
    assert not bad.any(), (what, "%d of %d" % (bad.sum(), bad.size), "first at", np.argwhere(bad)[:3].tolist(),
                           "worst", float(np.nanmax(off / np.maximum(bound, 1e-300))), "of the bound")


def rel2(got, want):
    n = np.linalg.norm(want)
    return float(np.linalg.norm(f64(got) - want) / n) if n else float(np.linalg.norm(f64(got)))


def linear_inputs(seed, lengths, H, dk, dv, dtype, decay="token", h0=False, packed=False, device="cuda"):
    r = gen(seed, device)
    T = sum(lengths)
    if packed:
        row = randn(r, T, H * (2 * dk + dv) + 8, dtype=dtype)  # and eight values that belong to nobody
        q, k = (row[:, i * H * dk:(i + 1) * H * dk].view(T, H, dk) for i in (0, 1))
        v = row[:, 2 * H * dk:2 * H * dk + H * dv].view(T, H, dv)
    else:
        q, k, v = (randn(r, T, H, d, dtype=dtype) for d in (dk, dk, dv))
    if decay == "head":
        g = -torch.pow(2.0, -8.0 * torch.arange(1, H + 1, device=device, dtype=torch.float32) / H)
    else:
        g = -0.2 * torch.nn.functional.softplus(2 * randn(r, T, H))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=device)
    return {"q": q, "k": k, "v": v, "g": g.contiguous(), "h0": randn(r, len(lengths), H, dk, dv) if h0 else None, "cu": cu}


def linear_bounds(n, dk, dtype, out_dtype, out, mag, state_mag):
    """Error bounds of a sequence of n tokens.
    fp32 path: sums of at most n + dk products in fp32 (each step F32), the decays' exponent (a running
    sum of at most n logs, of magnitude below 64 where it matters) and exp itself: (n + dk + 64) steps
    of 2 F32 on the terms' magnitudes.  bf16 path: also the attention weights of a chunk and the state
    before it are rounded to bf16 once each (HALF of the terms' magnitudes each), in the read-out only."""
    steps = 2 * F32 * (n + dk + 64)
    inner = steps + (2 * HALF[torch.bfloat16] if dtype == torch.bfloat16 else 0.0)
    return HALF[out_dtype] * (np.abs(out) + inner * mag) + inner * mag, steps * state_mag
