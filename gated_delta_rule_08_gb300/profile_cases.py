"""One workload of the hot path, run alone a few times: a target for a profiler (ncu) that should
see one kernel family on a small device footprint.

    python -m gated_delta_rule_08_gb300.profile_cases prefill|prefill_epi|varlen|decode|verify|backward|prefill_d64|
        prefill_d64_epi|norm|matmul|matmul_few|linear|linear_token|rope|window|window_token|tree
        [--calls N]

prefill      B=1, H=32, T=8192, dk=dv=128, bf16 (q, k, v, g, beta: 337 MB; records 310 MB)
prefill_epi  the same with the RMSNorm + sigmoid gate epilogue
varlen       8 sequences, 27,654 tokens, H=32, dk=dv=128, bf16, h0
decode       N=256 requests, H=32, 1024-slot fp32 pool (2 GiB), RMSNorm + gate
verify       the decode workload with 4 draft tokens per request, pool not written
backward     the prefill workload's gradients (chunkwise path)
prefill_d64  B=1, H=32, T=8192, dk=dv=64, bf16 (the CUDA-core prefill path)
prefill_d64_epi  the same with the RMSNorm + sigmoid gate epilogue
norm         8192 rows of 4096 bf16 values, residual added, e4m3 output with scales
matmul       8192 x 4096 by 4096 x 4096 e4m3 with block scales
matmul_few   64 x 4096 by 12288 x 4096
linear       linear attention, one decay per head: B=1, H=32, T=8192, dk=dv=128, bf16
linear_token the same for one token of each of N=256 requests on a pool of 512 states
rope         rotary positions and cache write: 16384 tokens, 32 heads of 8, d=128, bf16
window       one prompt of 8192 tokens, 32 heads of 8, d=128, a window of 1024 and 4 sinks
window_token one token of each of N=256 requests over 2000 tokens each, same heads and window
tree         64 drafted tokens of each of N=16 requests over 4000 tokens each, same heads, all keys

Every call goes through the C-ABI binding; the first call is a warm-up.  Nothing is timed here.
"""
from __future__ import annotations

import argparse
import dataclasses
import sys

import torch

from . import binding, inputs


def _prefill(cfg, calls, dev):
    P = inputs.prefill_inputs(cfg, device=dev)
    varlen = cfg.len_range is not None or cfg.lengths is not None
    kw = {"cu_seqlens": P["cu_seqlens"]} if varlen else {"B": len(P["lengths"])}
    if cfg.epilogue:
        kw.update(gate=P["gate"], norm_weight=P["norm_weight"])
    for _ in range(calls + 1):
        binding.kda_chunk_fwd(P["q"], P["k"], P["v"], P["g"], P["beta"], h0=P["h0"], **kw)


def _layer_operator(case, calls, dev):
    gen = torch.Generator(device=dev).manual_seed(12)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if case == "norm":
        x, r, w = randn(8192, 4096).to(torch.bfloat16), randn(8192, 4096).to(torch.bfloat16), 1 + 0.1 * randn(4096)
        for _ in range(calls + 1):
            binding.kda_rmsnorm_quant(x, w, residual=r)
    elif case.startswith("matmul"):
        M, N, K = (8192, 4096, 4096) if case == "matmul" else (64, 12288, 4096)
        a, b = (randn(n, K).to(torch.float8_e4m3fn) for n in (M, N))
        sa, sb = 0.01 + randn(M, K // 128).abs(), 0.01 + randn(N // 128, K // 128).abs()
        for _ in range(calls + 1):
            binding.kda_matmul_fp8(a, sa, b, sb)
    else:
        n, H = (8192, 32) if case == "linear" else (256, 32)
        q, k, v = (randn(n, H, 128).to(torch.bfloat16) for _ in range(3))
        g = -0.1 * randn(n, H).abs()
        if case == "linear":
            for _ in range(calls + 1):
                binding.kda_linear_chunk_fwd(q, k, v, g, scale=128 ** -0.5)
        else:
            pool = randn(512, H, 128, 128)
            slots = torch.randperm(512, generator=gen, device=dev)[:n].to(torch.int32)
            for _ in range(calls + 1):
                binding.kda_linear_decode_step(q, k, v, g, pool, slots, scale=128 ** -0.5)


def _attention_operator(case, calls, dev):
    gen = torch.Generator(device=dev).manual_seed(13)
    H, Hkv, d, block = 32, 8, 128, 64

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev).to(torch.bfloat16)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    if case == "rope":
        T = 16384
        row = randn(T, H + 2 * Hkv, d)
        cache = [torch.empty(T // block, block, Hkv, d, dtype=torch.bfloat16, device=dev) for _ in range(2)]
        freq = 10000.0 ** (-torch.arange(d // 2, device=dev, dtype=torch.float64) / (d // 2))
        pos = torch.arange(T, dtype=torch.int32, device=dev)
        for _ in range(calls + 1):
            binding.kda_rope_append(row[:, :H], row[:, H:H + Hkv], row[:, H + Hkv:], freq, pos, pos, *cache)
        return
    N, length, new = {"window": (1, 8192, 8192), "window_token": (256, 2000, 1), "tree": (16, 4000, 64)}[case]
    each = -(-length // block)
    cache = [randn(N * each, block, Hkv, d) for _ in range(2)]
    tables = torch.arange(N * each, dtype=torch.int32, device=dev).view(N, each)
    lengths, cu, q = ints([length] * N), ints([new * i for i in range(N + 1)]), randn(N * new, H, d)
    mask = torch.tensor([1 << i | 1 for i in range(63)] + [1 - (1 << 63)], dtype=torch.int64, device=dev)
    for _ in range(calls + 1):
        if case == "window":
            binding.kda_window_attention_fwd(q, *cache, tables, lengths, cu, window=1024, sinks=4)
        elif case == "window_token":
            binding.kda_window_attention_decode_step(q, *cache, tables, lengths, window=1024, sinks=4)
        else:
            binding.kda_tree_attention(q, *cache, tables, lengths, cu, mask.repeat(N)[:, None].contiguous())


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("case", choices=["prefill", "prefill_epi", "varlen", "decode", "verify", "backward", "prefill_d64",
                                     "prefill_d64_epi", "norm", "matmul", "matmul_few", "linear", "linear_token", "rope",
                                     "window", "window_token", "tree"])
    ap.add_argument("--calls", type=int, default=2)
    args = ap.parse_args(argv)
    dev = torch.device("cuda", 0)
    torch.cuda.set_device(dev)
    if args.case in ("prefill", "prefill_epi"):
        _prefill(dataclasses.replace(inputs.PREFILL, epilogue=args.case == "prefill_epi"), args.calls, dev)
    elif args.case == "varlen":
        _prefill(inputs.VARLEN, args.calls, dev)
    elif args.case in ("prefill_d64", "prefill_d64_epi"):
        _prefill(dataclasses.replace(inputs.PREFILL, dk=64, dv=64, name="prefill d64",
                                     epilogue=args.case.endswith("_epi")), args.calls, dev)
    elif args.case in ("decode", "verify"):
        cfg = inputs.DECODE if args.case == "decode" else dataclasses.replace(inputs.DECODE, n_tok=4)
        D = inputs.decode_inputs(cfg, device=dev)
        for _ in range(args.calls + 1):
            if args.case == "decode":
                binding.kda_decode_step(D["q"], D["k"], D["v"], D["g"], D["beta"], D["state_pool"], D["slot_idx"],
                                        gate=D["gate"], norm_weight=D["norm_weight"])
            else:
                binding.kda_decode_multi(D["q"], D["k"], D["v"], D["g"], D["beta"], D["state_pool"], D["slot_idx"],
                                         commit=False, gate=D["gate"], norm_weight=D["norm_weight"])
    elif args.case in ("norm", "matmul", "matmul_few", "linear", "linear_token"):
        _layer_operator(args.case, args.calls, dev)
    elif args.case in ("rope", "window", "window_token", "tree"):
        _attention_operator(args.case, args.calls, dev)
    else:
        P = inputs.prefill_inputs(inputs.PREFILL, device=dev)
        gen = torch.Generator(device=dev).manual_seed(11)
        dout = torch.randn(P["T_tot"], 32, 128, generator=gen, device=dev).to(torch.bfloat16)
        for _ in range(args.calls + 1):
            binding.kda_chunk_bwd(P["q"], P["k"], P["v"], P["g"], P["beta"], dout)
    torch.cuda.synchronize()
    flags = binding.kda_get_device_error(dev)
    if flags:
        sys.stderr.write(f"device error word {flags:#x}\n")
        return 1
    return 0


if __name__ == "__main__":
    sys.exit(main())
