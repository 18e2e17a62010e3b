"""Launch one stage of the verification step a few times on a workload, for an external
profiler (ncu).  It holds only that workload's inputs on the device, so a profiler that
saves and restores device memory between its passes stays quick, and it prints no timing.

    python -m tree_verify_b200.profile_case --workload vicuna7b_static --stage lm_head --launches 3

Stages: attention, lm_head, accept, step (eagle_verify_step), and the kernels around the step:
commit (the root and accepted nodes of one walk into a cache with room for them), rerank
(256 random candidates down to the workload's N nodes), draft (the children of 10 draft
nodes per sequence, k = 10, from logits over the workload's vocabulary), paged_attention (the
workload's trees over a cache in pages of 64 positions, half of the prefix shared) and
lm_head_scaled (the workload's LM head in e4m3, hidden rows quantised in the call).
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def main() -> None:
    import torch

    import workloads as wl
    from tree_verify_b200 import binding
    from tree_verify_b200.step import StepInputs, VerifyStep, shape_from_workload

    ap = argparse.ArgumentParser()
    ap.add_argument("--workload", default="vicuna7b_static", choices=sorted(wl.WORKLOADS))
    ap.add_argument("--stage", default="lm_head",
                    choices=["attention", "lm_head", "accept", "step", "commit", "rerank", "draft",
                             "paged_attention", "lm_head_scaled"])
    ap.add_argument("--temperature", type=float, default=1.0)
    ap.add_argument("--launches", type=int, default=3)
    args = ap.parse_args()

    import numpy as np

    w = wl.WORKLOADS[args.workload]
    dev = torch.device("cuda")
    B, N, T = w.batch, w.num_nodes, args.temperature
    if args.stage == "draft":
        rng = np.random.default_rng(1234)
        d_logits = torch.from_numpy((rng.standard_normal((B, 10, w.vocab)) * 2.0).astype(np.float32)).to(dev)
        d_tok = torch.empty((B, 10, 10), dtype=torch.int32, device=dev)
        d_conf = torch.empty((B, 10, 10), dtype=torch.float32, device=dev)
        d_probs = torch.empty_like(d_logits)
        for i in range(args.launches):
            binding.draft_select(d_logits, T, 10, 0, i, d_tok, d_conf, d_probs)
            torch.cuda.synchronize()
        assert binding.device_error(reset=True) == 0
        print(f"draft x{args.launches} on {w.name}: ok")
        return
    if args.stage == "rerank":
        rng = np.random.default_rng(1234)
        par = np.stack([wl.random_parents(rng, 256, 10) for _ in range(B)]).astype(np.int32)
        r_in = [torch.from_numpy(a).to(dev) for a in
                (par, rng.integers(0, w.vocab, par.shape).astype(np.int32),
                 rng.uniform(0.0, 1.0, par.shape).astype(np.float32))]
        r_out = [torch.empty((B, N), dtype=torch.int32, device=dev) for _ in range(3)]
        r_masks = torch.empty((B, N), dtype=torch.int64, device=dev)
        r_n = torch.empty((B,), dtype=torch.int32, device=dev)
        for i in range(args.launches):
            binding.tree_rerank(*r_in, N, *r_out, r_masks, r_n)
            torch.cuda.synchronize()
        assert binding.device_error(reset=True) == 0
        print(f"rerank x{args.launches} on {w.name}: ok")
        return

    if args.stage in ("paged_attention", "lm_head_scaled"):
        dtype = torch.bfloat16 if w.dtype == wl.BF16 else torch.float32
        gen = torch.Generator(device=dev).manual_seed(1234)

        def normal(*shape):
            return torch.randn(shape, generator=gen, device=dev).to(dtype)

        if args.stage == "paged_attention":
            page, D, Hkv, L = 64, w.head_dim, w.num_kv_heads, w.prefix_len
            shared, width = L // 2, -(-L // page)
            table = torch.arange(B * width, device=dev, dtype=torch.int32).view(B, width)
            table[:, :shared // page] = table[0, :shared // page].clone()
            lens = torch.full((B,), L, dtype=torch.int32, device=dev)
            rng = np.random.default_rng(1234)
            parents = torch.from_numpy(np.stack([wl.random_parents(rng, N, 10) for _ in range(B)])
                                       .astype(np.int32)).to(dev)
            q, k_tree, v_tree = normal(B, N, w.num_q_heads, D), normal(B, N, Hkv, D), normal(B, N, Hkv, D)
            k_pages, v_pages = normal(B * width, Hkv, page, D), normal(B * width, Hkv, page, D)
            out = torch.empty_like(q)
            shape = shape_from_workload(w)
            pages = binding.make_pages(B * width, page, width)
            work = torch.empty(max(256, binding.paged_workspace_bytes(shape, pages, shared)), dtype=torch.uint8,
                               device=dev)
            calls = [lambda: binding.tree_attention_paged(shape, pages, q, k_pages, v_pages, table, lens, shared,
                                                          k_tree, v_tree, parents, out, work)]
        else:
            M, H, V, e4m3 = B * N, w.hidden, w.vocab, torch.float8_e4m3fn
            hidden, weight = normal(M, H), normal(V, H)
            h8, w8 = torch.empty((M, H), dtype=e4m3, device=dev), torch.empty((V, H), dtype=e4m3, device=dev)
            hs = torch.empty((-(-H // 128), -(-M // 4) * 4), dtype=torch.float32, device=dev)
            ws = torch.empty((-(-V // 128), -(-H // 128)), dtype=torch.float32, device=dev)
            logits = torch.empty((M, V), dtype=torch.float32, device=dev)
            binding.quantize_blocks(weight, w8, ws)
            calls = [lambda: binding.quantize_rows(hidden, h8, hs),
                     lambda: binding.lm_head_logits_scaled(h8, hs, w8, ws, logits)]
        for _ in range(args.launches):
            for call in calls:
                call()
            torch.cuda.synchronize()
        assert binding.device_error(reset=True) == 0
        print(f"{args.stage} x{args.launches} on {w.name}: ok")
        return

    inp = wl.generate(w, args.temperature)
    x = StepInputs.from_numpy(inp, w.dtype)
    step = VerifyStep(shape_from_workload(w))
    step.lm_head(x)  # logits for the accept stage
    torch.cuda.synchronize()
    if args.stage == "commit":
        step.run(x, T, 0, 0)  # the walk whose accepted nodes are committed
        k_cache = torch.zeros((B, w.num_kv_heads, w.prefix_len + N, w.head_dim), dtype=x.k_prefix.dtype,
                              device=dev)
        v_cache = torch.zeros_like(k_cache)
        new_lens = torch.empty((B,), dtype=torch.int32, device=dev)
        feat = torch.empty((B, N, w.hidden), dtype=x.hidden.dtype, device=dev)
        torch.cuda.synchronize()
    for i in range(args.launches):
        if args.stage == "commit":
            step.commit(x, k_cache, v_cache, new_lens, feat)
        elif args.stage == "attention":
            step.attention(x)
        elif args.stage == "lm_head":
            step.lm_head(x)
        elif args.stage == "accept":
            step.accept(x, args.temperature, 0, i)
        else:
            step.run(x, args.temperature, 0, i)
        torch.cuda.synchronize()
    assert binding.device_error(reset=True) == 0
    print(f"{args.stage} x{args.launches} on {w.name}: ok")


if __name__ == "__main__":
    main()
