"""The dense feed-forward sub-layer on one GPU: training steps (forward,
backward, a plain update of float32 master weights) and single-token serving.

    python examples/dense_ffn_step.py [--tokens 4096 --hidden 7168 --inner 2048 --steps 5 --lr 0.01]
"""

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import fp8_block_scaled_dsmoe_amd as d


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--lr", type=float, default=0.01)
    a = ap.parse_args()
    torch.manual_seed(0)
    T, H, I = a.tokens, a.hidden, a.inner

    def randn(*shape, std=1.0):
        return torch.randn(*shape, device="cuda") * std

    master = {"gamma": torch.ones(H, device="cuda"), "beta": torch.zeros(H, device="cuda"),
              "w13": randn(2 * I, H, std=H ** -0.5), "w2": randn(H, I, std=I ** -0.5)}
    x, target = randn(T, H).bfloat16(), randn(T, H).bfloat16()
    w13, w2 = master["w13"].bfloat16(), master["w2"].bfloat16()
    for step in range(a.steps):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        y, saved = d.dense_ffn_forward(x, master["gamma"], master["beta"], w13, w2, training=True)
        dy = (y - target) * (2.0 / T)
        # every product on bf16 operands; without dz_dtype the float32 gradient
        # of w13 would take a second product for the rest of its operand
        g = d.dense_ffn_backward(dy, saved, master["gamma"], w13, w2, dz_dtype=torch.bfloat16)
        for name in master:
            master[name].sub_(g["d" + name], alpha=a.lr)
        w13.copy_(master["w13"])
        w2.copy_(master["w2"])
        torch.cuda.synchronize()
        ms = (time.perf_counter() - t0) * 1e3
        loss = float((y.float() - target.float()).square().mean())
        print(f"step {step}: loss {loss:.4f}, {ms:.3f} ms", flush=True)
    for _ in range(a.steps):
        y, _ = d.dense_ffn_forward(x[:1], master["gamma"], master["beta"], w13, w2)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(100):
        y, _ = d.dense_ffn_forward(x[:1], master["gamma"], master["beta"], w13, w2)
    torch.cuda.synchronize()
    print(f"one token: {(time.perf_counter() - t0) * 1e4:.1f} us, finite {bool(torch.isfinite(y).all())}")


if __name__ == "__main__":
    main()
