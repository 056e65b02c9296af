"""One MoE layer behind a grouped sigmoid router, with its shared FFN in FP8.

What a model of this kind does per layer, through the binding:
  once    the shared FFN's FP16 weights to FP8 in 128 x 128 blocks
          (moe_quantize_fp8), the router's settings, the workspaces;
  a call  y_shared = moe_shared_forward_fp8(x), then
          y = moe_layer_forward_scored(x, router logits, bias) + y_shared.
Runs a decode step (one token) and a prefill (512 tokens) on synthetic weights,
compares the FP8 shared path with the FP16 one, and times both.

  python examples/fp8_shared_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from int4_routed_expert_moe_gb300 import moe, synth  # noqa: E402

SHAPE, E, TOP_K = (2048, 1024, 128), 64, 8  # hidden, expert intermediate, group; experts, picks
SHARED = 4096                               # the shared FFN's intermediate size


class Layer:
    def __init__(self, seed: int = 1):
        H, self.dev = SHAPE[0], torch.device("cuda")
        self.pool = synth.device_pool(E, *SHAPE, seed=seed)
        self.slot_of = torch.arange(E, dtype=torch.int32, device=self.dev)
        self.fp16 = {n: torch.from_numpy(w).cuda() for n, w in synth.shared_weights(seed, H, SHARED).items()}
        self.fp8 = [t for n in ("wg", "wu", "wd") for t in self.to_fp8(self.fp16[n], 128)]
        self.router = moe.moe_route_config(score="sigmoid", n_groups=8, top_groups=4, group_rank="top2", renorm=True,
                                           scale=2.5)
        self.bias = torch.linspace(-0.05, 0.05, E, device=self.dev)[torch.randperm(E, device=self.dev)]

    @staticmethod
    def to_fp8(x: torch.Tensor, block_rows: int):
        rows, cols = x.shape
        q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
        s = torch.empty((-(-rows // block_rows), -(-cols // 128)), dtype=torch.float32, device=x.device)
        moe.moe_quantize_fp8(x, q, s, block_rows)
        return q, s

    def buffers(self, T: int) -> dict:
        H = SHAPE[0]
        zeros = lambda n: torch.zeros(n, dtype=torch.uint8, device=self.dev)
        new = lambda *s, d=torch.float16: torch.empty(s, dtype=d, device=self.dev)
        return {"ids": new(T, TOP_K, d=torch.int32), "w": new(T, TOP_K, d=torch.float32), "ysh": new(T, H),
                "y": new(T, H), "ws_shared": zeros(moe.moe_shared_fp8_workspace_bytes(T, H, SHARED)),
                "ws_fp16": zeros(moe.moe_shared_workspace_bytes(T, H, SHARED)),
                "ws": zeros(moe.moe_forward_workspace_bytes(SHAPE, T, TOP_K, E))}

    def __call__(self, x: torch.Tensor, logits: torch.Tensor, b: dict, fp8: bool = True) -> torch.Tensor:
        if fp8:
            moe.moe_shared_forward_fp8(x, *self.fp8, b["ysh"], b["ws_shared"])
        else:
            moe.moe_shared_forward(x, self.fp16["wg"], self.fp16["wu"], self.fp16["wd"], b["ysh"], b["ws_fp16"])
        moe.moe_layer_forward_scored(SHAPE, x, self.router, logits, TOP_K, self.bias, b["ids"], b["w"], self.pool,
                                     self.slot_of, E, b["ysh"], b["y"], b["ws"])
        return b["y"]


def timed(f, n: int = 200) -> float:
    """us per call, enqueued back to back."""
    for _ in range(20):
        f()
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(n):
        f()
    stop.record()
    torch.cuda.synchronize()
    return start.elapsed_time(stop) * 1e3 / n


def main():
    layer = Layer()
    for T in (1, 512):
        gen = torch.Generator(device="cuda").manual_seed(T)
        x = torch.randn((T, SHAPE[0]), generator=gen, device="cuda").half()
        logits = torch.randn((T, E), generator=gen, device="cuda")
        b = layer.buffers(T)
        y8 = layer(x, logits, b).float()
        used = torch.bincount(b["ids"].flatten().clamp(min=0), minlength=E)
        y16 = layer(x, logits, b, fp8=False).float()
        for ws in ("ws", "ws_shared", "ws_fp16"):
            assert moe.moe_workspace_flags(b[ws]) == 0
        off = float((y8 - y16).norm() / y16.norm())
        t8, t16 = timed(lambda: layer(x, logits, b)), timed(lambda: layer(x, logits, b, fp8=False))
        print(f"{T:4d} tokens: {int((used > 0).sum())} experts used, FP8 against FP16 shared path: relative difference "
              f"{off:.4f}, layer {t8:.1f} us against {t16:.1f} us")


if __name__ == "__main__":
    main()
