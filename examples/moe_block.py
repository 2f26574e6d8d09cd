"""A small offloaded-MoE decoder without attention, from bf16 weights to a token:

  experts   bf16 -> NVFP4 banks of pinned host blobs (moe_fp4_global_scale, moe_fp4_quantize);
  per layer  pre-norm (moe_block_norm) -> ids and weights (moe_route) -> cached experts
             (moe_decode_layer) -> post-norm, gate, residual and the next pre-norm in one
             pass (moe_block_norm);
  head       the last hidden state to 4 bits and through the 4-bit head (moe_fp4_linear).

Run on a GB300: python examples/moe_block.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import expert_slot_cache_lru_gb300 as m  # noqa: E402

BF16 = torch.bfloat16


def bank_offsets(hidden: int, inter: int) -> tuple[list[int], list[int], int]:
    """Byte offsets of an NVFP4 blob's gate / up / down code and scale banks and its
    three global scales (layout of moe_cache.h)."""
    ih = hidden * inter
    return ([0, ih // 2, ih], [3 * ih // 2 + i * (ih // 16) for i in range(3)],
            3 * ih // 2 + 3 * (ih // 16))


def quantize_matrix(w: torch.Tensor, codes, scales, glob) -> None:
    """One bf16 matrix into a code bank, a scale bank and its global scale (device addresses)."""
    rows, cols = w.shape
    m.moe_fp4_global_scale(w, m.MOE_T_BF16, rows, cols, glob)
    m.moe_fp4_quantize(m.MOE_W_NVFP4, w, m.MOE_T_BF16, rows, cols, glob, codes, scales)


def expert_blob(gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor) -> torch.Tensor:
    """A device NVFP4 blob of three bf16 matrices ([I][H], [I][H], [H][I])."""
    inter, hidden = gate.shape
    code, scale, glob = bank_offsets(hidden, inter)
    blob = torch.zeros(m.blob_bytes(m.MOE_W_NVFP4, hidden, inter), dtype=torch.uint8, device="cuda")
    at = blob.data_ptr()
    for i, w in enumerate((gate, up, down)):
        quantize_matrix(w, at + code[i], at + scale[i], at + glob + 4 * i)
    return blob


class Decoder:
    """n_layers MoE layers of n_experts each, of which n_slots fit the device."""

    def __init__(self, *, n_layers=4, n_experts=32, top_k=4, hidden=1024, inter=512, vocab=4096,
                 n_slots=64, rows=1, seed=0):
        self.L, self.E, self.k, self.H, self.V, self.B = n_layers, n_experts, top_k, hidden, vocab, rows
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(BF16)  # noqa: E731
        self.blobs = []  # pinned host copies, one per (layer, expert)
        for _ in range(n_layers * n_experts):
            w = [normal(inter, hidden, std=0.02), normal(inter, hidden, std=0.02),
                 normal(hidden, inter, std=0.02)]
            self.blobs.append(expert_blob(*w).cpu().pin_memory())
        nbytes = self.blobs[0].numel()
        stride = (nbytes + 255) // 256 * 256
        self.cache = m.SlotCache(
            n_layers=n_layers, n_experts=n_experts, n_slots=n_slots, pool_mode=m.MOE_POOL_SHARED,
            hidden=hidden, inter=inter, wfmt=m.MOE_W_NVFP4,
            slot_storage=torch.empty(n_slots * stride, dtype=torch.uint8, device="cuda"),
            slot_stride=stride, host_blob_ptrs=[b.data_ptr() for b in self.blobs],
            max_routes=rows * top_k, max_rows=rows, keepalive=self.blobs)
        self.router = [normal(n_experts, hidden, std=hidden ** -0.5) for _ in range(n_layers)]
        self.bias = [torch.randn(n_experts, generator=g, device="cuda") * 0.01 for _ in range(n_layers)]
        one = lambda: (1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).to(BF16)  # noqa: E731
        self.pre = [one() for _ in range(n_layers + 1)]   # the last one precedes the head
        self.post = [one() for _ in range(n_layers)]
        self.gate = [normal(hidden, std=0.5) for _ in range(n_layers)]
        self.embed = normal(vocab, hidden)
        # the head in 4 bits, with the scale its inputs are calibrated to
        self.head_c = torch.empty(vocab, hidden // 2, dtype=torch.uint8, device="cuda")
        self.head_s = torch.empty(vocab, hidden // 16, dtype=torch.uint8, device="cuda")
        self.head_g = torch.empty(1, device="cuda")
        quantize_matrix(normal(vocab, hidden, std=0.02), self.head_c, self.head_s, self.head_g)
        self.x_g = torch.tensor([8.0 / 2688.0], device="cuda")
        # work buffers of a step
        dev = dict(device="cuda")
        self.h = torch.empty(rows, hidden, **dev)
        self.x, self.y = (torch.empty(rows, hidden, dtype=BF16, **dev) for _ in range(2))
        self.z = torch.empty(rows, n_experts, **dev)
        self.ids, self.slots = (torch.empty(rows, top_k, dtype=torch.int32, **dev) for _ in range(2))
        self.w = torch.empty(rows, top_k, **dev)
        self.xc = torch.empty(rows, hidden // 2, dtype=torch.uint8, **dev)
        self.xs = torch.empty(rows, hidden // 16, dtype=torch.uint8, **dev)
        self.logits = torch.empty(rows, vocab, **dev)
        self.side = torch.cuda.Stream()

    def step(self, tokens: torch.Tensor, trace=None) -> torch.Tensor:
        """Next tokens [rows].  trace: called as trace(layer, decoder) after each layer's experts
        (layer < n_layers) and at the end."""
        B, H, h, x, y = self.B, self.H, self.h, self.x, self.y
        h.copy_(self.embed[tokens])
        m.moe_block_norm(h, None, None, None, self.pre[0], None, x, B, H, res_dtype=m.MOE_T_F32)
        for layer in range(self.L):
            m.moe_route(x, self.router[layer], self.bias[layer], B, H, self.E, self.k, self.z, self.ids,
                        self.w, score=m.MOE_SCORE_SIGMOID, n_groups=4, topk_groups=2, group_top=2,
                        scale=2.5)
            m.moe_decode_layer(self.cache.handle, layer, x, self.ids, self.w, self.slots, B, self.k, -1,
                               None, 0, None, None, y, None, self.side, m.MOE_OVERLAP)
            if trace:
                trace(layer, self)
            m.moe_block_norm(h, y, self.post[layer], self.gate[layer], self.pre[layer + 1], h, x, B, H,
                             res_dtype=m.MOE_T_F32, gate_kind=m.MOE_GATE_SIGMOID, alpha=0.5)
        m.moe_fp4_quantize(m.MOE_W_NVFP4, x, m.MOE_T_BF16, B, H, self.x_g, self.xc, self.xs)
        m.moe_fp4_linear(m.MOE_W_NVFP4, self.xc, self.xs, self.x_g, self.head_c, self.head_s, self.head_g,
                         B, self.V, H, self.logits, m.MOE_T_F32)
        if trace:
            trace(self.L, self)
        return self.logits.argmax(1)


def main(steps: int = 32) -> None:
    d = Decoder()
    tokens = torch.zeros(d.B, dtype=torch.long, device="cuda")
    out = []
    for _ in range(steps):
        tokens = d.step(tokens)
        out.append(tokens)
    print("tokens:", torch.stack(out, 1).tolist())
    misses = sum(d.cache.stats(layer)["misses"] for layer in range(d.L))
    print(f"{misses} expert misses in {steps} steps of {d.L} layers")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 32)
