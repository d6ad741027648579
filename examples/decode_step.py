"""A decode step that is captured once and replayed: pages planned on the device, projections in 4-bit floats,
rotary positions, the cache, its attention, the norms between the blocks and the MoE layer.

    lengths, pages      moe_kv_plan: each sequence's next tokens get positions, slots and, where needed, pages
    x                   moe_block_norm of the residual
    q, k, v             moe_linear_fp4, one projection
    q turned, k, v put  moe_rope_kv_write: heads normalised, turned, keys and values into the cache
    a                   moe_attn_paged
    residual, x         moe_linear_fp4 back to the model's width, then moe_block_norm: its output normalised, gated,
                        added to the residual, and the sum normalised for the experts
    residual            moe_layer_forward, then moe_block_norm again

Prompts of several lengths are run as one chunk each; then every step adds a token to each sequence, one of them ends on
the way and another takes its place in the batch.  The same graph serves all steps, since lengths live on the device.
The script checks its outputs against the same steps without a graph.

    python examples/decode_step.py [bf16|e4m3|int4]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_layer_sigmoid_gb300 as moe  # noqa: E402

FORMATS = {"bf16": moe.MOE_KV_BF16, "e4m3": moe.MOE_KV_E4M3, "int4": moe.MOE_KV_INT4}
d, H, H_kv, D, page, n_pages, max_pages, window = 256, 8, 2, 64, 16, 60, 12, 100     # attention
E, k, F, Fs, group = 16, 2, 128, 128, 32                                            # experts
EPS = 1e-6


class Block:
    """One block's weights, its cache and page state, and what a program keeps for its calls of up to T tokens."""

    def __init__(self, fmt, B, T, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        bf16 = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.fmt, self.B, self.T = FORMATS[fmt], B, T
        self.w_qkv = moe.fp4(*moe.moe_pack_fp4(rand((H + 2 * H_kv) * D, d) / math.sqrt(d)))
        self.w_o = moe.fp4(*moe.moe_pack_fp4(rand(d, H * D) / math.sqrt(H * D)))
        self.W_r, self.bias = rand(E, d) / math.sqrt(d), rand(E) * 0.5
        self.packed = [moe.moe_pack_w4(rand(r, c) / math.sqrt(c), group) for r, c in
                       ((E * 2 * F, d), (E * d, F), (2 * Fs, d), (d, Fs))]
        self.experts = [moe.w4(*p) for p in self.packed]
        self.norms = [1 + 0.1 * rand(d) for _ in range(4)]
        self.gate = rand(d)
        # angles for long contexts: frequencies below one turn in 64 positions eight times as slow
        table = torch.empty(max_pages * page, D // 2, device="cuda")
        moe.moe_rope_table(moe.RopeConfig(base=10000.0, factor=8.0, orig_len=64.0, lo=1.0, hi=4.0, magnitude=1.0, rot=D // 2,
                                          scaling=moe.MOE_ROPE_BAND), 0, table)
        self.rope = moe.rope(table, 0, 1 + 0.1 * rand(D), 1 + 0.1 * rand(D), EPS)
        row = {"bf16": D, "e4m3": D, "int4": D // 2}[fmt]
        kind = torch.bfloat16 if fmt == "bf16" else torch.uint8
        pool = [torch.zeros((n_pages, H_kv, page, row), dtype=kind, device="cuda") for _ in range(2)]
        scales = [None if fmt == "bf16" else torch.zeros((n_pages, H_kv, page), device="cuda") for _ in range(2)]
        self.pool = pool + scales
        self.cache = moe.kv_cache(*self.pool)
        self.kv_len, self.first, self.pages = ints(B), ints(B), ints(B, max_pages) - 1
        self.free, self.n_free = torch.arange(n_pages, dtype=torch.int32, device="cuda"), ints(1) + n_pages
        self.held = moe.kv_pages(self.kv_len, self.first, self.pages, self.free, self.n_free)
        self.new, self.q_off, self.pos, self.slots = ints(B), ints(B + 1), ints(T), ints(T)
        self.x, self.qkv, self.q, self.a = bf16(T, d), bf16(T, (H + 2 * H_kv) * D), bf16(T, H, D), bf16(T, H, D)
        self.y, self.residual = bf16(T, d), bf16(T, d)
        self.kv = moe.KvDims(T=T, B=B, H=H, H_kv=H_kv, D=D, page=page, n_pages=n_pages, max_pages=max_pages, max_new=0,
                             window=window, format=self.fmt, flags=0)
        self.ws_attn = moe.workspace(moe.moe_attn_workspace_bytes(self.kv))
        self.ws_fp4 = moe.workspace(max(moe.moe_linear_fp4_workspace_bytes(T, (H + 2 * H_kv) * D, d),
                                        moe.moe_linear_fp4_workspace_bytes(T, d, H * D)))
        self.layer = moe.Dims(T=T, d=d, E=E, k=k, F=F, F_s=Fs, group=group, flags=0)
        self.ws_moe = moe.workspace(moe.moe_layer_workspace_bytes(self.layer))

    def step(self):
        """One pass of self.residual [T][d] through the block: self.new[b] more tokens for each sequence."""
        plain = moe.NormDims(T=self.T, d=d, gate=moe.MOE_GATE_NONE, flags=0, eps=EPS, scale=1.0)
        gated = moe.NormDims(T=self.T, d=d, gate=moe.MOE_GATE_CHANNEL, flags=moe.MOE_NORM_SIGMOID, eps=EPS, scale=0.5)
        moe.moe_kv_plan(self.new, self.kv, self.held, self.q_off, self.pos, self.slots, self.ws_attn)
        moe.moe_block_norm(None, self.residual, None, None, self.norms[0], plain, None, self.x)
        moe.moe_linear_fp4(self.x, self.w_qkv, self.qkv, self.ws_fp4)
        q, kn, vn = self.qkv.split((H * D, H_kv * D, H_kv * D), dim=1)
        moe.moe_rope_kv_write(q.view(self.T, H, D), kn.view(self.T, H_kv, D), vn.view(self.T, H_kv, D), self.pos,
                              self.slots, self.rope, self.kv, self.cache, self.q, self.ws_attn)
        moe.moe_attn_paged(self.q, self.q_off, self.kv_len, self.pages, self.kv, self.cache, 1 / math.sqrt(D), self.a,
                           None, self.ws_attn)
        moe.moe_linear_fp4(self.a.view(self.T, H * D), self.w_o, self.y, self.ws_fp4)
        moe.moe_block_norm(self.y, self.residual, self.gate, self.norms[1], self.norms[2], gated, self.residual, self.x)
        moe.moe_layer_forward(self.x, self.W_r, self.bias, self.layer, *self.experts, self.y, self.ws_moe)
        moe.moe_block_norm(self.y, self.residual, None, self.norms[3], None, plain, self.residual, None)

    def status(self):
        return [moe.moe_check_device_status(ws) for ws in (self.ws_attn, self.ws_fp4, self.ws_moe)]


def plan(seed=0):
    """New tokens of each of three sequences, step by step: prompts, single tokens, an end and a new prompt."""
    yield [19, 7, 14]
    for i in range(90):
        yield [1, -(1 << 31), 1] if i == 30 else [1, 23, 1] if i == 31 else [1, 1, -3] if i == 50 else [1, 1, 1]


def main(fmt="e4m3", seed=0):
    """The largest difference between replayed and plain steps' outputs, whether the states are the same, and the lengths."""
    T = 40
    eager, graphed = Block(fmt, 3, T, seed), Block(fmt, 3, T, seed)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    graphed.step()                      # (a first pass on empty sequences: everything is loaded before the capture)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        graphed.step()
    g, off = torch.Generator(device="cuda").manual_seed(seed + 1), 0.0
    for new in plan():
        x = torch.randn((T, d), generator=g, device="cuda").to(torch.bfloat16)
        n = sum(v for v in new if v > 0)
        for block in (eager, graphed):
            block.new.copy_(torch.tensor(new, dtype=torch.int32))
            block.residual.copy_(x)
        eager.step()
        graph.replay()
        off = max(off, (eager.residual[:n].float() - graphed.residual[:n].float()).abs().max().item())
        assert torch.isfinite(eager.residual[:n].float()).all()
    torch.cuda.synchronize()
    assert eager.status() == graphed.status() == [moe.MOE_OK] * 3
    same = all(torch.equal(a, b) for a, b in zip((eager.kv_len, eager.pages, eager.first), (graphed.kv_len, graphed.pages, graphed.first)))
    print(f"{fmt}: lengths {eager.kv_len.tolist()}, outputs of replayed steps off by {off}, states {'the same' if same else 'differ'}")
    return off, same, eager.kv_len.tolist()


if __name__ == "__main__":
    main(*sys.argv[1:2])
