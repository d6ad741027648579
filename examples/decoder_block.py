"""A decoder block on the library: attention over a paged, quantised cache and the MoE layer.

Two prompts are prefilled in chunks and then decoded together, a batch per step:

    y = x + attention(norm(x))        moe_kv_write, then moe_attn_paged over the cache
    y = y + moe_layer(norm(y))        moe_layer_forward_residual

Each step writes the batch's new keys and values into the pages of their sequences and attends to
everything written so far.  The projections around the attention are plain matrix products; rotary
embedding and the vocabulary are left out.  The script checks the attention's outputs against the
whole sequences run as one chunk each, and reads one sequence's keys back from the cache.

    python examples/decoder_block.py [bf16|e4m3|int4]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_layer_sigmoid_gb300 as moe  # noqa: E402

FORMATS = {"bf16": moe.MOE_KV_BF16, "e4m3": moe.MOE_KV_E4M3, "int4": moe.MOE_KV_INT4}
d, H, H_kv, D, page, n_pages = 256, 8, 2, 64, 16, 64         # attention
E, k, F, Fs, group = 16, 2, 128, 128, 32                     # experts


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Block:
    """One block's weights, its cache pool and the workspaces a program keeps."""

    def __init__(self, fmt, max_tokens, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.w_qkv = (rand(d, (H + 2 * H_kv) * D) / math.sqrt(d)).to(torch.bfloat16)
        self.w_o = (rand(H * D, d) / math.sqrt(H * D)).to(torch.bfloat16)
        self.W_r, self.bias = rand(E, d) / math.sqrt(d), rand(E) * 0.5
        self.experts = [moe.w4(*p) for p in self._pack(rand)]
        row = {"bf16": D, "e4m3": D, "int4": D // 2}[fmt]
        dtype = torch.bfloat16 if fmt == "bf16" else torch.uint8
        pool = lambda: torch.zeros((n_pages, H_kv, page, row), dtype=dtype, device="cuda")  # noqa: E731
        scales = lambda: None if fmt == "bf16" else torch.zeros((n_pages, H_kv, page), device="cuda")  # noqa: E731
        self.tensors = [pool(), pool(), scales(), scales()]
        self.cache = moe.kv_cache(*self.tensors)
        self.fmt = FORMATS[fmt]
        self.ws_attn = moe.workspace(moe.moe_attn_workspace_bytes(self.kv_dims(max_tokens, 2, 16, 0)))
        self.ws_moe = moe.workspace(moe.moe_layer_workspace_bytes(self.moe_dims(max_tokens)))

    def _pack(self, rand):
        self._packed = [moe.moe_pack_w4(rand(r, c) / math.sqrt(c), group) for r, c in
                        ((E * 2 * F, d), (E * d, F), (2 * Fs, d), (d, Fs))]
        return self._packed

    def kv_dims(self, T, B, max_pages, max_new):
        return moe.KvDims(T=T, B=B, H=H, H_kv=H_kv, D=D, page=page, n_pages=n_pages,
                          max_pages=max_pages, max_new=max_new, window=0, format=self.fmt, flags=0)

    def moe_dims(self, T):
        return moe.Dims(T=T, d=d, E=E, k=k, F=F, F_s=Fs, group=group, flags=0)

    def forward(self, x, new, kv_len, pages):
        """x bf16 [T][d]: the `new[b]` next tokens of each sequence, kv_len[b] tokens with them;
        pages int32 [B][max_pages].  Returns (block output, attention output)."""
        T, B, dev = x.shape[0], len(new), x.device
        q_off = torch.tensor([0] + new).cumsum(0).to(torch.int32).to(dev)
        lens = torch.tensor(kv_len, dtype=torch.int32, device=dev)
        at = torch.cat([torch.arange(n_all - n, n_all) for n, n_all in zip(new, kv_len)]).to(dev)
        seq = torch.repeat_interleave(torch.arange(B), torch.tensor(new)).to(dev)
        slots = (pages[seq, at // page] * page + at % page).to(torch.int32)
        dims = self.kv_dims(T, B, pages.shape[1], max(new))
        qkv = norm(x) @ self.w_qkv
        q = qkv[:, :H * D].view(T, H, D)
        k_new = qkv[:, H * D:(H + H_kv) * D].view(T, H_kv, D)
        v_new = qkv[:, (H + H_kv) * D:].view(T, H_kv, D)
        moe.moe_kv_write(k_new, v_new, slots, dims, self.cache, self.ws_attn)
        a = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev)
        moe.moe_attn_paged(q, q_off, lens, pages, dims, self.cache, 1 / math.sqrt(D), a, None, self.ws_attn)
        y = x + a.view(T, H * D) @ self.w_o
        out = torch.empty_like(y)
        moe.moe_layer_forward_residual(norm(y), self.W_r, self.bias, self.moe_dims(T), *self.experts, y, out,
                                       self.ws_moe)
        return out, a


def main(fmt="e4m3", lengths=(75, 41), prompt=(64, 33), chunk=24, seed=0):
    """The largest difference of the attention's outputs, chunked and one by one against whole, over their
    root mean square."""
    B = len(lengths)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    xs = [torch.randn((n, d), generator=g, device="cuda").to(torch.bfloat16) for n in lengths]
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    pages = order[:B * 16].view(B, 16)
    # whole sequences, one chunk each
    whole = Block(fmt, sum(lengths), seed)
    ref_out, ref = whole.forward(torch.cat(xs), list(lengths), list(lengths), pages)
    # prompts in chunks, then all sequences a token at a time
    block, done = Block(fmt, sum(lengths), seed), [0] * B
    outs, attns = [[] for _ in xs], [[] for _ in xs]
    steps = 0
    while any(n < m for n, m in zip(done, lengths)):
        new = [min(chunk, p - n) if n < p else min(1, m - n) for n, p, m in zip(done, prompt, lengths)]
        done = [n + s for n, s in zip(done, new)]
        x = torch.cat([x[n - s:n] for x, n, s in zip(xs, done, new)])
        out, a = block.forward(x, new, done, pages)
        for b, (o, t) in enumerate(zip(out.split(new), a.split(new))):
            outs[b].append(o)
            attns[b].append(t)
        steps += 1
    for ws in (whole.ws_attn, whole.ws_moe, block.ws_attn, block.ws_moe):
        assert moe.moe_check_device_status(ws) == moe.MOE_OK
    got = torch.cat([torch.cat(t) for t in attns]).float()
    off = ((got - ref.float()).abs().max() / ref.float().square().mean().sqrt()).item()
    # both caches hold the same rows: read the second sequence's keys back from each
    at = torch.arange(lengths[1], device="cuda")
    slots = (pages[1][at // page] * page + at % page).to(torch.int32)
    dims = whole.kv_dims(lengths[1], 1, 16, 0)
    keys = torch.empty((2, 2, lengths[1], H_kv, D), dtype=torch.bfloat16, device="cuda")
    for i, b in enumerate((whole, block)):
        moe.moe_kv_read(slots, dims, b.cache, keys[i, 0], keys[i, 1], b.ws_attn)
    same = torch.equal(keys[0], keys[1])
    moved = (torch.cat([torch.cat(t) for t in outs]).float() - ref_out.float()).norm() / ref_out.float().norm()
    print(f"{fmt}: {steps} steps, attention off by at most {off:.2e} of its rms, block output by {moved:.2e} in "
          f"norm, caches {'the same' if same else 'differ'}")
    return off, same, moved.item()


if __name__ == "__main__":
    main(*sys.argv[1:2])
