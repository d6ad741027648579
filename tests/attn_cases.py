"""Paged-cache batches for the attention tests: a filled pool, a page table and the attention
of its new tokens in 64 bits, written from the definition without any of the library's code."""
import math
from dataclasses import dataclass

import torch

FORMATS = ("bf16", "e4m3", "int4")


def e4m3_table():
    """The 256 E4M3 values (1-4-3 bits, bias 7, no infinities, code 0x7F is NaN)."""
    out = []
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        x = math.nan if (e, f) == (15, 7) else f / 512 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        out.append(-x if c & 128 else x)
    return torch.tensor(out, dtype=torch.float64)


def quantise(x, fmt):
    """bf16 rows -> (codes, fp32 scales): the recipe in 64 bits, its two stated fp32 roundings
    (scale and quotient) made explicit."""
    x = x.double()
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    s = (x.abs().amax(-1) / (448 if fmt == "e4m3" else 7)).float()
    y = torch.where(s[..., None] > 0, x / s.double()[..., None], 0.0).float().double()
    if fmt == "int4":
        n = y.round().clamp(-8, 7).to(torch.int32) & 15
        return (n[..., 0::2] | n[..., 1::2] << 4).to(torch.uint8), s
    t = e4m3_table()[:127].to(y.device)  # the non-negative finite values, ascending by code
    a = y.abs().clamp(max=448.0)
    hi = torch.bucketize(a, t).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - t[lo], t[hi] - a
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | (torch.signbit(y) * 128)).to(torch.uint8), s


def values(codes, scales, fmt):
    """What codes and scales stand for, in 64 bits."""
    if fmt == "bf16":
        return codes.double()
    if fmt == "e4m3":
        x = e4m3_table().to(codes.device)[codes.long()]
    else:
        n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int32)
        x = ((n ^ 8) - 8).double()
    return x * scales.double()[..., None]


def slots_view(x, layout):
    """The same rows [pages][heads][slots][row] with token-major pages ("tokens"), or in a pool
    that holds other layers' pages between them ("strided")."""
    if layout == "tokens":
        return x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    if layout == "strided":
        wide = torch.zeros((x.shape[0], 3, *x.shape[1:]), dtype=x.dtype, device=x.device)
        wide[:, 1] = x
        return wide[:, 1]
    return x.contiguous()


@dataclass
class Batch:
    new: list
    total: list
    H: int
    H_kv: int
    D: int
    page: int
    fmt: str
    window: int
    scale: float
    q: torch.Tensor
    q_off: torch.Tensor
    kv_len: torch.Tensor
    pages: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    ks: torch.Tensor
    vs: torch.Tensor

    def dims(self, moe, **kw):
        d = dict(T=sum(self.new), B=len(self.new), H=self.H, H_kv=self.H_kv, D=self.D,
                 page=self.page, n_pages=self.k.shape[0], max_pages=self.pages.shape[1],
                 max_new=max(self.new), window=self.window, format=FORMATS.index(self.fmt), flags=0)
        d.update(kw)
        return moe.KvDims(**d)

    def cache(self, moe):
        return moe.kv_cache(self.k, self.v, self.ks, self.vs)


def make(new, total, H, H_kv, D, page, fmt, window=0, layout="heads", seed=0, spread=1.5, spare=2,
         first_page=0, poison=True, device="cuda"):
    """A batch with random rows.  Slots that no token sees, and page-table entries of pages
    without a seen key, hold what must never matter: NaN rows or codes, NaN scales, ids far
    outside the pool."""
    g = torch.Generator(device=device).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    need = [max(0, -(-t // page)) for t in total]
    n_pages, max_pages = first_page + sum(need) + spare, max(max(need), 1)
    order = first_page + torch.randperm(sum(need) + spare, generator=cpu)
    table = torch.full((len(new), max_pages), 0x7FFFFFF0, dtype=torch.int32)
    seen = torch.zeros((n_pages, page), dtype=torch.bool)
    o = 0
    for b, (n, t) in enumerate(zip(new, total)):
        ids = order[o:o + need[b]]
        o += need[b]
        # keys that some token of the sequence sees: those of its positions >= 0
        first, last = max(0, t - n), t - 1
        lo = max(0, first - window + 1) if window else 0
        if n == 0 or last < 0:
            continue
        for p in range(lo // page, last // page + 1):
            table[b, p] = ids[p]
            seen[ids[p], max(0, lo - p * page):min(page, last + 1 - p * page)] = True
    shape = (n_pages - first_page, H_kv, page, D)
    unseen = ~seen.to(device)[first_page:, None, :].expand(shape[:3])

    def pool(gain):
        x = torch.randn(shape, generator=g, device=device, dtype=torch.float32) * gain
        codes, s = quantise(x.to(torch.bfloat16), fmt)
        if poison:
            codes[unseen] = math.nan if fmt == "bf16" else 0x7F
            if s is not None:
                s[unseen] = math.nan
        if first_page:  # the rows live far from the pool's start
            far = torch.empty((n_pages, *shape[1:3], codes.shape[-1]), dtype=codes.dtype, device=device)
            far[first_page:] = codes
            codes = far
            if s is not None:
                far = torch.empty((n_pages, *shape[1:3]), dtype=s.dtype, device=device)
                far[first_page:] = s
                s = far
        return slots_view(codes, layout), s

    k, ks = pool(spread)
    v, vs = pool(1.0)
    T = sum(new)
    wide = torch.randn((T, (H + 2 * H_kv) * D), generator=g, device=device).to(torch.bfloat16)
    return Batch(new, total, H, H_kv, D, page, fmt, window, 1 / math.sqrt(D),
                 wide[:, :H * D].view(T, H, D),
                 torch.tensor([0] + new).cumsum(0).to(torch.int32).to(device),
                 torch.tensor(total, dtype=torch.int32).to(device), table.to(device), k, v, ks, vs)


def reference(b: Batch):
    """(out, lse, bound of out, bound of lse) in 64 bits.

    Bounds, from the stated numerics.  A score is a sum of D exact products in fp32: off by at
    most e = D * 2^-23 * S + |s| * 2^-22, S the sum of the products' magnitudes (2^-23, as a
    tensor core may cut instead of rounding).  Each weight e^s is then off by the factor e of
    its own score and the maximum's, by 2^-21 in the exponential, and by 2^-8 when it is
    rounded to bf16 (eight significant bits: half of the last is 2^-8 of the first); the sums
    add n * 2^-24 at most.  So out is off by at most A * (2^-8 + 2 * (2 e + 2^-21 + n * 2^-23))
    with A = sum p |v|, and its own rounding adds 2^-8 * A; lse by 2 e + 2^-20 + n * 2^-24.  A weight, or its product with a value's scale,
    below the smallest normal number 2^-126 may vanish before it meets a code of up to 448:
    n * 2^-117 * max(1, |v|) at most."""
    T, G = sum(b.new), b.H // b.H_kv
    dev = b.q.device
    out = torch.zeros((T, b.H, b.D), dtype=torch.float64, device=dev)
    lse = torch.full((T, b.H), -math.inf, dtype=torch.float64, device=dev)
    bo, bl = torch.zeros_like(out), torch.zeros_like(lse)
    t0 = 0
    for i, (n, t) in enumerate(zip(b.new, b.total)):
        for r in range(n):
            pos = t - n + r
            if pos < 0:
                continue
            lo = max(0, pos - b.window + 1) if b.window else 0
            j = torch.arange(lo, pos + 1, device=dev)
            pg, at = b.pages[i, j // b.page].long(), j % b.page
            k, v = (values(p[pg, :, at], None if s is None else s[pg, :, at], b.fmt)
                    for p, s in ((b.k, b.ks), (b.v, b.vs)))          # [keys][H_kv][D]
            q = b.q[t0 + r].double().view(b.H_kv, G, b.D)
            s = torch.einsum("hgd,jhd->hgj", q, k) * b.scale
            S = torch.einsum("hgd,jhd->hgj", q.abs(), k.abs()) * b.scale
            z = s.logsumexp(-1)
            p = (s - z[..., None]).exp()
            e = (b.D * 2.0 ** -23 * S + s.abs() * 2.0 ** -22).amax(-1)
            A = torch.einsum("hgj,jhd->hgd", p, v.abs())
            out[t0 + r] = torch.einsum("hgj,jhd->hgd", p, v).reshape(b.H, b.D)
            lse[t0 + r] = z.reshape(-1)
            rel = 2.0 ** -7 + 2 * (2 * e + 2.0 ** -21 + len(j) * 2.0 ** -23)
            tiny = len(j) * 2.0 ** -117 * v.abs().max().clamp(min=1.0)
            bo[t0 + r] = (A * rel[..., None] + tiny).reshape(b.H, b.D)
            bl[t0 + r] = (2 * e + 2.0 ** -20 + len(j) * 2.0 ** -24).reshape(-1)
        t0 += n
    return out, lse, bo, bl


def check(b: Batch, out, lse):
    ref, z, bo, bl = reference(b)
    assert torch.isfinite(out.float()).all()
    d = (out.double() - ref).abs()
    worst = (d / bo.clamp(min=2.0 ** -120)).max().item() if d.numel() else 0.0
    assert (d <= bo).all(), f"out is off by {worst:.2f} times its bound"
    empty = torch.isinf(z)
    assert torch.equal(torch.isinf(lse.double()), empty)
    dz = (lse.double() - z)[~empty].abs()
    assert (dz <= bl[~empty]).all()
