"""What a decoder block needs around its attention and its experts, as measured cases.

Four operators:

* ``plan`` -- block tables and slot maps from request lengths: pages of a cache given to sequences
  that grow, taken back from those that shrink or leave a window;
* ``rope`` -- rotary positions: the table of angles, and queries and keys rotated (their heads
  normalised first where the model does) as keys and values are written into the cache;
* ``norm`` -- the norms after one block and before the next with the gate, the scale and the residual
  between them;
* ``fp4``  -- microscaled 4-bit floats: rows to codes and back, and a projection of both operands in codes.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits) or,
with ``own`` set, through the library's calls.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

CASES = {
    # a decode step of a batch at chat lengths planned, and its tokens rejected again: all latency
    "plan_decode": dict(op="plan", B=32, chunks=0, idle=3, new_lo=1, new_hi=1, ctx_lo=63, ctx_hi=4095,
                        page=16, window=0, pad=3, lens=1),
    # chunks of prompts admitted beside a large decode batch with a sliding window
    "plan_chunks": dict(op="plan", B=500, chunks=37, idle=11, new_lo=300, new_hi=2048, ctx_lo=0, ctx_hi=8190,
                        page=16, window=1024, pad=100, lens=2),
    # the angles of a long context, frequencies scaled over a ramp of wavelengths
    "rope_table": dict(op="table", n_pos=131072, pos0=0, rot=128, base=500000.0, scaling="ramp", factor=32.0,
                       orig=4096.0, lo=1.0, hi=64.0, magnitude=1.3466),
    # one decoded token with normalised heads into an eight-bit cache: the smallest call, all latency
    "rope_token": dict(op="rope", T=1, pad=0, H=32, H_kv=8, D=128, rot=128, layout="half", norm=True,
                       format="e4m3", page=16, n_pos=8192, spread=True),
    # a decode step's batch, padded to a fixed size, half of narrow heads rotated in the interleaved
    # layout, into a four-bit cache
    "rope_batch": dict(op="rope", T=256, pad=17, H=28, H_kv=4, D=64, rot=32, layout="pairs", norm=False,
                       format="int4", page=32, n_pos=131072, spread=True),
    # a long prompt with normalised heads, half of each rotated, into a bf16 cache
    "rope_bulk": dict(op="rope", T=65537, pad=0, H=32, H_kv=8, D=128, rot=64, layout="half", norm=True,
                      format="bf16", page=64, n_pos=131072, spread=False),
    # one decoded token between attention and experts: the smallest call
    "norm_token": dict(op="norm", T=1, d=4096, post=True, pre=True, gate="none", sigmoid=False, res="bf16", scale=1.0),
    # a small batch with a gate per token, an odd width and a 32-bit residual
    "norm_batch": dict(op="norm", T=257, d=5000, post=True, pre=True, gate="token", sigmoid=True, res="fp32",
                       scale=0.5),
    # a prompt's chunk with a gate per element
    "norm_prefill": dict(op="norm", T=8192, d=4096, post=False, pre=True, gate="full", sigmoid=False, res="bf16",
                         scale=0.22),
    # one decoded token through the fused projection of queries, keys and values
    "fp4_token": dict(op="linear", T=1, K=4096, N=6144),
    # a prompt's chunk through the same
    "fp4_chunk": dict(op="linear", T=2048, K=4096, N=6144),
    # a batch of activations to codes and back
    "fp4_rows": dict(op="rows", T=8191, K=4096),
}
FORMATS = ("bf16", "e4m3", "int4")
SCALINGS = ("none", "linear", "ramp", "band")
GATES = ("none", "token", "channel", "full")
EPS = 1e-6


def listed():
    return [dict(c, name=name) for name, c in CASES.items()]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, even over the logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    most = max(_cost(c) for c in CASES.values())
    while True:
        op = rng.choice(("plan", "table", "rope", "rope", "norm", "norm", "linear", "linear", "rows"))
        if op == "plan":
            B = _spread(rng, 1, 4000)
            chunks = rng.choice((0, rng.randrange(0, min(B, 64) + 1)))
            c = dict(op=op, B=B, chunks=chunks, new_lo=1, new_hi=_spread(rng, 1, 1000), ctx_hi=_spread(rng, 1, 16000),
                     page=rng.choice((16, 32, 64, 128, 256)), window=rng.choice((0, 0, _spread(rng, 1, 4096))),
                     pad=rng.choice((0, _spread(rng, 1, 300))), lens=rng.randrange(1 << 20))
            c.update(ctx_lo=rng.randrange(0, c["ctx_hi"]), idle=rng.randrange(0, B - chunks) if B > chunks else 0)
        elif op == "table":
            c = dict(op=op, n_pos=_spread(rng, 1, 131072), pos0=rng.choice((0, _spread(rng, 1, 1 << 20))),
                     rot=16 * rng.randrange(1, 9), base=rng.choice((10000.0, 500000.0, 1e6)),
                     scaling=rng.choice(SCALINGS), factor=rng.choice((2.0, 8.0, 40.0)),
                     orig=rng.choice((2048.0, 8192.0)), lo=1.0, hi=rng.choice((4.0, 32.0)),
                     magnitude=rng.choice((1.0, 1.2079)))
        elif op == "rope":
            H_kv, D, T = rng.choice((1, 2, 4, 8)), rng.choice((64, 128)), _spread(rng, 1, 65537)
            fmt = rng.choice(FORMATS)
            c = dict(op=op, T=T, pad=rng.choice((0, rng.randrange(0, T))), H=H_kv * rng.choice((1, 2, 3, 4, 5, 7, 8)),
                     H_kv=H_kv, D=D, rot=16 * rng.randrange(1, D // 16 + 1), layout=rng.choice(("half", "pairs")),
                     # (a four-bit code is a seventh of the row's largest value wide, and a sum's last bit moves
                     # it where it lies on the border of two: heads are not normalised before those)
                     norm=fmt != "int4" and rng.random() < 0.5, format=fmt, page=rng.choice((16, 32, 64, 128)),
                     n_pos=max(T, _spread(rng, 1, 131072)), spread=rng.random() < 0.5)
        elif op == "norm":
            post, gate = rng.random() < 0.6, rng.choice(GATES)
            c = dict(op=op, T=_spread(rng, 1, 16384), d=8 * _spread(rng, 8, 2048), post=post, pre=rng.random() < 0.9,
                     gate=gate, sigmoid=gate != "none" and rng.random() < 0.5, res=rng.choice(("bf16", "bf16", "fp32")),
                     scale=rng.choice((1.0, 0.5, 1.4)))
        elif op == "linear":
            c = dict(op=op, T=_spread(rng, 1, 4096), K=64 * _spread(rng, 2, 128), N=8 * _spread(rng, 16, 1024))
        else:
            c = dict(op=op, T=_spread(rng, 1, 16384), K=64 * _spread(rng, 1, 160))
        if _cost(c) <= most:
            return c


# ------------------------------------------------------------------ shapes of a case

def _lengths(c):
    """New tokens and earlier tokens of each sequence: a case's own numbers."""
    rng = random.Random(c["lens"])
    new, ctx = [], []
    for b in range(c["B"]):
        if b >= c["B"] - c["idle"]:
            new.append(0)
            ctx.append(_spread(rng, c["ctx_lo"] + 1, c["ctx_hi"] + 1) - 1 if b % 2 else 0)
            continue
        new.append(_spread(rng, c["new_lo"], c["new_hi"]) if b < c["chunks"] else 1)
        ctx.append(_spread(rng, c["ctx_lo"] + 1, c["ctx_hi"] + 1) - 1)
    return new, ctx


def _row_bytes(c):
    """Bytes of one token's key (or value) of one head: codes and scale."""
    return {"bf16": 2 * c["D"], "e4m3": c["D"] + 4, "int4": c["D"] // 2 + 4}[c["format"]]


def work(case):
    c = case
    if c["op"] == "plan":
        new, ctx = _lengths(c)
        page, T = c["page"], sum(new) + c["pad"]
        grown = sum(-(-(n + m) // page) - -(-m // page) for n, m in zip(new, ctx))
        # two calls: lengths in and out; a position and a slot for each token; ids moved there and back
        return {"bytes": 4 * (2 * (3 * c["B"] + 2 + 2 * c["B"]) + 2 * T + 4 * grown), "flops": 4 * T}
    if c["op"] == "table":
        return {"bytes": 4 * c["n_pos"] * c["rot"], "flops": 20 * c["n_pos"] * c["rot"]}
    if c["op"] == "rope":
        T = c["T"] - c["pad"]
        heads = c["H"] + 2 * c["H_kv"]
        codes = 2 * c["H_kv"] * _row_bytes(c)
        back = 0 if c["format"] == "bf16" else T * codes + c["T"] * 4 * c["H_kv"] * c["D"]
        # new rows and table rows in, queries and cache rows out; cache rows of codes in and values out
        return {"bytes": T * (heads * 2 * c["D"] + 4 * c["rot"] + 2 * c["H"] * c["D"] + codes) + back,
                "flops": T * heads * c["D"] * (6 if c["norm"] else 3)}
    if c["op"] == "norm":
        res = 4 if c["res"] == "fp32" else 2
        row = c["d"] * (2 + 2 * res + (2 if c["pre"] else 0) + (2 if c["gate"] == "full" else 0))
        return {"bytes": c["T"] * row + 4 * c["d"] * (c["post"] + c["pre"]), "flops": 10 * c["T"] * c["d"]}
    T, K = c["T"], c["K"]
    if c["op"] == "rows":
        return {"bytes": T * (2 * K + 2 * (K // 2 + K // 16 + 4) + 2 * K), "flops": 4 * T * K}
    N = c["N"]
    return {"bytes": 2 * T * K + N * (K // 2 + K // 16 + 4) + 2 * T * N, "flops": 2 * T * N * K}


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


# ------------------------------------------------------------------ what a program has in hand

class _State:
    pass


def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _fp4_codes(x):
    """Rows to 4-bit codes (sign and magnitude index), block scales as E4M3 bytes and row scales."""
    x = x.float()
    s = x.abs().amax(dim=-1)
    s = s / torch.full_like(s, 2688.0)   # a division: by a plain number it would be a product
    blocks = x.view(*x.shape[:-1], -1, 16)
    m, six = blocks.abs().amax(dim=-1), (s * 6.0)[..., None].expand(blocks.shape[:-1])
    b = _e4m3(torch.where(six > 0, m / six, torch.zeros_like(m)))
    t = (b.float() * s[..., None])[..., None].expand_as(blocks)
    y = torch.where(t > 0, blocks / t, torch.zeros_like(blocks))
    a = y.abs()
    # the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; ties to the even index
    i = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    i = (i | (torch.signbit(y).to(torch.uint8) << 3)).view(x.shape)
    return i, b.view(torch.uint8), s


def _scale_place(R, blocks, device):
    """Where the scale of row r and block j lies: tiles of 128 rows and 4 blocks, 512 bytes each."""
    r = torch.arange(R, device=device)[:, None]
    j = torch.arange(blocks, device=device)
    return ((r // 128) * (blocks // 4) + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4


def _fp4_store(codes, b):
    """Two codes a byte, the even element low; block scales in their tiles."""
    R, blocks = b.shape
    tiles = torch.zeros(-(-R // 128) * (blocks // 4) * 512, dtype=torch.uint8, device=b.device)
    tiles[_scale_place(R, blocks, b.device)] = b
    return codes[:, 0::2] | codes[:, 1::2] << 4, tiles


def _fp4_values(q, tiles, s):
    """What stored codes stand for, in 32 bits."""
    R, blocks = q.shape[0], q.shape[1] // 8
    i = torch.stack((q & 15, q >> 4), dim=-1).view(R, blocks, 16).long()
    size = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    v = torch.cat((size, -size))[i]
    b = tiles[_scale_place(R, blocks, q.device)].view(torch.float8_e4m3fn).float()
    return (v * (b * s[:, None])[..., None]).view(R, -1)


def _frequencies(c, device):
    """The angle of each pair from one position to the next, in 64 bits."""
    half = torch.arange(c["rot"] // 2, dtype=torch.float64, device=device)
    f = torch.exp(half * (-2.0 * math.log(c["base"]) / c["rot"]))
    if c["scaling"] == "linear":
        return f / c["factor"]
    if c["scaling"] == "ramp":   # over the pair's index, between those that turn `hi` and `lo` times
        a, b = (c["rot"] * math.log(c["orig"] / (2 * math.pi * t)) / (2 * math.log(c["base"])) for t in (c["hi"], c["lo"]))
        a, b = max(math.floor(a), 0), min(math.ceil(b), c["rot"] - 1)
        m = ((half - a) / max(b - a, 0.001)).clamp(0, 1)
        return f * (1 - m) + f / c["factor"] * m
    if c["scaling"] == "band":   # over the turns themselves
        m = ((c["orig"] * f / (2 * math.pi) - c["lo"]) / (c["hi"] - c["lo"])).clamp(0, 1)
        return f * m + f / c["factor"] * (1 - m)
    return f


def _table(c, device):
    p = torch.arange(c["pos0"], c["pos0"] + c["n_pos"], dtype=torch.float64, device=device)
    a = p[:, None] * _frequencies(c, device)
    return torch.cat((a.cos(), a.sin()), dim=1).mul_(c["magnitude"])


def prepare(case, seed):
    c, s = case, _State()
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    randn = lambda *shape, dtype=torch.bfloat16: torch.randn(shape, generator=gen, device=dev, dtype=dtype)  # noqa: E731
    s.case = c
    if c["op"] == "plan":
        new, ctx = _lengths(c)
        page, W, B = c["page"], c["window"], c["B"]
        # pages behind the window have been given back by the steps before
        first = [max(0, m - W + 1) // page if W else 0 for m in ctx]
        held = [-(-m // page) for m in ctx]
        need = sum(-(-(n + m) // page) - h for n, m, h in zip(new, ctx, held))
        n_pages = sum(h - f for h, f in zip(held, first)) + need + 5
        s.max_pages = max(-(-(n + m) // page) for n, m in zip(new, ctx)) + 2
        order = torch.randperm(n_pages, generator=cpu).to(torch.int32)
        table, o = torch.full((B, s.max_pages), -1, dtype=torch.int32), 0
        for b in range(B):
            table[b, first[b]:held[b]] = order[o:o + held[b] - first[b]]
            o += held[b] - first[b]
        free = torch.full((n_pages,), -1, dtype=torch.int32)
        free[: n_pages - o] = order[o:]
        ints = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
        s.new, s.drop, s.kv_len, s.first = ints(new), ints([-n for n in new]), ints(ctx), ints(first)
        s.pages, s.free, s.n_free = table.cuda(), free.cuda(), ints([n_pages - o])
        s.n_pages, s.T = n_pages, sum(new) + c["pad"]
        empty = lambda n: torch.empty(n, dtype=torch.int32, device=dev)  # noqa: E731
        s.q_off, s.pos, s.slots = empty(B + 1), empty(s.T), empty(s.T)
        s.q_off2, s.pos2, s.slots2 = empty(B + 1), empty(s.T), empty(s.T)
    elif c["op"] == "table":
        s.out = torch.empty((c["n_pos"], c["rot"]), device=dev)
        # (a user's scaling is a setting; another seed is another first position and base)
        s.cfg = dict(c, pos0=c["pos0"] + seed % 1000, base=c["base"] * (1 + seed % 97 / 1000))
    elif c["op"] == "rope":
        T, H, H_kv, D, page = c["T"], c["H"], c["H_kv"], c["D"], c["page"]
        s.live = T - c["pad"]
        at = (torch.randint(0, c["n_pos"], (T,), generator=cpu) if c["spread"]
              else torch.arange(T) + torch.randint(0, c["n_pos"] - T + 1, (1,), generator=cpu))
        n_pages = -(-T // page) + 5
        slots = torch.randperm(n_pages, generator=cpu)[torch.arange(T) // page] * page + torch.arange(T) % page
        at[s.live:] = -1
        slots[s.live:] = -1
        s.pos, s.slots = at.to(torch.int32).cuda(), slots.to(torch.int32).cuda()
        s.table = _table(dict(pos0=0, n_pos=c["n_pos"], rot=c["rot"], base=500000.0, scaling="band", factor=8.0,
                              orig=8192.0, lo=1.0, hi=4.0, magnitude=1.0), dev).float()
        s.q_w = 1 + 0.1 * randn(D, dtype=torch.float32) if c["norm"] else None
        s.k_w = 1 + 0.1 * randn(D, dtype=torch.float32) if c["norm"] else None
        # queries, keys and values lie side by side, as one projection leaves them; a few channels of
        # the keys are much larger than the others, as in trained models
        qkv = randn(T, (H + 2 * H_kv) * D)
        s.q = qkv[:, : H * D].view(T, H, D)
        s.k_new = qkv[:, H * D: (H + H_kv) * D].view(T, H_kv, D)
        s.v_new = qkv[:, (H + H_kv) * D:].view(T, H_kv, D)
        gain = torch.ones(D, device=dev, dtype=torch.bfloat16)
        gain[torch.randperm(D, generator=cpu)[: D // 32].cuda()] = 4.0
        s.k_new *= gain
        s.q_out = torch.zeros((T, H, D), dtype=torch.bfloat16, device=dev)
        pool = (n_pages, H_kv, page)
        if c["format"] == "bf16":
            s.k, s.v, s.ks, s.vs = randn(*pool, D), randn(*pool, D), None, None
        else:
            row = D if c["format"] == "e4m3" else D // 2
            s.k, s.v = (torch.zeros((*pool, row), dtype=torch.uint8, device=dev) for _ in range(2))
            s.ks, s.vs = (torch.zeros(pool, device=dev) for _ in range(2))
        s.k_back = torch.empty((T, H_kv, D), dtype=torch.bfloat16, device=dev)
        s.v_back = torch.empty_like(s.k_back)
        s.n_pages = n_pages
    elif c["op"] == "norm":
        T, d = c["T"], c["d"]
        s.y = randn(T, d)
        s.r = randn(T, d, dtype=torch.float32).mul_(3.0).to(torch.float32 if c["res"] == "fp32" else torch.bfloat16)
        s.w_post = 1 + 0.2 * randn(d, dtype=torch.float32) if c["post"] else None
        s.w_pre = 1 + 0.2 * randn(d, dtype=torch.float32) if c["pre"] else None
        s.gate = {"none": lambda: None, "token": lambda: randn(T, dtype=torch.float32),
                  "channel": lambda: randn(d, dtype=torch.float32), "full": lambda: randn(T, d)}[c["gate"]]()
        s.r_out = torch.empty_like(s.r)
        s.x = torch.empty_like(s.y) if c["pre"] else None
    else:
        T, K = c["T"], c["K"]
        s.x = randn(T, K)
        # a few channels of the activations are much larger than the others, as in trained models
        s.x[:, torch.randperm(K, generator=cpu)[: max(1, K // 256)].cuda()] *= 16.0
        if c["op"] == "linear":
            N = c["N"]
            codes, b, s.s = _fp4_codes(randn(N, K, dtype=torch.float32) / math.sqrt(K))
            s.q, s.b = _fp4_store(codes, b)
            s.out = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
        else:
            blank = lambda n, t: torch.empty(n, dtype=t, device=dev)  # noqa: E731
            s.q, s.s = blank((T, K // 2), torch.uint8), blank(T, torch.float32)
            s.b = blank(-(-T // 128) * (K // 64) * 512, torch.uint8)
            s.out = torch.empty_like(s.x)
    if own:  # the sizes, handles and workspace that a program sets up once
        import moe_expert_layer_sigmoid_gb300 as moe
        if c["op"] == "plan":
            s.dims = moe.KvDims(T=s.T, B=c["B"], H=1, H_kv=1, D=64, page=c["page"], n_pages=s.n_pages,
                                max_pages=s.max_pages, max_new=0, window=c["window"], format=moe.MOE_KV_BF16, flags=0)
            s.held = moe.kv_pages(s.kv_len, s.first, s.pages, s.free, s.n_free)
            s.ws = moe.workspace(256)
        elif c["op"] == "table":
            g = s.cfg
            s.rope = moe.RopeConfig(base=g["base"], factor=g["factor"], orig_len=g["orig"], lo=g["lo"], hi=g["hi"],
                                    magnitude=g["magnitude"], rot=g["rot"], scaling=SCALINGS.index(g["scaling"]))
        elif c["op"] == "rope":
            s.dims = moe.KvDims(T=c["T"], B=1, H=c["H"], H_kv=c["H_kv"], D=c["D"], page=c["page"], n_pages=s.n_pages,
                                max_pages=1, max_new=0, window=0, format=FORMATS.index(c["format"]), flags=0)
            s.cache = moe.kv_cache(s.k, s.v, s.ks, s.vs)
            s.rope = moe.rope(s.table, moe.MOE_ROPE_PAIRS if c["layout"] == "pairs" else 0, s.q_w, s.k_w, EPS)
            s.ws = moe.workspace(256)
        elif c["op"] == "norm":
            s.dims = moe.NormDims(T=c["T"], d=c["d"], gate=GATES.index(c["gate"]),
                                  flags=(moe.MOE_NORM_SIGMOID if c["sigmoid"] else 0) |
                                        (moe.MOE_NORM_RESIDUAL_F32 if c["res"] == "fp32" else 0),
                                  eps=EPS, scale=c["scale"])
        elif c["op"] == "linear":
            s.w = moe.fp4(s.q, s.b, s.s)
            s.ws = moe.workspace(moe.moe_linear_fp4_workspace_bytes(c["T"], c["N"], c["K"]))
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    s, op = state, state.case["op"]
    if own:
        import moe_expert_layer_sigmoid_gb300 as moe
    if op == "plan":
        if own:
            moe.moe_kv_plan(s.new, s.dims, s.held, s.q_off, s.pos, s.slots, s.ws)
            moe.moe_kv_plan(s.drop, s.dims, s.held, s.q_off2, s.pos2, s.slots2, s.ws)
        else:
            _plain_plan(s, s.new, s.q_off, s.pos, s.slots)
            _plain_plan(s, s.drop, s.q_off2, s.pos2, s.slots2)
        return {"q_off": s.q_off, "pos": s.pos, "slots": s.slots, "q_off2": s.q_off2, "pos2": s.pos2,
                "slots2": s.slots2, "kv_len": s.kv_len, "first": s.first, "pages": s.pages, "free": s.free,
                "n_free": s.n_free}
    if op == "table":
        if own:
            moe.moe_rope_table(s.rope, s.cfg["pos0"], s.out)
        else:
            s.out.copy_(_table(s.cfg, s.out.device))
        return s.out
    if op == "rope":
        if own:
            moe.moe_rope_kv_write(s.q, s.k_new, s.v_new, s.pos, s.slots, s.rope, s.dims, s.cache, s.q_out, s.ws)
            if s.ks is not None:
                moe.moe_kv_read(s.slots, s.dims, s.cache, s.k_back, s.v_back, s.ws)
        else:
            _plain_rope(s)
        if s.ks is None:
            return {"q": s.q_out, "k": s.k, "v": s.v}
        return {"q": s.q_out, "k": s.k_back, "v": s.v_back, "ks": s.ks, "vs": s.vs}
    if op == "norm":
        if own:
            moe.moe_block_norm(s.y, s.r, s.gate, s.w_post, s.w_pre, s.dims, s.r_out, s.x)
        else:
            _plain_norm(s)
        return {"r": s.r_out} if s.x is None else {"r": s.r_out, "x": s.x}
    if op == "linear":
        if own:
            moe.moe_linear_fp4(s.x, s.w, s.out, s.ws)
        else:
            codes, b, sx = _fp4_codes(s.x)
            s.out.copy_(_fp4_values(*_fp4_store(codes, b), sx) @ _fp4_values(s.q, s.b, s.s).T)
        return s.out
    if own:
        moe.moe_quant_rows_fp4(s.x, s.q, s.b, s.s)
        moe.moe_unpack_fp4(s.q, s.b, s.s, s.out)
    else:
        codes, b, sx = _fp4_codes(s.x)
        s.s.copy_(sx)
        s.out.copy_(_fp4_values(*_fp4_store(codes, b), sx))
    return {"values": s.out, "s": s.s}


def _plain_plan(s, n, q_off, pos, slots):
    c, dev = s.case, n.device
    page, W, B, M, N, T = c["page"], c["window"], c["B"], s.max_pages, s.n_pages, s.T
    n, L, first = n.long(), s.kv_len.long(), s.first.long()
    up = lambda x: (x + page - 1).div(page, rounding_mode="floor")  # noqa: E731
    held = up(L)
    short = n < 0
    after = torch.where(short, (L + n).clamp(min=0), L)
    # what goes back: the tail of a sequence that gets shorter, what a growing one's window has left
    seen = (L - W + 1).clamp(min=0).div(page, rounding_mode="floor") if W else torch.zeros_like(L)
    new_first = torch.where(short, torch.where(after > 0, first, torch.zeros_like(first)), torch.maximum(first, seen))
    lo = torch.where(short, torch.maximum(up(after), first), first)
    hi = torch.where(short, held, new_first)
    back = hi - lo
    slot = torch.arange(M, device=dev)
    gone = (slot >= lo[:, None]) & (slot < hi[:, None])
    rank = (back.cumsum(0) - back - lo)[:, None] + slot
    R, have = back.sum(), s.n_free.long()
    total = have + R
    spill = torch.full((N + 1,), -1, dtype=torch.int32, device=dev)
    spill[:N] = s.free
    spill[torch.where(gone, have + R - 1 - rank, N)] = s.pages
    s.pages.masked_fill_(gone, -1)
    # what is given: sequences in order, as far as tokens and pages last
    want = torch.where(short, torch.zeros_like(n), n)
    need = torch.where(want > 0, up(after + want) - up(after), torch.zeros_like(n))
    fits = (want.cumsum(0) <= T) & ((need == 0) | (need.cumsum(0) <= total))
    want, need = torch.where(fits, want, 0), torch.where(fits, need, 0)
    start = need.cumsum(0) - need
    base = up(after)
    mine = (slot >= base[:, None]) & (slot < (base + need)[:, None])
    take = (total - 1 - start + base)[:, None] - slot
    s.pages.copy_(torch.where(mine, spill[torch.where(mine, take, N)], s.pages))
    s.free.copy_(spill[:N])
    s.n_free.copy_(total - need.sum())
    s.kv_len.copy_(after + want)
    s.first.copy_(new_first)
    q_off.zero_()
    q_off[1:] = want.cumsum(0)
    # tokens in order
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(q_off[1:].long(), t, right=True)
    live = b < B
    b = b.clamp(max=B - 1)
    at = after[b] + t - q_off[b]
    page_id = s.pages.view(-1)[(b * M + at.div(page, rounding_mode="floor")).clamp(0, B * M - 1)].long()
    pos.copy_(torch.where(live, at, -1))
    slots.copy_(torch.where(live, page_id * page + at.remainder(page), -1))


def _rotated(x, w, cos, sin, rot, pairs):
    """Rows [T][heads][D] in 32 bits: each head normalised with weights w, then its first part rotated."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * w
    part = x[..., :rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if pairs else (part[..., : rot // 2], part[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, v), dim=-1).flatten(-2) if pairs else torch.cat((u, v), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


def _coded(x, fmt):
    """The values that codes of rows stand for, in 32 bits, and the rows' scales."""
    top = 448.0 if fmt == "e4m3" else 7.0
    m = x.abs().amax(dim=-1, keepdim=True)
    m = m / torch.full_like(m, top)   # a division: by a plain number it would be a product
    y = torch.where(m > 0, x / m, torch.zeros_like(x))
    y = _e4m3(y).float() if fmt == "e4m3" else y.round().clamp(-8, 7)
    return y * m, m.squeeze(-1)


def _plain_rope(s):
    c, n = s.case, s.live
    rot, page, pairs = c["rot"], c["page"], c["layout"] == "pairs"
    row = s.table[s.pos[:n].long()][:, None]
    cos, sin = row[..., : rot // 2], row[..., rot // 2:]
    s.q_out[:n] = _rotated(s.q[:n], s.q_w, cos, sin, rot, pairs).to(torch.bfloat16)
    k = _rotated(s.k_new[:n], s.k_w, cos, sin, rot, pairs)
    v = s.v_new[:n].float()
    live = s.slots[:n].long()
    p, at = live.div(page, rounding_mode="floor"), live.remainder(page)
    if c["format"] == "bf16":
        s.k[p, :, at] = k.to(torch.bfloat16)
        s.v[p, :, at] = v.to(torch.bfloat16)
        return
    (k, ks), (v, vs) = _coded(k, c["format"]), _coded(v, c["format"])
    s.ks[p, :, at] = ks
    s.vs[p, :, at] = vs
    s.k_back.zero_()
    s.v_back.zero_()
    s.k_back[:n] = k.to(torch.bfloat16)
    s.v_back[:n] = v.to(torch.bfloat16)


def _plain_norm(s):
    c = s.case
    u = s.y.float()
    if s.w_post is not None:
        u = u * torch.rsqrt(u.square().mean(dim=-1, keepdim=True) + EPS) * s.w_post
    if s.gate is not None:
        g = s.gate.float()
        g = 1 / (1 + torch.exp(-g)) if c["sigmoid"] else g
        u = u * (g[:, None] if c["gate"] == "token" else g)
    r = s.r.float() + c["scale"] * u
    s.r_out.copy_(r)
    if s.x is not None:
        s.x.copy_(r * torch.rsqrt(r.square().mean(dim=-1, keepdim=True) + EPS) * s.w_pre)


# ------------------------------------------------------------------ the definition, in 64 bits

def _eight_bits_64(y):
    """The nearest E4M3 value, ties to the even code."""
    e = torch.frexp(y.abs())[1].clamp(min=-5) - 1   # exponent, not below the smallest normal's
    step = torch.ldexp(torch.ones_like(y), e - 3)
    return ((y / step).round() * step).clamp(-448, 448)


def _four_bits_64(y):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with either sign, ties to the even code."""
    a = y.abs().clamp(max=6)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((a / step).round() * step, y)


def _fp4_64(x):
    """Rows of values as their codes stand for them, and the row scales: the recipe's 32-bit
    quotients are kept, since bf16 values lie between codes so often that the last bit decides."""
    x = x.double()
    s = (x.abs().amax(dim=1) / 2688).float().double()
    blocks = x.reshape(x.shape[0], -1, 16)
    six = (6 * s).float().double()[:, None]
    b = torch.where(six > 0, (blocks.abs().amax(dim=2) / six).float().double(), 0.0)
    b = _eight_bits_64(b)
    t = (b * s[:, None]).float().double()[..., None]
    y = torch.where(t > 0, (blocks / t).float().double(), 0.0)
    return (_four_bits_64(y) * (b * s[:, None])[..., None]).reshape(x.shape), s


def _normed_64(x, w):
    x = x.double()
    return x / (x.pow(2).mean(dim=-1, keepdim=True) + EPS).sqrt() * w.double() if w is not None else x


def exact(case, seed):
    c = case
    if c["op"] == "plan":
        return None
    s = prepare(case, seed)
    if c["op"] == "table":
        g, half = s.cfg, c["rot"] // 2
        f = []
        for i in range(half):
            w = g["base"] ** (-2.0 * i / g["rot"])
            turns = g["orig"] * w / (2 * math.pi)
            keep = 1.0
            if g["scaling"] == "linear":
                keep = 0.0
            elif g["scaling"] == "band":
                keep = min(1.0, max(0.0, (turns - g["lo"]) / (g["hi"] - g["lo"])))
            elif g["scaling"] == "ramp":
                index = lambda t: g["rot"] * math.log(g["orig"] / (2 * math.pi * t), g["base"]) / 2  # noqa: E731
                lo, hi = max(math.floor(index(g["hi"])), 0), min(math.ceil(index(g["lo"])), g["rot"] - 1)
                keep = 1 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f.append(w * keep + w / g["factor"] * (1 - keep))
        f = torch.tensor(f, dtype=torch.float64, device="cuda")
        out = torch.empty((g["n_pos"], 2 * half), dtype=torch.float64, device="cuda")
        turn = torch.arange(g["n_pos"], device="cuda").double().add(g["pos0"]).outer(f)
        out[:, :half] = g["magnitude"] * torch.cos(turn)
        out[:, half:] = g["magnitude"] * torch.sin(turn)
        return out
    if c["op"] == "rope":
        n, rot, half = s.live, c["rot"], c["rot"] // 2
        row = s.table.double()[s.pos[:n].long()]
        z = torch.complex(row[:, :half], row[:, half:])[:, None]
        out = []
        for x, w in ((s.q[:n], s.q_w), (s.k_new[:n], s.k_w)):
            y = _normed_64(x, w)
            part = y[..., :rot]
            even = torch.arange(half, device="cuda") * (2 if c["layout"] == "pairs" else 1)
            odd = even + (1 if c["layout"] == "pairs" else half)
            turned = torch.complex(part[..., even], part[..., odd]) * z
            y = y.clone()
            y[..., even], y[..., odd] = turned.real, turned.imag
            out.append(y)
        q = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
        q[:n] = out[0]
        live = s.slots[:n].long()
        p, at = live // c["page"], live % c["page"]
        found = {"q": q}
        for name, x, pool, scales in (("k", out[1], s.k, s.ks), ("v", s.v_new[:n].double(), s.v, s.vs)):
            if c["format"] == "bf16":
                pool = pool.double()
                pool[p, :, at] = x
                found[name] = pool
                continue
            top = 448 if c["format"] == "e4m3" else 7
            m = (x.abs().amax(dim=-1) / top).float().double()   # scales are held in 32 bits
            y = torch.where(m[..., None] > 0, x / m[..., None], 0.0).float().double()
            y = _eight_bits_64(y) if c["format"] == "e4m3" else y.round().clamp(-8, 7)
            back = torch.zeros(s.k_back.shape, dtype=torch.float64, device="cuda")
            back[:n] = y * m[..., None]
            scales = scales.double()
            scales[p, :, at] = m
            found[name], found[name + "s"] = back, scales
        return found
    if c["op"] == "norm":
        u = _normed_64(s.y, s.w_post)
        if s.gate is not None:
            g = s.gate.double()
            g = torch.sigmoid(g) if c["sigmoid"] else g
            u = u * (g.reshape(-1, 1) if c["gate"] == "token" else g)
        r = s.r.double() + u * c["scale"]
        return {"r": r} if s.x is None else {"r": r, "x": _normed_64(r, s.w_pre)}
    x, sx = _fp4_64(s.x)
    if c["op"] == "rows":
        return {"values": x, "s": sx}
    size = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    size = torch.cat((size, -size))
    w = torch.empty((c["N"], c["K"]), dtype=torch.float64, device="cuda")
    w[:, 0::2], w[:, 1::2] = size[(s.q % 16).long()], size[(s.q // 16).long()]
    # tiles of 128 rows and 4 blocks: 32 rows of 16 bytes, each the 4 blocks of 4 rows 32 apart
    tiles = s.b.view(-1, c["K"] // 64, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, c["K"] // 16)[: c["N"]]
    code = tiles.long()
    e, f = code >> 3 & 15, (code & 7).double()
    b = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2(e.double() - 10))
    w = w * (b * s.s.double()[:, None]).repeat_interleave(16, dim=1)
    return x @ w.T
