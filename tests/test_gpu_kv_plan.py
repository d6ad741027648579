"""Page planning against a plain walk over the sequences, entry by entry: integers, so equal."""
import random

import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu


class Pool:
    """The state as plain lists, and the rules one by one."""

    def __init__(self, B, page, n_pages, max_pages, window, seed=0):
        self.B, self.page, self.n_pages, self.max_pages, self.window = B, page, n_pages, max_pages, window
        self.kv_len, self.first = [0] * B, [0] * B
        self.pages = [[-1] * max_pages for _ in range(B)]
        self.free = list(range(n_pages))
        random.Random(seed).shuffle(self.free)
        self.n_free = n_pages

    def up(self, n):
        return -(-n // self.page)

    def step(self, new, T):
        """(q_off, pos, slots, whether the device check trips)"""
        tripped = False
        back, grow = [], []
        for b, n in enumerate(new):
            L, f = self.kv_len[b], self.first[b]
            if n < 0:
                after = max(0, L + n)
                if after and f * self.page > max(0, after - self.window + 1):
                    tripped = True
                    continue
                back += [(b, i) for i in range(max(self.up(after), f), self.up(L))]
                self.kv_len[b] = after
                self.first[b] = f if after else 0
            elif L + n > self.max_pages * self.page:
                tripped = True
            else:
                if self.window:
                    now = max(f, max(0, L - self.window + 1) // self.page)
                    back += [(b, i) for i in range(f, now)]
                    self.first[b] = now
                grow.append((b, n))
        for b, i in reversed(back):
            self.free[self.n_free] = self.pages[b][i]
            self.n_free += 1
            self.pages[b][i] = -1
        tokens = need = 0
        room, q_off, rows = self.n_free, [0], []
        served = dict()
        for b, n in grow:
            more = self.up(self.kv_len[b] + n) - self.up(self.kv_len[b])
            tokens += n
            need += more
            if n and (tokens > T or (more and need > room)):
                tripped = True
                continue
            served[b] = n
            for i in range(self.up(self.kv_len[b]), self.up(self.kv_len[b]) + more):
                self.n_free -= 1
                self.pages[b][i] = self.free[self.n_free]
        for b in range(self.B):
            n = served.get(b, 0)
            for j in range(self.kv_len[b], self.kv_len[b] + n):
                rows.append((j, self.pages[b][j // self.page] * self.page + j % self.page))
            self.kv_len[b] += n
            q_off.append(q_off[-1] + n)
        rows += [(-1, -1)] * (T - len(rows))
        return q_off, [r[0] for r in rows], [r[1] for r in rows], tripped


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Device:
    def __init__(self, p):
        self.p = p
        self.kv_len, self.first, self.free, self.n_free = ints(p.kv_len), ints(p.first), ints(p.free), ints([p.n_free])
        self.pages = ints(p.pages).view(p.B, p.max_pages)
        self.state = moe.kv_pages(self.kv_len, self.first, self.pages, self.free, self.n_free)
        self.ws = moe.workspace(256)

    def dims(self, T):
        p = self.p
        return moe.KvDims(T=T, B=p.B, H=8, H_kv=2, D=64, page=p.page, n_pages=p.n_pages, max_pages=p.max_pages, max_new=0,
                          window=p.window, format=0, flags=0)

    def step(self, new, T):
        q_off, pos, slots = ints([7] * (self.p.B + 1)), ints([7] * T), ints([7] * T)
        moe.moe_kv_plan(ints(new), self.dims(T), self.state, q_off, pos, slots, self.ws)
        return q_off, pos, slots

    def check(self):
        p = self.p
        assert self.kv_len.tolist() == p.kv_len and self.first.tolist() == p.first
        assert self.pages.tolist() == p.pages
        assert self.n_free.tolist() == [p.n_free]
        assert self.free[:p.n_free].tolist() == p.free[:p.n_free]
        # every page is held by one sequence or free
        held = [i for row in p.pages for i in row if i >= 0]
        assert sorted(held + p.free[:p.n_free]) == list(range(p.n_pages))


def both(dev, new, T, tripped=None):
    want = dev.p.step(new, T)
    got = dev.step(new, T)
    for g, w in zip(got, want):
        assert g.tolist() == w
    dev.check()
    status = moe.moe_check_device_status(dev.ws)
    assert status == (moe.MOE_ERR_DEVICE_CHECK if want[3] else moe.MOE_OK)
    if tripped is not None:
        assert want[3] == tripped


@pytest.mark.parametrize("window", [0, 1, 20, 100])
@pytest.mark.parametrize("B,page,T", [(1, 16, 40), (5, 16, 64), (33, 32, 700), (700, 16, 3000)])
def test_steps(B, page, T, window):
    rng = random.Random(B * 1000 + window)
    dev = Device(Pool(B, page, 12 * B + 3, 20, window))
    for step in range(12):
        new = []
        for b in range(B):
            kind = rng.random()
            new.append(rng.randrange(0, 2 * T // B + 2) if kind < 0.3 else 1 if kind < 0.7 else 0 if kind < 0.8
                       else -rng.randrange(1, 8) if kind < 0.9 else -(1 << 31) if kind < 0.95 else -rng.randrange(1, 400))
        both(dev, new, T)


def test_room_runs_out():
    dev = Device(Pool(4, 16, 5, 10, 0))
    both(dev, [16, 40, 1, 16], 100, tripped=True)       # 1 + 3 + 1 pages: the fourth finds none left
    assert dev.p.kv_len == [16, 40, 1, 0]
    both(dev, [1, 8, 3, 0], 100, tripped=True)          # the first has a full page, the others room in theirs
    assert dev.p.kv_len == [16, 48, 4, 0]
    both(dev, [-16, 0, 0, 16], 100, tripped=False)      # what goes back serves the same step
    assert dev.p.kv_len == [0, 48, 4, 16]


def test_tokens_run_out():
    dev = Device(Pool(3, 16, 20, 10, 0))
    both(dev, [10, 10, 10], 20, tripped=True)
    assert dev.p.kv_len == [10, 10, 0]
    both(dev, [21, 5, 0], 20, tripped=True)     # what did not fit counts before those behind it
    assert dev.p.kv_len == [10, 10, 0]


def test_a_sequence_that_would_pass_its_table():
    dev = Device(Pool(2, 16, 40, 3, 0))
    both(dev, [48, 47], 200, tripped=False)
    both(dev, [1, 1], 200, tripped=True)
    assert dev.p.kv_len == [48, 48]
    both(dev, [(1 << 31) - 1, (1 << 31) - 1], 200, tripped=True)


def test_added_and_dropped_restores_the_state():
    dev = Device(Pool(9, 16, 100, 20, 0))
    both(dev, [5, 16, 17, 0, 31, 1, 2, 3, 48], 200)
    before = [t.clone() for t in (dev.kv_len, dev.first, dev.pages, dev.n_free)]
    free = dev.free[:dev.p.n_free].clone()
    new = [40, 1, 0, 16, 1, 15, 14, 13, 100]
    both(dev, new, 300, tripped=False)
    both(dev, [-n for n in new], 0, tripped=False)
    for t, w in zip((dev.kv_len, dev.first, dev.pages, dev.n_free), before):
        assert torch.equal(t, w)
    assert torch.equal(dev.free[:dev.p.n_free], free)


def test_no_sequences_and_no_rows():
    dev = Device(Pool(0, 16, 4, 2, 0))
    q_off, pos, slots = dev.step([], 5)
    assert q_off.tolist() == [0] and pos.tolist() == [-1] * 5 and slots.tolist() == [-1] * 5
    dev = Device(Pool(2, 16, 4, 2, 0))
    both(dev, [0, 0], 0, tripped=False)
    both(dev, [1, 0], 0, tripped=True)


def test_most_sequences():
    dev = Device(Pool(8192, 16, 8200, 1, 0))
    rng = random.Random(5)
    both(dev, [rng.randrange(0, 3) for _ in range(8192)], 16384)
    both(dev, [rng.randrange(-2, 3) for _ in range(8192)], 16384)


def test_long_sequences():
    # slots near 2^31, pages of 256, tables whose rows pass 2^31 bytes apart
    n, B = (1 << 23) - 1, 70
    pages = torch.full((B, n), -1, dtype=torch.int32, device="cuda")
    kv_len, first, free, n_free = ints([0] * B), ints([0] * B), torch.zeros(n, dtype=torch.int32, device="cuda"), ints([2])
    big = (n - 2) * 256 - 1
    kv_len[B - 1] = big
    free[:2] = ints([n - 1, 11])
    pages[B - 1, n - 3] = n - 2
    st, ws = moe.kv_pages(kv_len, first, pages, free, n_free), moe.workspace(256)
    new = ints([0] * B)
    new[0], new[B - 1] = 256, 2
    dims = moe.KvDims(T=300, B=B, H=8, H_kv=2, D=64, page=256, n_pages=n, max_pages=n, max_new=0, window=0, format=0,
                      flags=0)
    q_off, pos, slots = ints([0] * (B + 1)), ints([7] * 300), ints([7] * 300)
    moe.moe_kv_plan(new, dims, st, q_off, pos, slots, ws)
    assert q_off.tolist() == [0] + [256] * (B - 1) + [258]
    assert pos.tolist() == list(range(256)) + [big, big + 1] + [-1] * 42
    assert slots.tolist() == [11 * 256 + i for i in range(256)] + [(n - 2) * 256 + 255, (n - 1) * 256] + [-1] * 42
    assert pages[B - 1, n - 2].item() == n - 1 and pages[0, 0].item() == 11
    assert n_free.item() == 0 and moe.moe_check_device_status(ws) == moe.MOE_OK
    new.fill_(-(1 << 31))
    moe.moe_kv_plan(new, dims, st, q_off, pos, slots, ws)
    # the long sequence's entries, most of them never set, go back as they are, the last of the list first
    assert kv_len.sum().item() == 0 and n_free.item() == n and pages.max().item() == -1
    assert free[0].item() == n - 1 and free[1].item() == n - 2 and free[n - 1].item() == 11
    assert free[2:n - 1].max().item() == -1 and moe.moe_check_device_status(ws) == moe.MOE_OK


@pytest.mark.parametrize("what", ["kv_len_low", "kv_len_high", "first_low", "first_high", "n_free_low", "n_free_high", "page_id"])
def test_a_state_that_is_not_whole(what):
    dev = Device(Pool(3, 16, 12, 6, 0))
    both(dev, [20, 20, 20], 60, tripped=False)
    q_len, others = dev.kv_len.clone(), [1, 1, 1]
    if what == "kv_len_low":
        dev.kv_len[1] = -5
    if what == "kv_len_high":
        dev.kv_len[1] = 97
    if what == "first_low":
        dev.first[1] = -1
    if what == "first_high":
        dev.first[1] = 3
    if what == "n_free_low":
        dev.n_free[0] = -7
    if what == "n_free_high":
        dev.n_free[0] = 13
    if what == "page_id":
        dev.pages[1, 1] = 12
    q_off, pos, slots = dev.step(others, 8)
    assert moe.moe_check_device_status(dev.ws) == moe.MOE_ERR_DEVICE_CHECK
    if what.startswith(("kv_len", "first")):
        assert q_off.tolist() == [0, 1, 1, 2]
        assert dev.kv_len[0].item() == dev.kv_len[2].item() == 21
    else:
        assert q_off.tolist() == [0, 1, 2, 3] and pos.tolist()[:3] == [20] * 3
        assert (slots[1].item() == -1) == (what == "page_id")
    if what == "n_free_low":
        assert dev.n_free.item() == 0
    if what == "n_free_high":
        assert dev.n_free.item() == 12
    # ids for which the stack has no room are dropped
    if what == "n_free_high":
        dev.step([-30, -30, -30], 8)
        assert moe.moe_check_device_status(dev.ws) == moe.MOE_ERR_DEVICE_CHECK and dev.n_free.item() == 12


def test_the_binding_refuses():
    dev = Device(Pool(3, 16, 12, 6, 0))
    q_off, pos, slots = ints([0] * 4), ints([0] * 8), ints([0] * 8)
    for d in (dev.dims(8).replace(B=2), dev.dims(8).replace(n_pages=13), dev.dims(8).replace(max_pages=5)):
        with pytest.raises(ValueError):
            moe.moe_kv_plan(ints([1, 1, 1]), d, dev.state, q_off, pos, slots, dev.ws)
    for bad in ((ints([1, 1]), q_off, pos, slots), (ints([1, 1, 1]), q_off[:3], pos, slots),
                (ints([1, 1, 1]), q_off, pos[:7], slots), (ints([1, 1, 1]), q_off, pos, slots.cpu()),
                (ints([1, 1, 1]).long(), q_off, pos, slots)):
        with pytest.raises(ValueError):
            moe.moe_kv_plan(bad[0], dev.dims(8), dev.state, *bad[1:], dev.ws)


def test_captured_steps_follow_their_lengths():
    dev = Device(Pool(6, 16, 40, 10, 50))
    new = ints([3, 0, 17, 1, 1, 0])
    T = 40
    q_off, pos, slots = ints([0] * 7), ints([0] * T), ints([0] * T)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            moe.moe_kv_plan(new, dev.dims(T), dev.state, q_off, pos, slots, dev.ws)
    for n in ([3, 0, 17, 1, 1, 0], [1, 30, 1, 1, 1, 1], [-2, 1, 0, -50, 20, 0], [30, 0, 0, 0, 0, 30]):
        new.copy_(ints(n))
        g.replay()
        want = dev.p.step(n, T)
        torch.cuda.synchronize()
        assert [q_off.tolist(), pos.tolist(), slots.tolist()] == list(want[:3])
        dev.check()
