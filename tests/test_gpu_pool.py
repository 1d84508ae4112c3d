"""The pool's books (mla_pool_resize, mla_pool_fork, mla_pool_compact) against lists changed one
sequence after the other, and mla_cache_copy against whole blocks of bytes."""
import random

import numpy as np
import pytest

from oracle import upkeep

pytestmark = pytest.mark.gpu


class Pair:
    """A pool on the device and its oracle; every call is made of both and compared."""

    def __init__(self, S, W, N, bs, room=None):
        import mla_latent_kv_08_gb300 as mla
        import torch
        self.mla, self.torch = mla, torch
        self.shape = mla.Shape(num_heads=8, kv_lora_rank=32, rope_dim=8, v_head_dim=8, block_size=bs, num_blocks=N)
        self.pool, self.k = mla.Pool.allocate(self.shape, S, W), upkeep.Books(S, W, N, bs)
        self.room = room or max(S, N)
        self.copies = torch.full((self.room, 4), -5, dtype=torch.int32, device="cuda")
        self.n, self.left, self.status = (torch.full((1,), v, dtype=torch.int32, device="cuda") for v in (-5, -5, 0))

    def ints(self, v):
        return None if v is None else self.torch.tensor(v, dtype=self.torch.int32, device="cuda")

    def set(self, table, lens, ref):
        """Books made elsewhere."""
        self.pool.block_table.copy_(self.ints(table))
        self.pool.seq_lens.copy_(self.ints(lens))
        self.pool.ref_count.copy_(self.ints(ref))
        self.k = upkeep.Books.of(table, lens, ref, self.shape.block_size)

    def check(self, flags, copies, left, with_left=True):
        assert int(self.status) == flags
        assert int(self.n) == len(copies)
        got = self.copies.cpu().numpy()
        np.testing.assert_array_equal(got[:len(copies)], np.array(copies, np.int32).reshape(-1, 4))
        assert np.all(got[len(copies):] == -5)                  # the rest of the list is left as it was
        if with_left:
            assert int(self.left) == left
        np.testing.assert_array_equal(self.pool.block_table.cpu().numpy(), np.array(self.k.table()).reshape(self.pool.block_table.shape))
        np.testing.assert_array_equal(self.pool.seq_lens.cpu().numpy(), self.k.lens)
        np.testing.assert_array_equal(self.pool.ref_count.cpu().numpy(), self.k.ref)
        for t in (self.copies, self.n, self.left):
            t.fill_(-5)
        self.status.zero_()
        return flags

    def resize(self, new, with_left=True):
        new = list(new)
        self.mla.mla_pool_resize(self.pool, self.ints(new), self.copies, self.n, num_free=self.left if with_left else None, status=self.status)
        return self.check(*self.k.resize(new), with_left)

    def fork(self, parents, children, lens=None):
        self.mla.mla_pool_fork(self.pool, self.ints(parents), self.ints(children), self.copies, self.n, lens=self.ints(lens),
                               num_free=self.left, status=self.status)
        return self.check(*self.k.fork(parents, children, lens))

    def compact(self, room=None):
        c = self.copies if room is None else self.copies[:room]
        self.mla.mla_pool_compact(self.pool, c, self.n, num_live=self.left, status=self.status)
        return self.check(*self.k.compact(self.room if room is None else room))


def _books(rng, S, W, N, bs, empty=0.2, share=0.4):
    """Books as a pool of some age has them: blocks anywhere, common beginnings, some slots empty."""
    ids = list(range(N))
    rng.shuffle(ids)
    table, lens, ref = [], [], [0] * N
    for b in range(S):
        n = 0 if rng.random() < empty else rng.randint(1, W * bs)
        row = []
        if b and n and rng.random() < share:
            row = table[-1][:rng.randint(0, min(lens[-1], n) // bs)]
        fresh = -(-n // bs) - len(row)
        if fresh > len(ids) - S:
            n, row, fresh = 0, [], 0
        row = row + [ids.pop() for _ in range(fresh)]
        for i in row:
            ref[i] += 1
        table.append(row + [-1] * (W - len(row)))
        lens.append(n)
    return table, lens, ref


SIZES = [(1, 1, 1, 1), (2, 3, 7, 1), (3, 5, 12, 4), (17, 9, 130, 16), (40, 30, 700, 64), (5, 700, 3000, 2), (130, 3, 129, 64), (1030, 4, 2500, 3)]


@pytest.mark.parametrize("S,W,N,bs", SIZES)
def test_a_long_life(gpu_lib, S, W, N, bs):
    """Random calls in a row, refused ones among them."""
    rng = random.Random(S * 7 + N)
    p = Pair(S, W, N, bs)
    seen = set()
    for step in range(40):
        what = rng.random()
        lens = p.k.lens
        if what < 0.55:
            new = [n if rng.random() < 0.3 else 0 if rng.random() < 0.2 else min(W * bs, max(0, n + rng.randint(-2 * bs - 3, 2 * bs + 3)))
                   if rng.random() < 0.8 else rng.randint(0, W * bs) for n in lens]
            if rng.random() < 0.05:
                new[rng.randrange(S)] = rng.choice([-1, W * bs + 1, 2 ** 31 - 1, -2 ** 31])
            seen.add(("resize", p.resize(new, with_left=step % 3 > 0)))
        elif what < 0.85:
            empty = [b for b in range(S) if lens[b] == 0]
            rng.shuffle(empty)
            children = empty[:rng.randint(1, max(1, len(empty)))] or [rng.randrange(S)]
            parents = [rng.randrange(S) for _ in children]
            some = None if rng.random() < 0.5 else [rng.randint(0, lens[a]) for a in parents]
            if rng.random() < 0.1:
                rng.choice([parents, children])[0] = rng.choice([-1, S, 2 ** 31 - 1, 0])
            seen.add(("fork", p.fork(parents, children, some)))
        else:
            seen.add(("compact", p.compact(rng.choice([None, 0, 1, 3]))))
    if S > 2:
        assert ("resize", 0) in seen and ("compact", 0) in seen


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("S,W,N,bs", [(20, 40, 500, 16), (64, 300, 9000, 64), (300, 60, 70000, 64), (16, 2000, 20000, 1)])
def test_a_pool_of_some_age(gpu_lib, S, W, N, bs, seed):
    rng = random.Random(seed)
    p = Pair(S, W, N, bs)
    books = _books(rng, S, W, N, bs)
    p.set(*books)
    assert p.compact(rng.choice([None, 1, N // 10])) == 0
    p.set(*books)
    new = [rng.choice([n, 0, max(0, n - rng.randint(0, 3 * bs)), rng.randint(0, n), min(W * bs, n + rng.randint(0, bs + 2))]) for n in books[1]]
    assert p.resize(new) in (0, upkeep.FULL)
    p.set(*books)
    empty = [b for b in range(S) if books[1][b] == 0]
    full = [b for b in range(S) if books[1][b]]
    if empty and full:
        parents = [rng.choice(full) for _ in empty]
        assert p.fork(parents, empty, [rng.randint(0, books[1][a]) for a in parents]) in (0, upkeep.FULL)
        p.set(*books)
        assert p.fork([full[0]] * len(empty), empty) in (0, upkeep.FULL)


def test_everything_and_nothing(gpu_lib):
    """The last free block, one too many, all given back, none asked for."""
    p = Pair(3, 4, 8, 8)
    assert p.resize([32, 32, 0]) == 0                        # all eight blocks
    assert p.resize([32, 32, 1]) == upkeep.FULL
    assert p.resize([32, 25, 0]) == 0
    assert p.fork([1], [2], [25]) == upkeep.FULL             # its tail needs a block
    assert p.fork([1], [2], [24]) == 0                       # whole blocks need none
    assert p.compact() == 0                                  # nothing to move
    assert p.resize([0, 0, 0]) == 0
    assert p.resize([0, 0, 0]) == 0
    assert p.compact() == 0


def test_both_holders_cut(gpu_lib):
    """Two sequences cut inside the block that they share in one call: both get their own, the
    shared one is free; cut by one alone while the other gives it up or keeps it."""
    for other in (5, 0, 16):
        p = Pair(3, 4, 12, 8)
        p.resize([16, 0, 0])
        p.fork([0], [1])
        assert p.resize([3, other, 0]) == 0
        assert p.resize([30, 20, 9]) == 0


def test_refused_forks_change_nothing(gpu_lib):
    p = Pair(6, 4, 30, 8)
    p.resize([20, 32, 0, 0, 0, 7])
    for parents, children, lens in (([0, 1], [2, 2], None), ([0], [1], None), ([0, 6], [2, 3], None), ([0, -1], [2, 3], None),
                                    ([0, 1], [2, -1], None), ([0, 1], [2, 6], None), ([0, 1], [3, 4], [21, 1]), ([0, 1], [3, 4], [1, -1])):
        assert p.fork(parents, children, lens) == upkeep.BOUNDS
    assert p.fork([0, 0, 2], [2, 3, 4], [20, 8, 0]) == 0     # a parent twice; a child that is a parent, of no tokens
    assert p.fork([4], [4]) == 0                             # nothing of itself


def test_bad_block_ids_are_refused(gpu_lib):
    import torch
    for bad in (-1, 30, 2 ** 31 - 1, -2 ** 31):
        p = Pair(3, 4, 30, 8)
        p.resize([20, 32, 0])
        p.pool.block_table[0, 1] = bad
        before = [t.clone() for t in (p.pool.block_table, p.pool.seq_lens, p.pool.ref_count)]
        three = [p.ints(v) for v in ([12, 32, 8], [0, 40 - 8, 0], [4, 0, 32])]
        for new in three:
            p.mla.mla_pool_resize(p.pool, new, p.copies, p.n, num_free=p.left, status=p.status)
            assert int(p.status) & 1 and int(p.n) == 0 and int(p.left) == 30 - 7
            p.status.zero_()
        for n in (20, 12):                                   # among the shared ones, and the one that is copied
            p.mla.mla_pool_fork(p.pool, p.ints([0]), p.ints([2]), p.copies, p.n, lens=p.ints([n]), num_free=p.left, status=p.status)
            assert int(p.status) & 1 and int(p.n) == 0
            p.status.zero_()
        for t, b in zip((p.pool.block_table, p.pool.seq_lens, p.pool.ref_count), before):
            assert torch.equal(t, b)
        p.mla.mla_pool_compact(p.pool, p.copies, p.n, status=p.status)         # raises the flag; the entry stays as it is
        assert int(p.status) & 1 and int(p.pool.block_table[0, 1]) == bad


def test_bad_lengths_are_refused(gpu_lib):
    for bad in (-1, 33, 2 ** 31 - 1):
        p = Pair(3, 4, 30, 8)
        p.resize([20, 32, 0])
        p.pool.seq_lens[1] = bad
        for call in (lambda: p.mla.mla_pool_resize(p.pool, p.ints([1, 2, 3]), p.copies, p.n, status=p.status),
                     lambda: p.mla.mla_pool_fork(p.pool, p.ints([1]), p.ints([2]), p.copies, p.n, status=p.status),
                     lambda: p.mla.mla_pool_compact(p.pool, p.copies, p.n, status=p.status)):
            call()
            assert int(p.status) == upkeep.BOUNDS and int(p.n) == 0
            assert p.mla.mla_read_status_word(p.status)[0] == p.mla.MLA_ERR_BOUNDS
            p.status.zero_()
        assert int(p.pool.ref_count.sum()) == 7 and int(p.pool.seq_lens[0]) == 20


def test_many_sequences_and_blocks(gpu_lib):
    """As many sequences and forks as a call takes, in a pool of a million blocks."""
    S, N = 16384, 1 << 20
    p = Pair(S, 8, N, 4, room=S)
    new = [(b * 7) % 33 if b < S - 5000 else 0 for b in range(S)]
    assert p.resize(new) == 0
    assert p.fork([b for b in range(5000)], [S - 1 - b for b in range(5000)]) == 0
    assert p.resize([n // 3 for n in p.k.lens]) == 0
    p.room = p.copies.shape[0]
    assert p.compact() == 0


def test_a_table_past_32_bits(gpu_lib):
    """As many entries as a table may have (8.6 GB), the last rows in use, and half a billion blocks."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    S, W, N = 16384, 131071, 1 << 29
    shape = mla.Shape(num_heads=8, kv_lora_rank=32, rope_dim=8, v_head_dim=8, block_size=2, num_blocks=N)
    pool = mla.Pool.allocate(shape, S, W)
    copies, n, left, status = (torch.zeros(v, dtype=torch.int32, device="cuda") for v in ((S, 4), (1,), (1,), (1,)))
    pool.ref_count[:N - 200000] = 1                          # all but the last are somebody else's
    new = torch.zeros(S, dtype=torch.int32, device="cuda")
    new[S - 1], new[0] = 2 * W - 1, 3
    mla.mla_pool_resize(pool, new, copies, n, num_free=left, status=status)
    free = torch.arange(N - 200000, N, dtype=torch.int32, device="cuda")
    assert int(status) == 0 and int(n) == 0 and int(left) == 200000 - 2 - W
    assert torch.equal(pool.block_table[0, :2], free[:2]) and int(pool.block_table[0, 2]) == -1
    assert torch.equal(pool.block_table[S - 1], free[2:2 + W])
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    mla.mla_pool_fork(pool, (S - 1) * one, (S - 2) * one, copies, n, num_free=left, status=status)
    assert int(status) == 0 and copies[0].tolist() == [int(free[1 + W]), int(free[2 + W]), 0, 1]
    assert torch.equal(pool.block_table[S - 2, :W - 1], free[2:1 + W]) and int(pool.block_table[S - 2, W - 1]) == int(free[2 + W])
    assert int(pool.ref_count[int(free[W])]) == 2 and int(pool.seq_lens[S - 2]) == 2 * W - 1
    pool.ref_count[:1000] = 0                                # room at the front, for some of them
    mla.mla_pool_compact(pool, copies, n, num_live=left, status=status)
    assert int(status) == 0 and int(n) == 1000 and int(left) == N - 200000 + W + 3 - 1000
    assert copies[:3, :2].tolist() == [[int(left) + i, i] for i in range(3)]
    moved = torch.arange(1000, dtype=torch.int32, device="cuda")
    assert torch.equal(pool.block_table[S - 1, W - 999:], moved[:999]) and int(pool.block_table[S - 2, W - 1]) == 999
    new.zero_()
    mla.mla_pool_resize(pool, new, copies, n, num_free=left, status=status)
    assert int(status) == 0 and int(left) == 200000 + 1000 and not pool.ref_count[:1000].any()
    assert int(pool.block_table[S - 2:].max()) == -1 and not pool.ref_count[N - 200000:].any()


def test_a_large_pool_captured(gpu_lib):
    """A cluster of 16 CTAs and much shared memory, asked for while a graph is captured."""
    import torch
    S = 2000
    p = Pair(S, 70, 60000, 4)
    new = p.ints([(b * 31) % 90 for b in range(S)])
    half = p.ints([(b * 31) % 90 // 2 for b in range(S)])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.mla.mla_pool_resize(p.pool, new, p.copies, p.n, status=p.status)
        p.mla.mla_pool_resize(p.pool, half, p.copies, p.n, num_free=p.left, status=p.status)
        p.mla.mla_pool_compact(p.pool, p.copies, p.n, status=p.status)
    k = upkeep.Books(S, 70, 60000, 4)
    for _ in range(2):
        g.replay()
        k.resize([(b * 31) % 90 for b in range(S)])
        left = k.resize([(b * 31) % 90 // 2 for b in range(S)])[2]
        k.compact(60000)
        assert int(p.status) == 0 and int(p.left) == left
        np.testing.assert_array_equal(p.pool.block_table.cpu().numpy(), k.table())
        np.testing.assert_array_equal(p.pool.ref_count.cpu().numpy(), k.ref)


def test_books_at_any_address(gpu_lib):
    """Arrays that begin four bytes behind a boundary."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    p = Pair(5, 3, 50, 4)
    base = torch.full((1 + 15 + 5 + 50,), -1, dtype=torch.int32, device="cuda")
    base[16:] = 0
    p.pool = mla.Pool(p.shape, base[1:16].view(5, 3), base[16:21], base[21:])
    assert p.resize([12, 5, 0, 0, 7]) == 0
    assert p.fork([0, 1], [2, 3]) == 0
    assert p.resize([0, 5, 9, 6, 7]) == 0
    assert p.compact() == 0


def test_captured_and_on_two_streams(gpu_lib):
    """A step's calls in a graph, replayed while another pool's run on another stream."""
    import torch
    p, o = Pair(30, 20, 400, 8), Pair(1500, 3, 4000, 4)
    want = upkeep.Books(30, 20, 400, 8)
    lens = [(b * 13) % 100 if b < 25 else 0 for b in range(30)]
    new, parents, children = p.ints(lens), p.ints([3, 4]), p.ints([27, 28])
    again = p.ints([n // 2 for n in lens])

    def step():
        m, a = p.mla, (p.copies, p.n)
        m.mla_pool_resize(p.pool, new, *a, status=p.status)
        m.mla_pool_fork(p.pool, parents, children, *a, status=p.status)
        m.mla_pool_resize(p.pool, again, *a, num_free=p.left, status=p.status)
        m.mla_pool_compact(p.pool, *a, status=p.status)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    p.mla.mla_pool_resize(p.pool, p.ints([0] * 30), p.copies, p.n)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    big = o.ints([b % 13 for b in range(1500)])
    want.resize(lens), want.fork([3, 4], [27, 28]), want.resize([n // 2 for n in lens]), want.compact(400)
    for _ in range(3):
        g.replay()
        p.mla.mla_pool_resize(o.pool, big, o.copies, o.n, num_free=o.left, status=o.status, stream=other)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(p.pool.block_table.cpu().numpy(), want.table())
        np.testing.assert_array_equal(p.pool.ref_count.cpu().numpy(), want.ref)
        assert int(p.status) == 0
        p.mla.mla_pool_resize(p.pool, p.ints([0] * 30), p.copies, p.n, status=p.status)
    want_o = upkeep.Books(1500, 3, 4000, 4)
    want_o.resize([b % 13 if b % 13 <= 12 else 0 for b in range(1500)])
    np.testing.assert_array_equal(o.pool.block_table.cpu().numpy(), want_o.table())


def test_the_binding_refuses(gpu_lib):
    import mla_latent_kv_08_gb300 as mla
    p = Pair(3, 4, 30, 8, room=3)
    ok = dict(new_lens=p.ints([1, 2, 3]), copies=p.copies, num_copies=p.n)
    for k, v in (("new_lens", p.ints([1, 2])), ("new_lens", p.ints([1, 2, 3]).long()), ("new_lens", p.ints([1, 2, 3]).cpu()),
                 ("copies", p.copies[:2]), ("copies", p.copies[:, :3]), ("copies", p.copies.view(-1)), ("num_copies", p.n[:0]),
                 ("num_copies", p.n.float())):
        with pytest.raises(mla.MlaError) as e:
            mla.mla_pool_resize(p.pool, **{**ok, k: v})
        assert e.value.code == mla.MLA_ERR_INVALID
    for kw in (dict(parents=p.ints([0, 1]), children=p.ints([2])), dict(parents=p.ints([0] * 4), children=p.ints([2] * 4)),
               dict(parents=p.ints([0]), children=p.ints([1]), lens=p.ints([1, 2])), dict(parents=p.ints([]), children=p.ints([]))):
        with pytest.raises(mla.MlaError):
            mla.mla_pool_fork(p.pool, copies=p.copies, num_copies=p.n, **kw)
    assert int(p.pool.ref_count.sum()) == 0


@pytest.mark.parametrize("S,W,N,bs", [(6, 600, 2500, 4), (40, 900, 30000, 2), (200, 1100, 90000, 3)])
def test_what_lies_behind_a_sequence_is_not_given_back(gpu_lib, S, W, N, bs):
    """Tables padded with valid block ids, as the attention calls take them: a sequence gives back
    what it held, and nothing of what its row has behind that."""
    for seed in range(4):
        rng = random.Random(seed)
        table, lens, ref = _books(rng, S, W, N, bs)
        for b in range(S):                                   # ends at and around whole pieces of the walk
            if lens[b] and rng.random() < 0.3:
                n = rng.choice([1, 255, 256, 257, 512, 513])
                while -(-lens[b] // bs) > n:
                    j = -(-lens[b] // bs) - 1
                    ref[table[b][j]] -= 1
                    table[b][j] = -1
                    lens[b] = j * bs
        p = Pair(S, W, N, bs)
        p.set(table, lens, ref)
        held = [-(-n // bs) for n in lens]
        pad = _padding(p, rng)
        mask = p.torch.arange(W, device="cuda") >= p.ints(held)[:, None]
        p.pool.block_table.copy_(p.torch.where(mask, pad, p.pool.block_table))
        new = [rng.choice([0, rng.randint(0, n), max(0, n - rng.randint(0, 2 * bs)), n // bs // 2 * bs, n, min(W * bs, n + rng.randint(0, bs))]) for n in lens]
        p.mla.mla_pool_resize(p.pool, p.ints(new), p.copies, p.n, num_free=p.left, status=p.status)
        flags, copies, left = p.k.resize(new)
        assert flags == 0 and int(p.status) == 0 and int(p.n) == len(copies) and int(p.left) == left
        np.testing.assert_array_equal(p.copies.cpu().numpy()[:len(copies)], np.array(copies, np.int32).reshape(-1, 4))
        np.testing.assert_array_equal(p.pool.ref_count.cpu().numpy(), p.k.ref)
        np.testing.assert_array_equal(p.pool.seq_lens.cpu().numpy(), p.k.lens)
        want, pads = np.array(p.k.table()), pad.cpu().numpy()
        for b, (h, n) in enumerate(zip(held, new)):
            end = max(h, -(-n // bs))
            want[b, end:] = pads[b, end:]
        np.testing.assert_array_equal(p.pool.block_table.cpu().numpy(), want)


def _padding(p, rng):
    """Entries behind the sequences' ends: 0, and any block there is."""
    S, W = p.pool.block_table.shape
    g = p.torch.Generator(device="cuda").manual_seed(rng.randrange(1 << 30))
    some = p.torch.randint(0, p.shape.num_blocks, (S, W), generator=g, device="cuda", dtype=p.torch.int32)
    return some * (p.torch.rand((S, W), generator=g, device="cuda") < 0.3).int()


@pytest.mark.parametrize("S,W,N,bs", [(3, 4, 30, 8), (60, 300, 9000, 4), (300, 500, 60000, 2)])
def test_compaction_changes_everything_or_nothing(gpu_lib, S, W, N, bs):
    """A table entry out of range, wherever it is: no block moves, and no copy is listed."""
    import torch
    rng = random.Random(S)
    books = _books(rng, S, W, N, bs, empty=0.0)
    p = Pair(S, W, N, bs)
    p.set(*books)
    full = [b for b in range(S) if books[1][b]]
    for bad in (-1, N, 2 ** 31 - 1, -2 ** 31):
        b = rng.choice(full)
        held = -(-books[1][b] // bs)
        for j in (0, held - 1, rng.randrange(held)):
            p.pool.block_table[b, j] = bad
            before = [t.clone() for t in (p.pool.block_table, p.pool.seq_lens, p.pool.ref_count)]
            p.mla.mla_pool_compact(p.pool, p.copies, p.n, num_live=p.left, status=p.status)
            assert int(p.status) == 1 and int(p.n) == 0 and int(p.left) == sum(c > 0 for c in books[2])
            assert p.mla.mla_read_status_word(p.status)[0] == p.mla.MLA_ERR_BOUNDS
            assert bool((p.copies == -5).all())
            for t, was in zip((p.pool.block_table, p.pool.seq_lens, p.pool.ref_count), before):
                assert torch.equal(t, was)
            p.status.zero_()
            p.pool.block_table[b, j] = books[0][b][j]
    end = -(-books[1][full[0]] // bs)
    if end < W:                                              # behind a sequence's end nothing is looked at
        p.pool.block_table[full[0], end] = N
        p.mla.mla_pool_compact(p.pool, p.copies, p.n, status=p.status)
        assert int(p.status) == 0 and int(p.pool.block_table[full[0], end]) == N
    p.copies.fill_(-5)
    p.set(*books)
    assert p.compact() == 0


def test_two_host_threads(gpu_lib):
    """Pools of many and of few sequences, each with a thread and a stream of its own: what one call
    needs of shared memory is not what another's launch finds."""
    import ctypes
    import threading
    import mla_latent_kv_08_gb300 as mla
    import torch
    pairs = [(Pair(16384, 2, 5000, 4), 3000), (Pair(3000, 2, 5000, 4), 3000)]
    failed, jobs = [], []
    for p, calls in pairs:
        S = p.pool.seq_lens.numel()
        S_new = [p.ints([b % 5 if b < 2500 else 0 for b in range(S)]), p.ints([b % 3 if b < 2500 else 0 for b in range(S)])]
        n = 3000 if S > 3000 else 2100
        forks = p.ints([0] * n)                              # refused, all of them: a child several times
        jobs.append((p, calls, S_new, forks, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(p, calls, new, forks, stream):
        shape, pool, s = p.pool._args[0], p.pool._args[1], ctypes.c_void_p(stream.cuda_stream)
        ptr = [ctypes.c_void_p(t.data_ptr()) for t in (*new, forks, p.copies, p.n, p.status)]
        for i in range(calls):
            codes = [gpu_lib.mla_pool_resize(shape, pool, ptr[i % 2], ptr[3], ptr[4], None, ptr[5], s),
                     gpu_lib.mla_pool_fork(shape, pool, forks.numel(), ptr[2], ptr[2], None, ptr[3], ptr[4], None, None, s),
                     gpu_lib.mla_pool_compact(shape, pool, 0, ptr[3], ptr[4], None, ptr[5], s)]
            failed.extend(c for c in codes if c != mla.MLA_OK)
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, (len(failed), set(failed))
    for p, calls, new, _, _ in jobs:
        assert int(p.status) == 0
        np.testing.assert_array_equal(p.pool.seq_lens.cpu().numpy(), new[1].cpu().numpy())
        assert int((p.pool.ref_count > 0).sum()) == int((new[1] > 0).sum()) == int((p.pool.block_table >= 0).sum())


# ------------------------------------------------------------------ copies

KINDS = ["BF16", "FP32", "MXFP8", "INT2_ROT", "INT2_ROT_QR", "INT2_JOINT"]


def _caches(kind, layers, N, bs, seed, **dims):
    import mla_latent_kv_08_gb300 as mla
    import torch
    shape = mla.Shape(num_heads=8, v_head_dim=16, block_size=bs, num_blocks=N, kind=getattr(mla, "MLA_KV_" + kind), **dims)
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(layers):
        c = mla.Cache.allocate(shape)
        for t in _planes(c):
            _bytes(t).random_(0, 256, generator=g)
        out.append(c)
    return out


def _planes(c):
    return [t for t in (c.latent, c.codes, c.scale_zero, c.rope) if t is not None]


def _bytes(t):
    import torch
    return t.view(torch.uint8) if t.dim() else t


def _copy_check(caches, entries, room=None, handle=None, count=None):
    """The copies made on the host, byte by byte."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    N, bs = caches[0].shape.num_blocks, caches[0].shape.block_size
    room = len(entries) if room is None else room
    lst = torch.full((max(room, len(entries)), 4), 10 ** 9, dtype=torch.int32, device="cuda")
    if entries:
        lst[:len(entries)] = torch.tensor(entries, dtype=torch.int32)
    count = len(entries) if count is None else count
    want, flags = [[_bytes(t).cpu().numpy().copy() for t in _planes(c)] for c in caches], 0
    for s, d, f, n in entries[:max(0, min(count, room))]:
        if not (0 <= s < N and 0 <= d < N and f >= 0 and n >= 0 and f + n <= bs):
            flags = 1
            continue
        for w in want:
            for a in w:
                a[d, f:f + n] = a[s, f:f + n]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_cache_copy(handle or mla.Caches(caches), lst[:room], torch.tensor([count], dtype=torch.int32, device="cuda"), status=status)
    torch.cuda.synchronize()
    for c, w in zip(caches, want):
        for t, a in zip(_planes(c), w):
            np.testing.assert_array_equal(_bytes(t).cpu().numpy(), a)
    assert int(status) == flags


def _entries(rng, N, bs, n):
    ids = list(range(N))
    rng.shuffle(ids)
    out = []
    for i in range(n):
        f = rng.randint(0, bs)
        out.append([ids[i % max(1, n // 2)], ids[N - 1 - i], f, rng.randint(0, bs - f)] if rng.random() < 0.5 else [ids[i], ids[N - 1 - i], 0, bs])
    return out


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", [1, 7, 64])
@pytest.mark.parametrize("dims", [dict(kv_lora_rank=512, rope_dim=64), dict(kv_lora_rank=32, rope_dim=32), dict(kv_lora_rank=96, rope_dim=64),
                                  dict(kv_lora_rank=1024, rope_dim=128)])
def test_copies_of_every_kind(gpu_lib, kind, bs, dims):
    rng = random.Random(bs)
    caches = _caches(kind, 2, 40, bs, 1, **dims)
    _copy_check(caches, _entries(rng, 40, bs, 18))


@pytest.mark.parametrize("kind,dims", [("INT2_ROT", dict(kv_lora_rank=8, rope_dim=8, group_size=4)), ("FP32", dict(kv_lora_rank=8, rope_dim=0)),
                                       ("BF16", dict(kv_lora_rank=8, rope_dim=8, index_dim=8)), ("BF16", dict(kv_lora_rank=512, rope_dim=64, index_dim=64)),
                                       ("INT2_ROT_QR", dict(kv_lora_rank=24, rope_dim=8, group_size=8)), ("INT2_ROT", dict(kv_lora_rank=40, rope_dim=24, group_size=8))])
def test_copies_of_narrow_rows(gpu_lib, kind, dims):
    rng = random.Random(3)
    for bs in (3, 16):
        _copy_check(_caches(kind, 1, 30, bs, 2, **dims), _entries(rng, 30, bs, 14))


@pytest.mark.parametrize("layers", [1, 3, 64, 65, 130])
def test_copies_in_many_layers(gpu_lib, layers):
    caches = _caches("MXFP8", layers, 12, 16, 4, kv_lora_rank=64, rope_dim=16)
    _copy_check(caches, _entries(random.Random(layers), 12, 16, 5))


def test_the_copy_list_and_its_count(gpu_lib):
    """None, fewer than there is room for, a count past the room and below zero; one cache alone."""
    caches = _caches("BF16", 1, 20, 8, 5, kv_lora_rank=64, rope_dim=16)
    e = _entries(random.Random(9), 20, 8, 9)
    _copy_check(caches, [], room=6)
    _copy_check(caches, e, room=30)
    _copy_check(caches, e, count=4)
    _copy_check(caches, e[:5], count=1000)
    _copy_check(caches, e, count=-3)
    _copy_check(caches, e, handle=caches[0])


def test_copies_out_of_range_are_skipped(gpu_lib):
    caches = _caches("MXFP8", 3, 20, 8, 6, kv_lora_rank=64, rope_dim=16)
    big = 2 ** 31 - 1
    bad = [[-1, 3, 0, 8], [20, 3, 0, 8], [3, 20, 0, 8], [3, -1, 0, 8], [3, 4, -1, 4], [3, 4, 0, 9], [3, 4, 5, 4], [3, 4, big, big], [3, 4, 1, -1],
           [big, big, 0, 1], [3, 4, -2 ** 31, 1]]
    _copy_check(caches, [[0, 10, 0, 8]] + bad + [[1, 11, 2, 6], [2, 12, 8, 0], [5, 5, 0, 8]])


def test_copies_past_32_bits(gpu_lib):
    """Blocks whose bytes begin behind 2^32."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    N = (1 << 32) // (64 * 1152) + 300
    shape = mla.Shape(num_heads=8, kv_lora_rank=512, rope_dim=64, v_head_dim=128, block_size=64, num_blocks=N)
    c = mla.Cache.allocate(shape)
    c.latent[N - 3:].normal_()
    c.latent[1].normal_()
    lst = torch.tensor([[N - 1, 5, 0, 64], [1, N - 200, 3, 60]], dtype=torch.int32, device="cuda")
    mla.mla_cache_copy(c, lst, torch.tensor([2], dtype=torch.int32, device="cuda"))
    assert torch.equal(c.latent[5], c.latent[N - 1])
    assert torch.equal(c.latent[N - 200, 3:63], c.latent[1, 3:63]) and not c.latent[N - 200, :3].any() and not c.latent[N - 200, 63:].any()
    assert not c.latent[N - 201].any() and not c.latent[4].any() and not c.latent[6].any()


def test_lists_of_long_blocks(gpu_lib):
    """As many entries as a resize or a fork may list, in blocks of 2^28 rows: 2^32 tasks, of which the
    first, the last, and some in between do anything."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    bs, n = 1 << 28, 16384
    shape = mla.Shape(num_heads=8, kv_lora_rank=8, rope_dim=0, v_head_dim=16, block_size=bs, num_blocks=4)
    c = mla.Cache.allocate(shape)
    g = torch.Generator(device="cuda").manual_seed(1)
    c.latent[0].random_(-100, 100, generator=g)
    lst = torch.zeros((n, 4), dtype=torch.int32, device="cuda")
    entries = {0: [0, 1, 0, 5000], 8191: [0, 2, bs - 3000, 3000], 8192: [0, 2, 1025, 1023], n - 1: [0, 3, bs - 1500, 1500]}
    for i, e in entries.items():
        lst[i] = torch.tensor(e, dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_cache_copy(c, lst, torch.tensor([n], dtype=torch.int32, device="cuda"), status=status)
    assert int(status) == 0
    for _, d, f, k in entries.values():
        assert torch.equal(c.latent[d, f:f + k], c.latent[0, f:f + k])
    assert not c.latent[1, 5000:].any() and not c.latent[3, :bs - 1500].any()
    assert not c.latent[2, :1025].any() and not c.latent[2, 2048:bs - 3000].any()
