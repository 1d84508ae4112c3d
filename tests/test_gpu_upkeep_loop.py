"""A serving loop's step with the calls as they are used together: lengths, appends, verify,
acceptance, forks, compaction and copies, against sequences that share nothing."""
import numpy as np
import pytest

from oracle import upkeep
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

H, r, dR, dv, bs = 16, 512, 64, 128, 64


class Loop:
    """Sequences in a pool of blocks in several layers, and beside each its tokens' rows."""

    def __init__(self, mla, kind, S, W, N, layers=2):
        import torch
        self.mla, self.torch = mla, torch
        self.shape = mla.Shape(num_heads=H, kv_lora_rank=r, rope_dim=dR, v_head_dim=dv, block_size=bs, num_blocks=N, kind=kind)
        self.pool = mla.Pool.allocate(self.shape, S, W)
        self.layers = [mla.Cache.allocate(self.shape) for _ in range(layers)]
        self.caches = mla.Caches(self.layers)
        self.copies = torch.zeros((max(S, N), 4), dtype=torch.int32, device="cuda")
        self.n, self.status = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
        self.rows = [[torch.empty((0, r + dR), dtype=torch.bfloat16, device="cuda") for _ in range(S)] for _ in range(layers)]
        self.g = torch.Generator(device="cuda").manual_seed(1)
        self.W_UV = self.normal(H, r, dv) * r ** -0.5

    def normal(self, *shape):
        return self.torch.randn(shape, generator=self.g, device="cuda").to(self.torch.bfloat16)

    def ints(self, v):
        return self.torch.tensor(v, dtype=self.torch.int32, device="cuda")

    def lens(self):
        return self.pool.seq_lens.cpu().tolist()

    def resize(self, new):
        self.mla.mla_pool_resize(self.pool, new if hasattr(new, "device") else self.ints(new), self.copies, self.n, status=self.status)
        self.mla.mla_cache_copy(self.caches, self.copies, self.n, status=self.status)
        for rows in self.rows:
            for b, n in enumerate(self.lens()):
                rows[b] = rows[b][:n]

    def fork(self, parents, children, lens):
        self.mla.mla_pool_fork(self.pool, self.ints(parents), self.ints(children), self.copies, self.n, lens=self.ints(lens), status=self.status)
        self.mla.mla_cache_copy(self.caches, self.copies, self.n, status=self.status)
        for rows in self.rows:
            for a, c, n in zip(parents, children, lens):
                rows[c] = rows[a][:n]

    def compact(self):
        self.mla.mla_pool_compact(self.pool, self.copies, self.n, status=self.status)
        self.mla.mla_cache_copy(self.caches, self.copies, self.n, status=self.status)

    def append(self, counts):
        """New tokens for every sequence, in every layer; the room is there already."""
        start = self.ints([n - k for n, k in zip(self.lens(), counts)])
        cu = self.ints(np.concatenate([[0], np.cumsum(counts)]))
        for cache, rows in zip(self.layers, self.rows):
            x = self.normal(sum(counts), r + dR)
            self.mla.mla_latent_append(cache, self.pool.block_table, start, cu, x[:, :r].contiguous(), x[:, r:].contiguous(), status=self.status)
            at = 0
            for b, k in enumerate(counts):
                rows[b] = self.torch.cat([rows[b], x[at:at + k]])
                at += k

    def grow(self, counts):
        self.resize([n + k for n, k in zip(self.lens(), counts)])
        self.append(counts)

    def check(self):
        """Every layer's rows as they are read back, and its attention, are those of caches of its own
        for each sequence, in order."""
        torch, mla = self.torch, self.mla
        lens = self.lens()
        used = [b for b, n in enumerate(lens) if n]
        some = self.ints([lens[b] for b in used])
        blocks = [-(-lens[b] // bs) for b in used]
        own = mla.Shape(**{**self.shape.__dict__, "num_blocks": sum(blocks)})
        table = torch.full((len(used), max(blocks)), -1, dtype=torch.int32, device="cuda")
        first = 0
        for i, k in enumerate(blocks):
            table[i, :k] = torch.arange(first, first + k)
            first += k
        cu = self.ints(np.concatenate([[0], np.cumsum([lens[b] for b in used])]))
        q = self.normal(len(used), 1, H, r + dR)
        mine = self.pool.block_table[used].contiguous()
        for cache, rows in zip(self.layers, self.rows):
            flat = torch.cat([rows[b] for b in used])
            apart = mla.Cache.allocate(own)
            mla.mla_latent_append(apart, table, torch.zeros_like(some), cu, flat[:, :r].contiguous(), flat[:, r:].contiguous(), status=self.status)
            got = []
            for c, t, s in ((cache, mine, self.shape), (apart, table, own)):
                back = torch.empty((int(cu[-1]), r + dR), dtype=torch.bfloat16, device="cuda")
                mla.mla_latent_read(c, t, torch.zeros_like(some), cu, back, status=self.status)
                out = torch.empty((len(used), 1, H, dv), dtype=torch.bfloat16, device="cuda")
                lse = torch.empty((len(used), 1, H), device="cuda")
                ws = mla.alloc_workspace(s, len(used))
                mla.mla_decode(c, t, some, q, self.W_UV, 0.05, out, lse, ws)
                assert mla.mla_get_status(ws)[0] == mla.MLA_OK
                got.append((back, out, lse))
            for a, b in zip(*got):                           # the same kernels on the same values
                assert torch.equal(a, b)
            if self.shape.kind == mla.MLA_KV_BF16:
                assert torch.equal(got[0][0], flat)
        assert int(self.status) == 0


@pytest.mark.parametrize("kind", ["BF16", "MXFP8"])
def test_forks_cuts_and_compaction(gpu_lib, kind):
    import mla_latent_kv_08_gb300 as mla
    k = Loop(mla, getattr(mla, "MLA_KV_" + kind), 8, 12, 60)
    k.grow([300, 65, 64, 1, 0, 0, 0, 0])
    k.fork([0, 0, 2, 1], [4, 5, 6, 7], [300, 256, 64, 30])
    k.check()
    k.grow([5, 0, 3, 70, 9, 130, 2, 40])                     # everyone writes on behind what is shared
    k.check()
    k.resize([130, 65, 10, 71, 309, 200, 64, 0])             # cuts inside shared blocks, and an end
    k.check()
    k.grow([7, 1, 60, 0, 1, 57, 3, 90])
    k.check()
    k.resize([0, 66, 70, 0, 310, 100, 67, 90])
    k.compact()
    k.check()
    k.grow([64, 1, 1, 200, 1, 1, 1, 1])
    k.check()


def test_speculative_steps(gpu_lib):
    """Drafts are appended, verified, partly accepted, and the sequences cut back to what stands;
    nothing of it passes through the host but what the test compares."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    S, K, V = 5, 7, 1000
    k = Loop(mla, mla.MLA_KV_BF16, S, 10, 40)
    k.grow([200, 63, 64, 128, 1])
    new = torch.empty(S, dtype=torch.int32, device="cuda")
    accepted, tokens = torch.empty(S, dtype=torch.int32, device="cuda"), torch.empty((S, K + 1), dtype=torch.int32, device="cuda")
    ws = mla.alloc_workspace(k.shape, S, K + 1)
    out, lse = torch.empty((S, K + 1, H, dv), dtype=torch.bfloat16, device="cuda"), torch.empty((S, K + 1, H), device="cuda")
    for step in range(4):
        k.grow([K + 1] * S)
        mla.mla_verify(k.layers[0], k.pool.block_table, k.pool.seq_lens, k.normal(S, K + 1, H, r + dR), k.W_UV, 0.05, out, lse, ws)
        logits = out.float().mean(2) @ k.normal(dv, V).float() * 20
        p = torch.softmax(logits, -1)
        q = torch.softmax(logits[:, :K] + torch.randn((S, K, V), generator=k.g, device="cuda"), -1)
        x = torch.multinomial(q.view(S * K, V), 1, generator=k.g).view(S, K).int()
        u = torch.rand((S, K + 1), generator=k.g, device="cuda")
        before = k.lens()
        mla.mla_draft_accept(p, x, u, accepted, tokens, draft_probs=q, seq_lens=k.pool.seq_lens, new_lens=new, status=k.status)
        k.resize(new)
        want = upkeep.accept(*[t.double().cpu().numpy().tolist() for t in (p, q)], x.cpu().tolist(), u.double().cpu().numpy().tolist(), lens=before)
        assert tokens.cpu().tolist() == [w[2] for w in want] and k.lens() == [w[3] for w in want]
        k.check()
