"""The 8-bit cache's entry points called the ways a server calls them: without a workspace,
from two captured graphs that share one, from two streams at once, over blocks that several
sequences share, with a block table and row buffers that are longer than what is used."""
import numpy as np
import pytest

from tests import gpu_util as gu
from tests.test_gpu_mx import _check, _roomy, _shape, _stored, _workload
from tests.test_gpu_prefill import Case

pytestmark = pytest.mark.gpu


def _decode_args(mla, w, shape):
    import torch
    bf = torch.bfloat16
    return dict(block_table=gu.dev(w.block_table), seq_lens=gu.dev(w.seq_lens.astype(np.int32)), q=gu.dev(w.q, bf),
                W_UV=gu.dev(w.W_UV, bf), scale=w.scale, out=torch.empty((w.B, 1, w.H, w.d_v), dtype=bf, device="cuda"),
                lse=torch.empty((w.B, 1, w.H), device="cuda"), workspace=mla.alloc_workspace(shape, w.B, 1))


@pytest.mark.parametrize("H,room", [(16, True), (16, False), (64, True), (128, False)])
def test_without_a_workspace(gpu_lib, H, room):
    import mla_latent_kv_08_gb300 as mla
    import torch
    w = _workload(70, [700, 1, 65], H=H)
    if room:
        _roomy(w)
    shape = _shape(mla, w)
    cache, _ = gu.fill_cache(w, shape)
    a = _decode_args(mla, w, shape)
    del a["workspace"]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_decode_noalloc(cache, status=st, **a)
    torch.cuda.synchronize()
    assert mla.mla_read_status_word(st)[0] == mla.MLA_OK
    _check(w, a["out"].float().cpu().numpy(), a["lse"].cpu().numpy(), _stored(w))


def _capture(f):
    import torch
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        f()
    return g


def test_two_graphs_share_a_workspace(gpu_lib):
    """One workspace, large enough for both, under a decode and a prefill replayed in turn."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    w = _workload(71, [900, 70], H=128)
    shape = _shape(mla, w)
    cache, _ = gu.fill_cache(w, shape)
    a = _decode_args(mla, w, shape)
    case = Case(72, [140, 60], [200, 0], H=4, kind="mxfp8")
    pshape = case.shape(mla)
    pcache, b = case.cache(mla, pshape), case.args(mla, pshape)
    both = max(a["workspace"].numel(), b["workspace"].numel())
    a["workspace"] = b["workspace"] = torch.empty(both, dtype=torch.uint8, device="cuda")
    g1, g2 = _capture(lambda: mla.mla_decode(cache, **a)), _capture(lambda: mla.mla_prefill(pcache, **b))
    b["workspace"].fill_(0xFF)
    for _ in range(3):
        for t in (a["out"], a["lse"], b["out"], b["lse"]):
            t.fill_(float("nan"))
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        _check(w, a["out"].float().cpu().numpy(), a["lse"].cpu().numpy(), _stored(w))
        case.check(b["out"].double().cpu().numpy(), b["lse"].cpu().numpy())


def test_two_streams_at_once(gpu_lib):
    """Calls of every kind on two streams, each with buffers of its own: as one after the other."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    jobs = []
    for seed, H in ((73, 16), (74, 128)):
        w = _workload(seed, [1500, 300, 64], H=H)
        if H == 16:
            _roomy(w)
        shape = _shape(mla, w)
        cache, _ = gu.fill_cache(w, shape)
        a = _decode_args(mla, w, shape)
        case = Case(seed, [300, 40], [500, 100], H=8, kind="mxfp8")
        pshape = case.shape(mla)
        pcache, b = case.cache(mla, pshape), case.args(mla, pshape)
        start, cu = gu.dev(np.array([3, 0, 1], np.int32)), gu.dev(np.array([0, 1400, 1400, 1460], np.int32))
        rows = torch.zeros((1460, 576), dtype=torch.bfloat16, device="cuda")

        def run(cache=cache, a=a, pcache=pcache, b=b, start=start, cu=cu, rows=rows):
            mla.mla_decode(cache, **a)
            mla.mla_prefill(pcache, **b)
            mla.mla_latent_read(cache, a["block_table"], start, cu, rows)
        jobs.append((run, (a["out"], a["lse"], b["out"], b["lse"], rows)))
    want = []
    for run, outs in jobs:
        run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    streams = [torch.cuda.Stream() for _ in jobs]
    for _, outs in jobs:
        for t in outs:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (run, _) in zip(streams, jobs):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for (_, outs), ref in zip(jobs, want):
        for t, r in zip(outs, ref):
            assert torch.equal(t, r)


@pytest.mark.parametrize("H", [16, 128])
def test_blocks_that_sequences_share(gpu_lib, H):
    """A prefix in the same blocks for every sequence, each with a tail of its own."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    w = _workload(75, [300, 200, 129], H=H)
    for b in (1, 2):                                                    # two blocks of the first sequence's
        w.block_table[b, :2] = w.block_table[0, :2]
        w.latent[b][:128], w.rope[b][:128] = w.latent[0][:128], w.rope[0][:128]
    shape = _shape(mla, w)
    cache = mla.Cache.allocate(shape)
    first = [0, 128, 128]
    gu.append_tokens(cache, w, [c[s:] for c, s in zip(w.latent, first)], [c[s:] for c, s in zip(w.rope, first)],
                     np.array(first, np.int32))
    out, lse, ws = gu.attend(w, shape, cache, w.q)
    assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
    lat = _stored(w)
    _check(w, out, lse, lat)
    cu = np.concatenate([[0], np.cumsum(w.seq_lens)]).astype(np.int32)
    rows = torch.zeros((int(cu[-1]), 576), dtype=torch.bfloat16, device="cuda")
    mla.mla_latent_read(cache, gu.dev(w.block_table), gu.dev(np.zeros(3, np.int32)), gu.dev(cu), rows)
    got = rows.double().cpu().numpy()
    for b in range(3):
        np.testing.assert_array_equal(got[cu[b]:cu[b + 1], :512], lat[b])
        np.testing.assert_array_equal(got[cu[b]:cu[b + 1], 512:], w.rope[b])


def test_bounds_above_what_is_used(gpu_lib):
    """num_q and max_tokens well above the sums, a table with unused columns, sequences without
    new tokens at both ends: the used rows as they should be, the others as they were."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    case = Case(76, [0, 30, 257, 0], [50, 0, 100, 7], H=3, kind="mxfp8")
    shape = case.shape(mla)
    cache = case.cache(mla, shape, poison=True)
    a = case.args(mla, shape)
    n = int(case.cu[-1])
    pad = 700

    def longer(t, fill):
        x = torch.full((n + pad, *t.shape[1:]), fill, dtype=t.dtype, device="cuda")
        x[:n] = t
        return x
    a["q"], a["out"], a["lse"] = longer(a["q"], float("nan")), longer(a["out"], 7.0), longer(a["lse"], 7.0)
    a["block_table"] = torch.cat([a["block_table"], torch.full((4, 33), -1, dtype=torch.int32, device="cuda")], 1)
    a["max_tokens"] = 5000
    a["workspace"] = mla.alloc_prefill_workspace(shape, 4, n + pad, 5000, 128)
    mla.mla_prefill(cache, **a)
    torch.cuda.synchronize()
    assert mla.mla_get_status(a["workspace"]) == (mla.MLA_OK, 0)
    out, lse = a["out"].double().cpu().numpy(), a["lse"].cpu().numpy()
    assert (out[n:] == 7.0).all() and (lse[n:] == 7.0).all()
    case.check(out[:n], lse[:n])


def test_blocks_past_32_bits(gpu_lib):
    """A pool whose codes are more than 2^32 bytes, its last blocks in use: as in a small pool."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    big = 140000
    for H, room in ((16, True), (128, False)):
        w = _workload(77, [300, 65], H=H)
        if room:
            _roomy(w)
        got = []
        for blocks in (w.num_blocks, big):
            shape = _shape(mla, w, num_blocks=blocks)
            cache = mla.Cache.allocate(shape, zero=False)
            table = w.block_table
            w.block_table = np.where(table >= 0, table + blocks - w.num_blocks, -1).astype(np.int32)
            gu.append_tokens(cache, w, w.latent, w.rope, np.zeros(2, np.int32))
            out, lse, ws = gu.attend(w, shape, cache, w.q)
            assert mla.mla_get_status(ws) == (mla.MLA_OK, 0)
            rows = torch.zeros((365, 576), dtype=torch.bfloat16, device="cuda")
            bt = gu.dev(w.block_table)
            cu = gu.dev(np.array([0, 300, 365], np.int32))
            mla.mla_latent_read(cache, bt, gu.dev(np.zeros(2, np.int32)), cu, rows)
            case = Case(78, [40, 65], [260, 0], H=2, kind="mxfp8")
            pshape = case.shape(mla)
            pshape.num_blocks = blocks
            a = case.args(mla, pshape)
            a["block_table"] = bt
            mla.mla_prefill(cache, shape=pshape, **a)
            torch.cuda.synchronize()
            got.append((out, lse, rows.float().cpu().numpy(), a["out"].float().cpu().numpy()))
            w.block_table = table
            del cache
        for small, large in zip(*got):
            np.testing.assert_array_equal(small, large)
        _check(w, got[1][0], got[1][1], _stored(w))
