"""Calls of several host threads at once, each on a stream, caches and workspaces of its own: kernels
that both use, with different needs of shared memory."""
import threading

import pytest

pytestmark = pytest.mark.gpu

H, dv, bs, n = 2, 64, 16, 20


def _calls(r, dR, gs, dn, kind, g):
    """(a function of a stream, its outputs) for the calls of one kind on the CUDA cores."""
    import mla_latent_kv_08_gb300 as mla
    import torch
    fp32, int2 = kind == "FP32", kind.startswith("INT2")
    shape = mla.Shape(num_heads=H, kv_lora_rank=r, rope_dim=dR, v_head_dim=dv, block_size=bs, num_blocks=2, group_size=gs,
                      kind=getattr(mla, "MLA_KV_" + kind), impl=mla.MLA_IMPL_SIMT)
    dt = torch.float32 if fp32 else torch.bfloat16

    def normal(*s, dtype=dt):
        return torch.randn(s, generator=g, device="cuda").to(dtype)

    def ints(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    cache = mla.Cache.allocate(shape)
    table, zero, cu, lens = ints(0, 1).view(1, 2), ints(0), ints(0, n), ints(n)
    c, k, q, W = normal(n, r), normal(n, dR), normal(1, 1, H, r + dR), normal(H, r, dv)
    R = torch.linalg.qr(torch.randn((r, r), generator=g, device="cuda"))[0].contiguous() if int2 else None
    clip = torch.full((r // gs,), 2.0, device="cuda") if int2 else None
    out, lse = torch.empty((1, 1, H, dv), dtype=dt, device="cuda"), torch.empty((1, 1, H), device="cuda")
    ws = mla.alloc_workspace(shape, 1)
    if not int2:
        qn, uk = normal(n, H, dn + dR), normal(H, dn, r)
        rows = torch.empty((n, H, dv), dtype=dt, device="cuda")
        pre = mla.alloc_prefill_workspace(shape, 1, n, n, dn)

    def call(stream):
        mla.mla_latent_append(cache, table, zero, cu, c, k, R=R, clip=clip, stream=stream)
        mla.mla_decode(cache, table, lens, q, W, 0.05, out, lse, ws, R=R, stream=stream)
        if not int2:
            mla.mla_prefill(cache, table, lens, cu, qn, uk, W, 0.05, rows, pre, n, stream=stream)
    return call, [out, lse] + ([] if int2 else [rows])


@pytest.mark.parametrize("kind", ["BF16", "FP32", "MXFP8", "INT2_ROT"])
def test_two_sizes_of_a_model_at_once(gpu_lib, kind):
    import mla_latent_kv_08_gb300 as mla
    import torch
    g = torch.Generator(device="cuda").manual_seed(7)
    jobs = []
    for r, dR, gs, dn in ((1024, 64, 32, 512), (800, 32, 32, 64)):
        call, outs = _calls(r, dR, gs, dn, kind, g)
        call(None)
        torch.cuda.synchronize()
        jobs.append((call, outs, [t.clone() for t in outs], torch.cuda.Stream()))
    failed = []

    def work(call, stream):
        for _ in range(1500):
            try:
                call(stream)
            except mla.MlaError as e:
                failed.append(str(e))
    threads = [threading.Thread(target=work, args=(j[0], j[3])) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, (len(failed), failed[0])
    for _, outs, want, _ in jobs:
        for t, w in zip(outs, want):
            assert torch.equal(t, w)
