"""Calls of kvq_verify_attention that its documentation allows, at the ends of its ranges."""
import pytest
import torch

import fp8_int8_quantized_gb300 as kvq
from tests.test_gpu_verify import Batch
from tests.test_gpu_verify_range import check

pytestmark = pytest.mark.gpu

FORMATS = [("e4m3", 0), ("e5m2", 0), ("int8", 0), ("int4", 0), ("int8", 4), ("int4", 4)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kvq.build()
    torch.cuda.init()


def batch(ctx, n, hkv, g, d, bs, fmt, parts, **kw):
    return Batch(ctx, n, hkv, g, d, bs, fmt, d // parts if parts else 0, outliers=False, **kw)


@pytest.mark.parametrize("fmt,parts", FORMATS)
@pytest.mark.parametrize("g,n", [(4, 3), (8, 4), (8, 8)])
def test_the_largest_batch_of_the_tcgen05_kernels(fmt, parts, g, n):
    """1024 sequences: the scan and the lengths fill the last of their shared memory."""
    ctx = [n + i * 53 % 190 for i in range(1024)]
    b = batch(ctx, [n if i % 5 else 0 for i in range(1024)], 2, g, 128, 16, fmt, parts, tree=True, seed=51)
    out = b.run()
    check(b, out, [1, 2, 511, 768, 1022, 1023])
    assert torch.equal(out, b.run())


@pytest.mark.parametrize("fmt,parts", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
def test_bounds_far_above_the_lengths(fmt, parts, d):
    """max_query_len and max_context_len as a server sets them once: 64 and 2^24 for chunks of 1 to 5 and contexts
    of 5 to 700 (block tables as wide as they are)."""
    b = batch([5, 700, 131, 64], [5, 1, 4, 2], 3, 5, d, 32, fmt, parts, tree=True, seed=52)
    out = kvq.verify_attention(b.q, b.cache, b.bt, b.cl, b.qs, 64, 1 << 24, tree_mask=b.mask, scale=b.scale)
    check(b, out, range(4))


@pytest.mark.parametrize("fmt,parts", [("e4m3", 0), ("int8", 0), ("int4", 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_captured_call_replayed_while_contexts_grow(fmt, parts, d):
    b = batch([4000, 1500, 900], [4, 4, 4], 2, 8, d, 16, fmt, parts, tree=False, seed=53)
    out = torch.empty_like(b.q)
    ws = torch.empty(kvq.verify_workspace_size(3, 16, 2, d, 4, 4096, fmt), dtype=torch.uint8, device="cuda")
    call = lambda o, w: kvq.verify_attention(b.q, b.cache, b.bt, b.cl, b.qs, 4, 4096, scale=b.scale, out=o, workspace=w)  # noqa: E731
    call(out, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws)
    full = list(b.ctx)
    for lens in ([4, 4, 4], [5, 130, 16], [129, 1500, 17], [2047, 33, 900], full):
        b.cl.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7.0)
        ws.fill_(255)     # nothing of an earlier call is needed
        graph.replay()
        want = call(torch.empty_like(b.q), torch.empty_like(ws))
        assert torch.equal(out, want)
        slots, b.ctx = b.slots, lens
        b.slots = torch.cat([slots[sum(full[:i]):sum(full[:i]) + x] for i, x in enumerate(lens)])
        check(b, out, range(3))
        b.slots, b.ctx = slots, full


@pytest.mark.parametrize("fmt,parts,d", [("e4m3", 0, 128), ("int8", 0, 128), ("int4", 4, 128), ("e5m2", 0, 64), ("int8", 4, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_query_spoils_its_own_row(fmt, parts, d, bad):
    b = batch([900] * 20, [3] * 20, 2, 8, d, 16, fmt, parts, tree=True, seed=54)
    clean = b.run()
    b.q[7, 5, 11] = bad
    out = b.run()
    rest = torch.ones(60, 16, dtype=torch.bool)
    rest[7, 5] = False
    assert torch.equal(out[rest], clean[rest]) and torch.isnan(out[7, 5]).all()
    assert kvq.device_error_check() == (0, 0)


def test_contexts_longer_than_their_table_are_refused():
    b = batch([100, 50], [3, 4], 1, 2, 128, 16, "e4m3", 0, tree=True, seed=55)
    good = b.run()
    long = b.cl.clone()
    long[1] = b.bt.shape[1] * 16 + 1
    out = torch.full_like(b.q, 7.0)
    kvq.verify_attention(b.q, b.cache, b.bt, long, b.qs, 4, 1000, tree_mask=b.mask, scale=b.scale, out=out)
    assert kvq.device_error_check() == (4, 1) and (out[3:] == 7).all()
    assert ((out[:3].float() - good[:3].float()).abs() <= 2 ** -9 * good[:3].float().abs() + 2e-5).all()


def test_a_scale_for_e5m2_and_none_for_e4m3():
    for fmt, value in (("e5m2", 0.125), ("e4m3", None)):
        b = batch([600, 33], [4, 2], 2, 4, 128, 16, fmt, 0, tree=True, seed=56)
        b.scale_value, b.scale = value, torch.tensor([value], device="cuda") if value else None
        kvq.append(b.k, b.v, b.cache, b.slots, b.scale)
        check(b, b.run(), range(2))


def test_two_streams_at_once():
    """Calls with workspaces of their own that may overlap, next to an append into other blocks of the same cache."""
    a = batch([3000] * 6, [4] * 6, 4, 8, 128, 16, "int8", 0, tree=True, seed=57)
    b = batch([2500] * 5, [7] * 5, 4, 8, 128, 16, "int4", 4, tree=True, seed=58)
    wa, wb = a.run(), b.run()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs.append((a.run(stream=sa), b.run(stream=sb)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, wa) and torch.equal(y, wb) for x, y in outs)


@pytest.mark.parametrize("fmt,parts", FORMATS)
def test_sequences_that_share_blocks(fmt, parts):
    """A common prefix held once: the tables of all sequences begin with the same blocks."""
    b = batch([640] * 4, [4] * 4, 2, 8, 128, 16, fmt, parts, tree=True, seed=59)
    b.bt[1:, :30] = b.bt[0, :30]
    per = torch.arange(480, device="cuda")
    shared = b.bt[0, :30].long()[per // 16] * 16 + per % 16
    s = b.slots.view(4, 640)
    s[1:, :480] = shared
    b.slots = s.reshape(-1)
    check(b, b.run(), range(4))


@pytest.mark.parametrize("fmt,group,d", [("e4m3", 0, 128), ("int8", 32, 128), ("int4", 0, 128), ("e5m2", 0, 64)])
def test_caches_beyond_four_gigabytes(fmt, group, d):
    """append_rotary, verify_attention and move_rows in the last blocks of a cache whose rows (and scales) lie past
    2^32 bytes: what the same calls give in a small one."""
    hkv, bs, T = 8, 16, 300
    row = d // 2 if fmt == "int4" else d
    many = (1 << 32) // (hkv * bs * row) + 64
    gen = torch.Generator(device="cuda").manual_seed(60)
    x = torch.randn(T, 16 + 2 * hkv, d, generator=gen, device="cuda").half()
    q, k, v = x.split([16, hkv, hkv], 1)
    ang = torch.rand(512, d // 2, generator=gen, device="cuda") * 6
    table = torch.cat([ang.cos(), ang.sin()], 1).contiguous()
    pos = torch.arange(T, device="cuda")
    scale = torch.tensor([0.02], device="cuda") if fmt[0] == "e" else None
    ids = torch.randperm(20, generator=torch.Generator().manual_seed(1)).cuda()[:19]
    results = []
    for blocks in (20, many):
        c = kvq.KVCache(blocks, hkv, bs, d, fmt, "cuda", group_size=group)
        at = ids + blocks - 20
        slots = (at[:, None] * bs + torch.arange(bs, device="cuda")).flatten()[:T]
        rq = kvq.append_rotary(q, k, v, c, slots, pos, table, scale=scale)
        args = (rq[-5:].contiguous(), c, at.int()[None], torch.tensor([T], dtype=torch.int32, device="cuda"),
                torch.tensor([0, 5], dtype=torch.int32, device="cuda"), 5, T)
        o = kvq.verify_attention(*args, scale=scale)
        kvq.move_rows(c, slots[[299, 296, 297]].contiguous(), slots[[296, 297, 298]].contiguous(),
                      torch.tensor([0, 3], dtype=torch.int32, device="cuda"), 3)
        results.append((rq, o, kvq.verify_attention(*args, scale=scale), *kvq.dequant(c, slots.contiguous(), scale=scale)))
        assert kvq.device_error_check() == (0, 0)
        del c, args
    assert all(torch.equal(a, b) for a, b in zip(*results)) and not torch.equal(results[0][1], results[0][2])
