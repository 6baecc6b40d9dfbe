"""kvq_verify_attention over the range of V: small rows, rows of very different size, and a token that takes most of
the softmax.  The results are held to bounds that shrink with V (tests/verify_bound.py)."""
import pytest
import torch

import fp8_int8_quantized_gb300 as kvq
from tests import spec_ref as R
from tests import verify_bound as VB
from tests.test_gpu_verify import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kvq.build()
    torch.cuda.init()


def fill(b, kind):
    """Rewrites the batch's K, V and queries."""
    gen = torch.Generator(device="cuda").manual_seed(77)
    if kind == "sink":   # the first tokens' logits lie 12 above the others', their V is 2^-8 as large
        c = 12.0 * b.d ** 0.5 / 8.0
        b.q[..., 0] = 8.0
        b.k[..., 0] = 0.0
        first = [sum(b.ctx[:i]) for i in range(len(b.ctx))]
        b.k[first, :, 0] = c
        b.v[first] *= 2.0 ** -8
    elif kind == "mixed":   # every row its own size
        e = torch.randint(0, 21, (b.v.shape[0], b.v.shape[1], 1), generator=gen, device="cuda")
        b.v.copy_((b.v.float() * torch.exp2(-e.float())).half())
    else:
        b.v.copy_((b.v.float() * kind).half())
    kvq.append(b.k, b.v, b.cache, b.slots, b.scale)


def check(b, out, seqs):
    in_v = b.group and b.group < b.d and b.d == 128 and len(b.ctx) <= 1024   # tcgen05: V carries its group scales
    for i in seqs:
        if not b.n[i]:
            continue
        k, v = b.kv(i)
        at = sum(b.ctx[:i])
        s = b.slots[at:at + b.ctx[i]]
        if b.cache.v_scales is None:
            unit, codes = torch.ones_like(v[..., 0]), v.abs()
        else:
            sc = b.cache.v_scales[s // b.bs, :, s % b.bs].double().reshape(*v.shape[:2], -1)
            full = sc.repeat_interleave(b.d // sc.shape[-1], -1)
            if in_v:
                unit, codes = torch.ones_like(v[..., 0]), v.abs()
            else:
                unit, codes = sc.amax(-1), torch.where(full > 0, v.abs() / full, 0.0)
        q = b.q[b.start[i]:b.start[i + 1]].double()
        o, bound = VB.attention(q, k, v, unit, codes, b.masks[i], b.d ** -0.5, b.ctx[i] - b.n[i], in_v)
        got = out[b.start[i]:b.start[i + 1]].double()
        assert torch.isfinite(got).all()
        far = ((got - o).abs() / bound).max().item()
        assert far <= 1.0, (i, b.ctx[i], far)
        e = VB.rms(got - o)
        assert e <= VB.rms_bound(o, b.ctx[i]), (i, b.ctx[i], e / VB.rms(o))
    assert kvq.device_error_check() == (0, 0)


@pytest.mark.parametrize("kind", [1.0, "sink"])
@pytest.mark.parametrize("fmt,group,d", [("e4m3", 0, 128), ("e5m2", 0, 128), ("e4m3", 0, 64), ("e5m2", 0, 64), ("int8", 32, 128),
                                         ("int8", 64, 128), ("int4", 32, 128), ("int4", 64, 128)])
@pytest.mark.parametrize("hkv,g,n", [(2, 2, 3), (1, 8, 4), (1, 8, 7)])
def test_one_token_takes_most_of_the_softmax(fmt, group, d, hkv, g, n, kind):
    ctx = [8000, 700, 90, n]
    b = Batch(ctx, [n] * 4, hkv, g, d, 16, fmt, group, tree=True, seed=31, outliers=False)
    fill(b, kind)
    check(b, b.run(), range(4))


@pytest.mark.parametrize("kind", [1.0, 2.0 ** -7, 2.0 ** -10, 2.0 ** -14, 2.0 ** -20, "mixed", "sink"])
@pytest.mark.parametrize("fmt,group,d", [("int8", 0, 128), ("int4", 0, 128), ("int8", 0, 64), ("int4", 0, 64), ("int8", 16, 64),
                                         ("int4", 32, 64), ("int8", 32, 128), ("int4", 64, 128), ("e4m3", 0, 128), ("e5m2", 0, 64)])
@pytest.mark.parametrize("hkv,g,n", [(2, 2, 3), (1, 8, 4), (1, 8, 7)])
def test_small_and_mixed_values(fmt, group, d, hkv, g, n, kind):
    ctx = [8000, 700, 90, n]
    b = Batch(ctx, [n] * 4, hkv, g, d, 16, fmt, group, tree=True, seed=31, outliers=False)
    fill(b, kind)
    check(b, b.run(), range(4))


@pytest.mark.parametrize("fmt,group,d", [("e4m3", 0, 128), ("int8", 0, 128), ("int4", 32, 128), ("e5m2", 0, 64), ("int8", 16, 64)])
@pytest.mark.parametrize("g,n", [(2, 4), (8, 4), (8, 7)])
def test_large_logits_of_a_draft_leave_its_siblings_alone(fmt, group, d, g, n):
    """Draft 2's K grows by 40: its own query's logits do, and nothing of the others changes, to the bit."""
    b = Batch([3000 + i for i in range(16)], [n] * 16, 8, g, d, 16, fmt, group, tree=True, seed=32, outliers=False)
    masks = [1 | 1 << i for i in range(n)]   # all children of the first
    mask = R.signed(masks * 16).cuda()
    clean = b.run(tree_mask=mask)
    at = torch.tensor([sum(b.ctx[:i + 1]) - n + 2 for i in range(16)], device="cuda")
    b.k[at] = (b.k[at].float() * 40).half()
    kvq.append(b.k, b.v, b.cache, b.slots, b.scale)
    out = b.run(tree_mask=mask)
    own = torch.arange(16 * n, device="cuda") % n == 2
    assert torch.equal(out[~own], clean[~own]) and not torch.equal(out[own], clean[own])


@pytest.mark.parametrize("fmt,group,d", [("int8", 0, 128), ("int4", 0, 128), ("int8", 0, 64), ("int4", 16, 64)])
@pytest.mark.parametrize("g,n", [(2, 4), (8, 4), (8, 7)])
def test_large_values_of_a_draft_leave_its_siblings_alone(fmt, group, d, g, n):
    """Draft 2's V grows by 2000, from rows of 2^-7: the maxima count V's scale, of the rows that see it only."""
    b = Batch([3000 + i for i in range(16)], [n] * 16, 8, g, d, 16, fmt, group, tree=True, seed=33, outliers=False)
    fill(b, 2.0 ** -7)
    mask = R.signed([1 | 1 << i for i in range(n)] * 16).cuda()
    clean = b.run(tree_mask=mask)
    at = torch.tensor([sum(b.ctx[:i + 1]) - n + 2 for i in range(16)], device="cuda")
    b.v[at] = (b.v[at].float() * 2000).half()
    kvq.append(b.k, b.v, b.cache, b.slots, b.scale)
    out = b.run(tree_mask=mask)
    own = torch.arange(16 * n, device="cuda") % n == 2
    assert torch.equal(out[~own], clean[~own]) and not torch.equal(out[own], clean[own])
    b.masks = [[1 | 1 << i for i in range(n)]] * 16
    check(b, out, [0, 15])


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("fmt,group,bad", [(f, w, x) for f in ("int8", "int4") for w in (0, 32, 64) for x in (NAN, INF, 1e6)]
                         + [("e4m3", 0, NAN), ("e5m2", 0, NAN)])
@pytest.mark.parametrize("g,n", [(2, 4), (8, 4)])
def test_bad_drafts_of_many_short_sequences(fmt, group, bad, g, n):
    """Segments of one tile each, about twenty per CTA: every fifth sequence holds a draft whose V is not finite, or
    with a scale of 10^6.  With group scales (a scale beyond fp16) its own row is NaN or infinite every time; a finite
    row scale gives what 64 bits give, infinite from fp16's largest value on.  Nothing else changes."""
    ctx = [20 + 7 * i % 109 for i in range(400)]
    b = Batch(ctx, [n] * 400, 8, g, 128, 16, fmt, group, tree=True, seed=34, outliers=False)
    b.masks = [[1 | 1 << i for i in range(n)]] * 400
    mask = R.signed(b.masks[0] * 400).cuda()
    clean = b.run(tree_mask=mask)
    at = torch.tensor([sum(ctx[:i + 1]) - n + 2 for i in range(0, 400, 5)], device="cuda")
    blk, row = b.slots[at] // 16, b.slots[at] % 16
    if fmt[0] == "e":
        b.cache.v_codes[blk, :, row] = 0x7F
    else:
        b.cache.v_scales[blk, :, row] = bad
    own = torch.zeros(400, n, dtype=torch.bool, device="cuda")
    own[::5, 2] = True
    own = own.flatten()
    for _ in range(5):
        out = b.run(tree_mask=mask)
        assert torch.equal(out[~own], clean[~own])
        if group or bad != 1e6:
            assert not torch.isfinite(out[own]).any()
    if not group and bad == 1e6:
        for i in range(0, 400, 50):
            k, v = b.kv(i)
            s = b.slots[sum(ctx[:i]):sum(ctx[:i + 1])]
            unit = b.cache.v_scales[s // 16, :, s % 16].double()
            q = b.q[b.start[i]:b.start[i + 1]].double()
            o, bound = VB.attention(q, k, v, unit, v.abs() / unit[..., None], b.masks[i], 128 ** -0.5, ctx[i] - n, False)
            got = out[b.start[i]:b.start[i + 1]].double()
            fits, beyond = o.abs() + bound < 65504, o.abs() - bound > 65520
            assert ((got - o).abs() <= bound)[fits].all() and torch.isinf(got[beyond]).all() and beyond.any()
    assert kvq.device_error_check() == (0, 0)


@pytest.mark.parametrize("fmt,group,d,hkv,g,n,ctx", [
    ("e4m3", 0, 128, 1, 8, 4, [20011]), ("e5m2", 0, 64, 2, 1, 3, [9000, 31]), ("int8", 0, 128, 2, 4, 8, [4999, 1, 5000]),
    ("int4", 32, 128, 1, 8, 5, [12345, 800]), ("e4m3", 0, 128, 4, 8, 13, [3000, 2999, 50]), ("int8", 32, 64, 4, 8, 3, [9000] * 30),
    ("int8", 32, 128, 8, 8, 4, [12000] * 8), ("int8", 64, 128, 4, 8, 2, [9000] * 16), ("int4", 64, 128, 8, 8, 4, [12000] * 8),
    ("int8", 0, 128, 8, 8, 8, [9000] * 8), ("int4", 0, 128, 8, 8, 4, [12000] * 8), ("int4", 0, 64, 8, 8, 4, [12000] * 8),
    ("int8", 0, 128, 8, 1, 5, [5, 0, 9000, 130, 0, 0, 4097, 128, 129, 1, 20000, 640, 0]),
    ("int4", 32, 128, 8, 8, 4, [5, 0, 9000, 130, 0, 0, 4097, 128, 129, 1, 20000, 640, 0])])
def test_long_contexts_to_the_rounding_of_the_output(fmt, group, d, hkv, g, n, ctx):
    """Contexts split over the GPU, held to a bound that a lost tile of 32 tokens breaks."""
    b = Batch(ctx, [min(n, c) for c in ctx], hkv, g, d, 64, fmt, group, tree=False, seed=35, outliers=False)
    check(b, b.run(), range(min(3, len(ctx))) if len(ctx) < 9 else [1, 2, 6, 10, 11] if len(ctx) < 14 else [0, len(ctx) - 1])


@pytest.mark.parametrize("fmt,group", [("int4", 32), ("int8", 64)])
def test_long_sums_of_group_scaled_values(fmt, group):
    """How many results are the 64-bit ones rounded to fp16.  A sum on the tensor cores loses half a step of 2^-23 per
    addition on average (it truncates), always to the same side: after n additions it is off by n 2^-24, and a result lies
    that near a border of fp16's steps (2^-10.5 of it on average) with a chance of n 2^-13.5.  n: 8 products of 16 tokens
    per tile of 128, half of a CTA's tiles; the products with V's residuals have a sum of their own."""
    n, ctx = 4, 115000
    b = Batch([ctx] * 3, [n] * 3, 8, 8, 128, 64, fmt, group, tree=False, seed=36, outliers=False)
    out = b.run().double()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    additions = 8 * -(-3 * 8 * -(-ctx // 128) // sms) / 2
    k, v = b.kv(1)
    q, off = b.q[n:2 * n].double(), 0
    sees = VB.visible(b.masks[1], n, ctx, ctx - n, "cuda")
    for h in range(64):
        w = torch.softmax((q[:, h] @ k[:, h // 8].T * 128 ** -0.5).masked_fill(~sees, -torch.inf), -1)
        off += (out[n:2 * n, h] != (w @ v[:, h // 8]).half().double()).sum().item()
    assert off / (64 * n * 128) <= additions * 2.0 ** -13.5
