"""The mma.sync kernels of kvq_verify_attention where large calls take them: head_dim 64 with a range of tiles per
warp (what every serving batch of that head_dim is), and head_dim 128 with more than 1024 sequences, a range per warp
and per CTA, row tiles of 8, 16 and 32, up to the largest batch."""
import pytest
import torch

import fp8_int8_quantized_gb300 as kvq
from tests import spec_ref as R
from tests.test_gpu_verify import Batch
from tests.test_gpu_verify_range import check, fill

pytestmark = pytest.mark.gpu

FORMATS = [("e4m3", 0), ("e5m2", 0), ("int8", 0), ("int4", 0), ("int8", 4), ("int8", 2), ("int4", 4), ("int4", 2)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    kvq.build()
    torch.cuda.init()


def range_per_warp(b, rows):
    """Whether the call has so many tiles of 32 tokens that every warp takes a range of its own (12 tiles each)."""
    tiles = len(b.ctx) * b.hkv * -(-max(b.n) * b.g // rows) * -(-max(b.ctx) // 32)
    return tiles >= torch.cuda.get_device_properties(0).multi_processor_count * 8 * 12


@pytest.mark.parametrize("fmt,parts", FORMATS)
@pytest.mark.parametrize("g,n,rows", [(1, 1, 8), (3, 5, 16), (8, 4, 32), (8, 13, 32)])
@pytest.mark.parametrize("kind", [1.0, "mixed"])
def test_head_dim_64_with_a_range_per_warp(fmt, parts, g, n, rows, kind):
    """Ragged, some sequences without new tokens or of one token; results repeat to the bit."""
    ctx = [n + (i * 389) % 1100 for i in range(120)]
    ctx[5], ctx[6], ctx[9] = n, 1100 + n, 32
    new = [i % 4 * n // 3 for i in range(120)]
    new[5] = new[6] = n
    b = Batch(ctx, [min(x, c) for x, c in zip(new, ctx)], 8, g, 64, 32, fmt, 64 // parts if parts else 0, tree=True, seed=41, outliers=False)
    assert range_per_warp(b, rows)
    fill(b, kind)
    out = b.run()
    check(b, out, [1, 5, 6, 7, 9, 30, 61, 90, 117, 119])
    assert torch.equal(out, b.run())


@pytest.mark.parametrize("fmt,parts", FORMATS)
@pytest.mark.parametrize("g,n,rows", [(2, 2, 8), (4, 3, 16), (8, 4, 32), (8, 9, 32)])
@pytest.mark.parametrize("hkv", [1, 8])
def test_head_dim_128_with_more_than_1024_sequences(fmt, parts, g, n, rows, hkv):
    ctx = [n + (i * 37) % 70 for i in range(1025)]
    b = Batch(ctx, [n if i % 7 else i % 2 for i in range(1025)], hkv, g, 128, 16, fmt, 128 // parts if parts else 0, tree=True, seed=42,
              outliers=False)
    assert range_per_warp(b, rows) == (hkv == 8)
    fill(b, 2.0 ** -7)
    out = b.run()
    check(b, out, [0, 1, 2, 511, 767, 1023, 1024])
    assert torch.equal(out, b.run())


@pytest.mark.parametrize("fmt,parts", [("int8", 4), ("int4", 0), ("e4m3", 0)])
def test_head_dim_128_at_the_largest_batch(fmt, parts):
    b = Batch([3 + i % 30 for i in range(4096)], [2] * 4096, 1, 8, 128, 16, fmt, 128 // parts if parts else 0, tree=True, seed=43, outliers=False)
    check(b, b.run(), [0, 1, 2047, 4094, 4095])
    c = Batch([4 + i % 30 for i in range(4096)], [4] * 4096, 1, 8, 128, 16, fmt, 128 // parts if parts else 0, tree=False, seed=44, outliers=False)
    check(c, c.run(), [0, 1, 2047, 4094, 4095])


@pytest.mark.parametrize("fmt,parts", FORMATS)
@pytest.mark.parametrize("d,batch", [(64, 300), (128, 1100)])
def test_bad_drafts_and_empty_rows(fmt, parts, d, batch):
    """A range per warp: NaN in every fifth sequence's draft reaches the row that sees it alone; rows whose mask is
    empty and have nothing before the chunk are zeros."""
    n, g = 4, 4
    ctx = [n + 41 * i % (260 if d == 64 else 60) for i in range(batch)]
    b = Batch(ctx, [n] * batch, 8, g, d, 16, fmt, d // parts if parts else 0, tree=True, seed=45, outliers=False)
    assert range_per_warp(b, 16)
    mask = R.signed([1, 3, 5, 0] * batch).cuda()
    clean = b.run(tree_mask=mask)
    assert not clean[3].any()   # sequence 0: nothing before the chunk
    at = torch.tensor([sum(ctx[:i + 1]) - n + 2 for i in range(0, batch, 5)], device="cuda")
    blk, row = b.slots[at] // 16, b.slots[at] % 16
    if fmt[0] == "e":
        b.cache.v_codes[blk, :, row] = 0x7F
        b.cache.k_codes[blk, :, row] = 0xFF
    else:
        b.cache.v_scales[blk, :, row] = float("nan")
        b.cache.k_scales[blk, :, row] = float("inf")
    out = b.run(tree_mask=mask)
    own = torch.zeros(batch, n, dtype=torch.bool, device="cuda")
    own[::5, 2] = True
    own = own.flatten()
    assert torch.equal(out[~own], clean[~own]) and not torch.isfinite(out[own]).any()
    assert kvq.device_error_check() == (0, 0)
