"""kvq_append_rotary with its rows side by side in one buffer."""
import pytest
import torch

import fp8_int8_quantized_gb300 as kvq
from tests.test_gpu_rotary import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 50, 3000])
@pytest.mark.parametrize("first", [True, False])
def test_rotated_queries_beside_the_inputs(T, first):
    """q_out as columns of the same rows as q, k and v, before or behind them: accepted, and the inputs stay."""
    kvq.build()
    c = Case(T, 8, 2, 128, 16, "e4m3", seed=9, fused=False)
    want = c.run(c.fresh()).clone()
    parts = [c.q, c.k, c.v]
    buf = torch.cat([torch.zeros_like(c.q), *parts] if first else [*parts, torch.zeros_like(c.q)], 1)
    out, q, k, v = buf.split([8, 8, 2, 2], 1) if first else [buf[:, 12:], *buf[:, :12].split([8, 2, 2], 1)]
    c.q, c.k, c.v = q, k, v
    cache = c.fresh()
    got = c.run(cache, q_out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, want)
    assert all(torch.equal(a, b) for a, b in zip((q, k, v), parts))
    c.check(cache, out)
    # the last head over k's (or behind it, over the next token's q) is refused
    with pytest.raises(kvq.KvqError) as e:
        c.run(cache, q_out=buf[:, 1:9] if first else buf[:, 11:19])
    assert e.value.status == 1
