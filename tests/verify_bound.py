"""Error bounds of kvq_verify_attention that follow the weights' own size: every token is charged what
its weight loses, so the bound shrinks with V and with the weight (attention_bound of spec_ref charges
every token the loss of the largest).

What a weight loses: it enters P V as 2^(z - M) s, an fp16 value and an fp16 residual, s the scale of V
that it carries (1 where it carries none; the largest of a row's groups for M) and M at most 8 above the largest z + log2 s that the row
has met, less 6: the largest weight lies in 2^6 .. 2^14, a pair holds 2^-22 of its value or an absolute
2^-25, i.e. 2^-31 of the largest weight: 2^-31 max_t(a_t s_t) sum_t |code_t| per output element, a_t
the softmax weights.  The others are those of attention_bound: logits 2 x 24 x 2^-23 A V; 2 ulp of
ex2, the rounding of its argument (below 64: half an ulp 2^-19, times ln 2, numerator and
denominator), scales, residual x residual, merges: 2^-18 V; fp32 sums over the tokens ctx / 4 x 2^-23 V;
V as code x scale in an fp16 pair (group scales on the tcgen05 kernels) 4 x 2^-25; the output 2^-11 |o|, or
2^-25 below the normal range."""
from __future__ import annotations

import torch


def visible(masks, n, ctx, prefix, device):
    sees = torch.zeros(n, ctx, dtype=torch.bool, device=device)
    sees[:, :prefix] = True
    for i, m in enumerate(masks):
        for j in range(n):
            sees[i, prefix + j] = bool(m >> j & 1)
    return sees


def attention(q, k, v, s, codes, masks, sm_scale, prefix, pair):
    """One sequence in 64 bits: q [n][Hq][D]; k, v, codes (|code|) [ctx][Hkv][D], s [ctx][Hkv] the largest scale
    of V a token's weight carries; pair: V enters as an fp16 pair.  Returns (o, bound), [n][Hq][D]."""
    n, Hq, D = q.shape
    ctx, Hkv = k.shape[:2]
    sees = visible(masks, n, ctx, prefix, q.device)
    o = torch.zeros(n, Hq, D, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    for h in range(Hq):
        kv = h // (Hq // Hkv)
        kk, vv = k[:, kv], v[:, kv]
        z = ((q[:, h] @ kk.T) * sm_scale).masked_fill(~sees, -torch.inf)
        w = torch.where(sees.any(-1)[:, None], torch.softmax(z, -1), 0.0)
        A = torch.where(sees, (q[:, h].abs() @ kk.abs().T) * abs(sm_scale), 0.0).amax(-1)[:, None]
        o[:, h] = w @ vv
        top = (w * s[:, kv]).amax(-1)[:, None]
        bound[:, h] = (2.0 ** -11 * o[:, h].abs() + (5 if pair else 1) * 2.0 ** -25
                       + (w @ vv.abs()) * coefficient(A, ctx) + 2.0 ** -31 * top * (sees.double() @ codes[:, kv]))
    return o, bound


def coefficient(A, ctx):
    """Of sum_t w_t |v_t|: what logits, weights and sums may be off by."""
    return 2 * 24 * 2.0 ** -23 * A + 2.0 ** -18 + ctx / 4 * 2.0 ** -23


def rms(x):
    return x.square().mean().sqrt().item()


def rms_bound(o, ctx, A=28.0):
    """Root mean square error over a sequence of ctx tokens with sum |q k| sm_scale <= A: the output's rounding is at
    most 2^-11 of every element; the other errors are per token, of either sign, and sum like the terms of o itself,
    at most the coefficient above of its root mean square."""
    return (2.0 ** -11 + coefficient(A, ctx)) * rms(o) + 2.0 ** -25
