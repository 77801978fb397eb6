"""Forward and backward beside relative-position biases that mask with large finite numbers: what such keys
leave in a row's running maximum must not reach the row's other keys. Against plain attention in fp64."""
import numpy as np
import pytest
import torch

import attention_relative_position_gb300 as fa
from exact_buckets import exact_bucket_array

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _plain(q, k, v, cu, bias, causal, scale):
    """out, lse, sum P |v| and the largest scale * sum |q k|, in fp64."""
    total, heads, _ = q.shape
    out, a = torch.zeros_like(q, dtype=torch.float64), torch.zeros_like(q, dtype=torch.float64)
    lse = torch.full((heads, total), -float("inf"), dtype=torch.float64, device=DEV)
    most = 0.0
    for s, e in zip(cu[:-1], cu[1:]):
        n = e - s
        d = np.arange(n)[None] - np.arange(n)[:, None]
        bucket = torch.as_tensor(exact_bucket_array(d, 32, 128, not causal), device=DEV).long()
        for h in range(heads):
            qh, kh, vh = (x[s:e, h].double() for x in (q, k, v))
            x = scale * (qh @ kh.t()) + bias[bucket, h].double()
            most = max(most, float((qh.abs() @ kh.abs().t()).max()) * scale)
            if causal:
                x = x.masked_fill(torch.as_tensor(d > 0, device=DEV), -float("inf"))
            lse[h, s:e] = torch.logsumexp(x, 1)
            p = torch.exp(x - torch.where(torch.isfinite(lse[h, s:e]), lse[h, s:e], 0.0)[:, None])
            out[s:e, h], a[s:e, h] = p @ vh, p @ vh.abs()
    return out, lse, a, most


@pytest.mark.parametrize("low", [-1e6, -1e10, -1e30])
@pytest.mark.parametrize("std", [1.0, 8.0])
@pytest.mark.parametrize("pattern", ["near", "far", "odd"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_large_masking_biases(d, causal, pattern, std, low):
    torch.manual_seed(d + causal)
    lens, heads, scale = [700, 1, 300, 129], 2, d ** -0.5
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v, dout = (torch.randn(int(cu[-1]), heads, d, device=DEV) for _ in range(4))
    q, k, v, dout = (x.to(torch.bfloat16) for x in (q * std, k * std, v, dout))
    bias = 0.5 * torch.randn(32, heads, device=DEV)
    per = 32 if causal else 16  # buckets of a direction
    b = bias.view(32 // per, per, heads)
    if pattern == "near":
        b[:, :per - 1] = low
    elif pattern == "far":
        b[:, per // 2:] = low
    else:
        b[:, 1::2] = low
    args = dict(bias_table=bias, num_buckets=32, max_distance=128, bidirectional=not causal, causal=causal,
                softmax_scale=scale)
    cud = torch.as_tensor(cu, dtype=torch.int32, device=DEV)
    out, lse = fa.fat_attn_fwd(q, k, v, cud, max(lens), **args)
    torch.cuda.synchronize()
    assert fa.fat_attn_get_device_error() == 0
    hidden = torch.where(bias <= low, -float("inf"), bias)
    ro, rl, a, s = _plain(q, k, v, cu, hidden, causal, scale)
    fin = torch.isfinite(rl)
    assert float(fin.float().mean()) > 0.1 and torch.isfinite(out).all() and torch.isfinite(lse).all()
    # a logit: d products, scale and bias in fp32; P rounded to bf16; the output rounded
    big = float(bias[bias > low].abs().max())
    ex = (d * s + 4 * (s + big)) * 2.0 ** -24
    rows = fin.t()
    tol = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2 * ex + 2.0 ** -18) * a * 1.01 + 1e-30
    assert ((out.double() - ro).abs() <= tol)[rows].all()
    assert ((lse.double() - rl).abs() <= ex + 2.0 ** -18 + 2.0 ** -22 * rl.abs())[fin].all()
    # the gradient of the values: sums of P dout over the rows
    dv = fa.fat_attn_bwd(q, k, v, cud, max(lens), out, lse, dout, **args)[2]
    assert fa.fat_attn_get_device_error() == 0 and torch.isfinite(dv).all()
