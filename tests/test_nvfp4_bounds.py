"""The bounds that the GPU tests of long attentions use see what they are for: a part of the keys lost or weighed
wrongly (on the CPU, mistakes planted in the 64-bit form)."""
import math

import pytest
import torch

import nvfp4_plain as P


def long_case(hq, hkv, hd, n):
    g = torch.Generator().manual_seed(n)
    k, v = (torch.randn((n, hkv, hd), generator=g, dtype=torch.float64) for _ in range(2))
    q = 2.0 * torch.randn((1, hq, hd), generator=g, dtype=torch.float64)
    return q, k, v


def attend(q, k, v, hq, hkv, keep=None):
    hd = q.shape[2]
    return P.attention(q, k, v, [(0, k.shape[0])], lambda i, p: p if keep is None else torch.where(keep[p], p, -1),
                       1 / math.sqrt(hd), lambda h: h // (hq // hkv))


@pytest.mark.parametrize("hq,hkv,hd,n,parts", [(8, 1, 64, 60000, 75), (4, 2, 128, 50001, 98), (8, 8, 256, 20011, 53)])
def test_norm_bound_sees_a_lost_part(hq, hkv, hd, n, parts):
    q, k, v = long_case(hq, hkv, hd, n)
    ref, _, smax = attend(q, k, v, hq, hkv)
    bound = P.attention_norm_bound(smax, hd, 1000, torch.bfloat16)      # [M, Hq]

    def off(out):
        return ((out - ref).norm(dim=-1) / ref.norm(dim=-1) > bound).any()
    assert not off(ref.bfloat16().double())
    part = n // parts
    for first in (0, part * (parts // 2), n - part):
        keep = torch.ones(n, dtype=torch.bool)
        keep[first:first + part] = False
        assert off(attend(q, k, v, hq, hkv, keep)[0])
    # the part's weights doubled
    lost = torch.zeros(n, dtype=torch.bool)
    lost[part:2 * part] = True
    rest, _, _ = attend(q, k, v, hq, hkv, ~lost)
    only, _, _ = attend(q, k, v, hq, hkv, lost)
    s = torch.einsum("hd,nhd->hn", q[0], k[:, [h // (hq // hkv) for h in range(hq)]]) / math.sqrt(hd)
    w = torch.softmax(s, -1)[:, lost].sum(-1).view(1, hq, 1)
    assert off((rest * (1 - w) + 2 * only * w) / (1 + w))
