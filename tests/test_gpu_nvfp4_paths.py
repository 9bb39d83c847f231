"""Paths of the attention over the NVFP4 cache: which kernel a shape takes, keys cut into parts that a second kernel
joins (with bounds and inputs that show every part), workspaces on streams other than the current one."""
import math

import pytest
import torch

import memory_bound_non_b200 as frt
import nvfp4_plain as P
from test_gpu_nvfp4_ops import DEV, DT, Case, gen

pytestmark = pytest.mark.gpu


def takes_tiles(c, **kw):
    """Does the call take the kernel for many rows?  Without polls it gives up its waits and reports bit 1; the kernel
    for few rows has no waits."""
    prev = frt.frt_get_wait_polls()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    try:
        frt.frt_set_wait_polls(0)
        c.run(status=status, **kw)
        torch.cuda.synchronize()
    finally:
        frt.frt_set_wait_polls(prev)
    return bool(status.item() & 2)


def takes_join(c, **kw):
    """Are the keys cut into parts that a second kernel joins?  Only such a call needs a workspace."""
    try:
        c.run(workspace=torch.empty(16, dtype=torch.uint8, device=DEV), **kw)
    except frt.FrtError as e:
        assert e.status == frt.FRT_ERR_INVALID_ARG
        return True
    torch.cuda.synchronize()
    return False


def check_norms(c, out):
    """The error of each head as a norm: see attention_norm_bound."""
    n = sum(c.tokens)
    k, v = c.cache.values("k"), c.cache.values("v")
    ref, _, smax = P.attention(c.q[:n], k, v, c.spans(), c.slots, c.scale, lambda h: h // (c.hq // c.hkv))
    # a warp's (or CTA's) keys follow one another in its sums, then warps and parts
    bound = P.attention_norm_bound(smax, c.hd, c.longest / 8 + 128, DT[c.dt])
    err, size = (out[:n].double() - ref).norm(dim=-1), ref.norm(dim=-1)
    assert (err <= bound * size).all(), float((err / (bound * size)).max())


MANY = [([300], [1200], 16, 1, 64, {}), ([300], [1200], 16, 2, 64, {}), ([700], [1500], 5, 5, 80, {}),
        ([500], [1500], 6, 2, 96, {}), ([200], [900], 16, 8, 128, {}), ([300], [900], 7, 1, 192, {}),
        ([200], [900], 8, 1, 256, {}), ([400, 3, 0, 200], [900, 700, 5, 190], 16, 2, 64, dict(page=16)),
        ([300], [1200], 16, 1, 128, dict(page=64, window=33)), ([41], [8192], 8, 1, 256, {})]
FEW = [([1], [60000], 8, 1, 64, {}), ([10], [978], 8, 1, 256, {}), ([47], [137], 4, 2, 128, {}), ([1], [50001], 4, 2, 128, {}),
       ([41], [600], 8, 1, 256, {})]


@pytest.mark.parametrize("tiles,case", [(True, c) for c in MANY] + [(False, c) for c in FEW])
def test_attn_which_kernel(tiles, case):
    tokens, lens, hq, hkv, hd, kw = case
    assert takes_tiles(Case(tokens, lens, hq, hkv, hd, **kw)) == tiles


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("page,window", [(0, 0), (16, 0), (0, 3000), (20, 5000)])
@pytest.mark.parametrize("tokens,hq,hkv,hd,n", [(41, 8, 1, 256, 8192), (12, 32, 4, 128, 12001), (100, 4, 4, 64, 20003)])
def test_attn_many_rows_joined(tokens, hq, hkv, hd, n, page, window, dt):
    """The kernel for many rows over a long prefix: its parts joined by the second kernel."""
    c = Case([tokens], [n], hq, hkv, hd, dt, page=page, window=window, seed=tokens)
    assert takes_tiles(c) and takes_join(c)
    out = c.check()
    check_norms(c, out)
    assert torch.equal(out, c.run())


def test_attn_many_rows_joined_batch():
    """Sequences of different lengths, one without keys and one without tokens, in parts."""
    c = Case([50, 0, 60], [12001, 40, 37], 8, 1, 128, page=16, extra_tokens=3)
    assert takes_tiles(c) and takes_join(c)
    check_norms(c, c.check())
    c = Case([50, 49], [12001, 0], 8, 1, 128, page=16, causal=False)
    assert takes_tiles(c) and takes_join(c)
    assert (c.check()[50:] == 0).all()


@pytest.mark.parametrize("hq,hkv,hd,n,page,q", [(8, 1, 64, 60000, 0, 1), (4, 2, 128, 50001, 20, 1), (8, 8, 256, 20011, 16, 1),
                                                (40, 2, 128, 33000, 64, 1), (32, 8, 128, 131072, 0, 1), (6, 2, 192, 70000, 0, 2),
                                                (8, 2, 80, 40000, 0, 3)])
def test_attn_long_norms(hq, hkv, hd, n, page, q):
    """Long calls of the kernel for few rows, joined: an error that a part of the keys, lost or weighed wrongly, would
    exceed (test_nvfp4_bounds plants such)."""
    c = Case([q], [n], hq, hkv, hd, page=page, seed=n)
    assert not takes_tiles(c) and takes_join(c)
    check_norms(c, c.run())


@pytest.mark.parametrize("tokens,hq,hkv,hd,n,page", [(1, 8, 1, 64, 60000, 0), (1, 4, 2, 128, 50001, 20), (1, 8, 8, 256, 20011, 16),
                                                     (1, 32, 8, 128, 131072, 0), (2, 6, 2, 192, 70000, 0),
                                                     (41, 8, 1, 256, 8192, 0), (100, 4, 4, 64, 20003, 16),
                                                     (10, 8, 1, 256, 978, 0), (1, 8, 8, 128, 3000, 16)])
def test_attn_every_part_counts(tokens, hq, hkv, hd, n, page):
    """Equal scores (K is zero), and V zero but for one position of each dimension, spread over the whole length: every
    output is that value over n.  A part that is lost, doubled or weighed wrongly changes all outputs by its share of
    the keys, a position that is lost its own."""
    c = Case([tokens], [n], hq, hkv, hd, page=page, causal=False, seed=n)
    c.cache.scales.fill_(1.0)
    c.cache.k.zero_()
    c.cache.v.zero_()
    c.cache.ksf.fill_(0x38)  # 1
    c.cache.vsf.fill_(0x7E)  # 448
    pos = (torch.arange(hd, device=DEV) * (n - 1)) // (hd - 1)  # the first and the last among them
    slots = c.slots(0, pos)
    for d in range(hd):
        c.cache.v[slots[d], :, d // 2] |= 7 << 4 * (d % 2)  # 6
    out = c.run()
    want = 2688.0 / n
    # weights of 2^11, their sums exact in fp32 below 2^24 of them; the reciprocal, two products, half a step of the result
    tol = want * (2.0 ** -21 + torch.finfo(out.dtype).eps / 2)
    assert ((out.double() - want).abs() <= tol).all()


def test_attn_on_another_stream():
    """Calls on streams that are not the current one, with a workspace of their own allocation each: it belongs to
    that stream, so that memory taken on the current stream meanwhile is not the same."""
    cases = [Case([1], [60000], 8, 1, 64, seed=s) for s in (1, 2)] + [Case([41], [8192], 8, 1, 256)]
    refs = [c.run() for c in cases]
    torch.cuda.synchronize()
    sizes = [frt.attn_nvfp4_workspace(c.q, c.hkv, c.longest, max_q_len=len(c.seq)).numel() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        outs = [torch.full_like(r, 9.0) for r in refs]
        torch.cuda.synchronize()
        for c, st, o in zip(cases, streams, outs):
            with torch.cuda.stream(st):
                torch.cuda._sleep(20000000)  # the call's kernels start after what follows here
            frt.frt_attn_nvfp4_kvcache(c.q, *c.cache.args, c.kv_len, o, c.scale, max_kv_len=c.longest, stream=st)
        taken = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
        for st in streams:
            st.synchronize()
        torch.cuda.synchronize()
        for o, r in zip(outs, refs):
            assert torch.equal(o, r)
        assert all((t == 0xFF).all() for t in taken)


@pytest.mark.parametrize("bits", [20, 23, 24, 25])
@pytest.mark.parametrize("tokens,hq,hd,n", [(2400, 16, 64, 131072), (2400, 16, 128, 131072), (1200, 16, 256, 131072),
                                            (2400, 16, 64, 524288), (1, 8, 64, 131072), (400, 4, 128, 131072)])
def test_attn_one_key_above_a_long_tail(tokens, hq, hd, n, bits):
    """One key whose weight is 2^bits times that of every other; V is zero there and one elsewhere.  The output is the
    tail's share of the sum of the weights.  All weights are powers of two (2^11 and 2^(11 - bits)), so products and the
    tail's sum are exact in fp32; a sum that takes the weights one by one would lose all those of half its step or
    less, n 2^-24 of it."""
    q = torch.ones((tokens, hq, hd), device=DEV, dtype=torch.float16)
    one = torch.full(frt.nvfp4_kv_sf_shape(n, 1, hd), 0x38, device=DEV, dtype=torch.uint8)
    scales = torch.ones(2, device=DEV)
    kv_len = torch.full((tokens,), n, device=DEV, dtype=torch.int32)
    out = torch.empty_like(q)
    for at in (0, n // 3):
        k = torch.zeros((n, 1, hd // 2), device=DEV, dtype=torch.uint8)
        v = torch.full((n, 1, hd // 2), 0x22, device=DEV, dtype=torch.uint8)  # 1.0
        k[at], v[at] = 0x22, 0
        frt.frt_attn_nvfp4_kvcache(q, k, one, v, one, scales, kv_len, out, bits * math.log(2) / hd)
        tail = (n - 1) * 2.0 ** -bits
        want = tail / (1 + tail)
        # half a step of the result, and 2^-20 for the exponential, the division and the rescaling of the sums
        assert ((out.double() - want).abs() <= want * (2.0 ** -11 + 2.0 ** -20)).all(), (at, float(out[0, 0, 0]), want)


@pytest.mark.parametrize("tokens", [1, 3, 400])
def test_cache_past_32_bits(tokens):
    """A cache of more than 2^32 bytes a tensor: written, read back and attended to at its ends, through slots and
    pages, by both attention kernels (one token, three, and many rows)."""
    hkv, hd, hq, page = 8, 128, 16, 16
    cap = 2 ** 23 + 2 ** 16
    g = gen(tokens)
    k, v = (torch.empty((cap, hkv, hd // 2), dtype=torch.uint8, device=DEV) for _ in range(2))
    ksf, vsf = (torch.empty(frt.nvfp4_kv_sf_shape(cap, hkv, hd), dtype=torch.uint8, device=DEV) for _ in range(2))
    scales = torch.tensor([0.002, 0.0021], device=DEV)
    n = 2000
    pages = torch.cat((torch.arange(cap // page - 100, cap // page), torch.arange(0, 100)))[torch.randperm(
        200, generator=torch.Generator().manual_seed(1))][:n // page].int().to(DEV)
    slots = (pages.long().repeat_interleave(page) * page + torch.arange(n, device=DEV) % page).int()
    qkv = torch.randn((n, (hq + 2 * hkv) * hd), generator=g, device=DEV).half()
    cos, sin = torch.ones((n, hd // 2), device=DEV), torch.zeros((n, hd // 2), device=DEV)
    q = torch.empty((n, hq, hd), dtype=torch.float16, device=DEV)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    frt.frt_qkv_norm_rope_nvfp4_kvcache(qkv, None, None, cos, sin, pos, q, k, ksf, v, vsf, scales, hq, hkv, hd, slots=slots)
    ko, vo = (torch.empty((n, hkv, hd), dtype=torch.float16, device=DEV) for _ in range(2))
    frt.frt_nvfp4_kvcache_read(k, ksf, v, vsf, scales, slots, ko, vo)
    heads = qkv.view(n, hq + 2 * hkv, hd)
    values = []
    for x, got, gs in ((heads[:, hq:hq + hkv], ko, scales[0]), (heads[:, hq + hkv:], vo, scales[1])):
        codes, sf = P.quantise(x.float(), gs)
        values.append(P.decode(codes, sf, gs))
        assert torch.equal(got, values[-1].float().half())
    out = torch.empty((tokens, hq, hd), dtype=torch.float16, device=DEV)
    kv_len = torch.arange(n - tokens + 1, n + 1, dtype=torch.int32, device=DEV)
    frt.frt_attn_nvfp4_kvcache(q[:tokens].contiguous(), k, ksf, v, vsf, scales, kv_len, out, 0.1, page_table=pages.view(1, -1),
                               page_size=page, max_kv_len=n)
    ref, vmax, smax = P.attention(q[:tokens], *values, [(0, int(m)) for m in kv_len], lambda i, p: p, 0.1, lambda h: h // 2)
    assert ((out.double() - ref).abs() <= P.attention_bound(ref, vmax, smax, n, hd, torch.float16)).all()
