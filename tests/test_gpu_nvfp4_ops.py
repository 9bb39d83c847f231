"""NVFP4 KV cache (writer, reader, attention) and the NVFP4 matrix-vector
product on the GPU, against plain 64-bit forms (nvfp4_plain): head layouts,
lengths from none to long, odd sizes, masks that leave rows empty, pages,
factors that are NaN in unseen places, streams, captured graphs, and a run of
the operators together."""
import math
import threading

import pytest
import torch

import memory_bound_non_b200 as frt
import nvfp4_plain as P
from test_gpu_debug_bounds import both_builds

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def gen(seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    return g


def randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV)


# ------------------------------------------------------------------ cache --
def rope_tables(n, hd):
    ang = torch.outer(torch.arange(n, dtype=torch.float64),
                      1e4 ** (-2.0 * torch.arange(hd // 2, dtype=torch.float64) / hd))
    return ang.cos().float().to(DEV), ang.sin().float().to(DEV)


class Cache:
    """A cache whose bytes are all set: 0xA5 codes, 0x5A factors."""

    def __init__(self, capacity, hkv, hd, scales):
        self.capacity, self.hkv, self.hd = capacity, hkv, hd
        self.k, self.v = (torch.full((capacity, hkv, hd // 2), 0xA5, dtype=torch.uint8, device=DEV) for _ in range(2))
        shape = frt.nvfp4_kv_sf_shape(capacity, hkv, hd)
        self.ksf, self.vsf = (torch.full(shape, 0x5A, dtype=torch.uint8, device=DEV) for _ in range(2))
        self.scales = torch.tensor(scales, dtype=torch.float32, device=DEV)

    @property
    def args(self):
        return self.k, self.ksf, self.v, self.vsf, self.scales

    def set(self, which, values):
        """Quantise values [n, hkv, hd] into slots 0 .. n-1; the other slots get NaN factors."""
        codes, sf = P.quantise(values, self.scales[0 if which == "k" else 1])
        n = values.shape[0]
        getattr(self, which)[:n] = codes
        rows = torch.full((self.capacity, self.hkv, self.hd // 16), 0x7F, dtype=torch.uint8, device=DEV)
        rows[:n] = sf
        setattr(self, which + "sf", P.sf_pack(rows))

    def values(self, which):
        sf = P.sf_rows(getattr(self, which + "sf"), self.capacity)
        return P.decode(getattr(self, which), sf, self.scales[0 if which == "k" else 1])


def write(c, qkv, qw, kw, cos, sin, pos, hq, slots=None, status=None):
    q = torch.full((qkv.shape[0], hq, c.hd), 7.0, dtype=qkv.dtype, device=DEV)
    frt.frt_qkv_norm_rope_nvfp4_kvcache(qkv, qw, kw, cos, sin, pos, q, *c.args, hq, c.hkv, c.hd, slots=slots,
                                        status=status)
    return q


def check_write(dt, m, hq, hkv, hd, norm, with_slots, seed=1, mutate=None):
    g = gen(seed)
    t = DT[dt]
    max_pos, cap = 300, m + 37
    qkv = randn((m, (hq + 2 * hkv) * hd), g).to(t)
    if mutate is not None:
        mutate(qkv)
    qw, kw = [(1 + 0.2 * randn((hd,), g)).to(t) if norm else None for _ in range(2)]
    cos, sin = rope_tables(max_pos, hd)
    if with_slots:
        pos = torch.randint(0, max_pos, (m,), generator=g, device=DEV, dtype=torch.int32)
        slots = torch.randperm(cap, generator=g, device=DEV)[:m].int()
    else:
        max_pos = cap if cap <= max_pos else max_pos
        pos = torch.randperm(min(cap, max_pos), generator=g, device=DEV)[:m].int()
        slots = None
    where = (slots if slots is not None else pos).long()
    c = Cache(cap, hkv, hd, (0.0019, 0.0021))
    q = write(c, qkv, qw, kw, cos, sin, pos, hq, slots)
    heads = qkv.view(m, hq + 2 * hkv, hd)
    cs, sn = cos[pos.long()], sin[pos.long()]
    ref = P.norm_rope(heads[:, :hq], qw, cs, sn, 1e-6)
    # norm and rotation in 32 bits: a few roundings of the largest term each, then half a step
    big = P.norm_rope(heads[:, :hq], qw, cs, sn, 1e-6).abs().amax(-1, keepdim=True) * 2
    half_step = torch.finfo(t).eps / 2
    fine = torch.isfinite(ref)
    tol = 8 * 2.0 ** -23 * big + 1.01 * half_step * ref.abs() + torch.finfo(t).smallest_normal * half_step
    assert (((q.double() - ref).abs() <= tol) | ~fine).all()
    k = P.norm_rope(heads[:, hq:hq + hkv], kw, cs, sn, 1e-6).float()
    v = heads[:, hq + hkv:].float()
    for which, y, gs in (("k", k, c.scales[0]), ("v", v, c.scales[1])):
        codes, sf = P.quantise(y, gs)
        assert torch.equal(getattr(c, which)[where], codes), which
        rows = P.sf_rows(getattr(c, which + "sf"), cap)
        assert torch.equal(rows[where], sf), which
        # every other byte as it was, the factors that pad the last quad too
        other = torch.ones(cap, dtype=torch.bool, device=DEV)
        other[where] = False
        assert (getattr(c, which)[other] == 0xA5).all() and (rows[other] == 0x5A).all()
        assert (getattr(c, which + "sf").permute(0, 3, 1, 2).flatten(0, 1)[cap:] == 0x5A).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,hd", [(1, 1, 16), (2, 1, 32), (3, 1, 48), (8, 8, 64), (5, 5, 80), (6, 2, 96), (8, 2, 112),
                                       (32, 8, 128), (4, 4, 176), (9, 3, 192), (8, 1, 256)])
def test_write_head_layouts(dt, hq, hkv, hd):
    check_write(dt, 21, hq, hkv, hd, norm=True, with_slots=True)
    check_write(dt, 5, hq, hkv, hd, norm=False, with_slots=False, seed=2)


@pytest.mark.parametrize("m", [1, 2, 3, 33, 700])
def test_write_batches(m):
    check_write("bf16", m, 16, 8, 128, norm=True, with_slots=True, seed=m)


def test_write_special_blocks():
    """All-zero blocks, values that saturate, NaN and infinite elements."""
    def mutate(qkv):
        x = qkv.view(qkv.shape[0], 4, 64)  # q, q, k, v of 64
        x[0, 3, :16] = 0
        x[1, 3] = 1000.0
        x[2, 3, 5] = float("nan")
        x[3, 3, 40] = float("inf")
        x[4, 2, 7] = float("nan")
        x[5, 3] = 1e-30
    check_write("bf16", 9, 2, 1, 64, norm=False, with_slots=True, seed=5, mutate=mutate)


def test_write_skips_rows_and_reports():
    g = gen(3)
    qkv = randn((6, 3 * 64), g).bfloat16()
    cos, sin = rope_tables(10, 64)
    c = Cache(8, 1, 64, (0.002, 0.002))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pos = torch.tensor([0, 9, 10, -1, 3, 4], dtype=torch.int32, device=DEV)
    slots = torch.tensor([0, -1, 2, 3, 8, 5], dtype=torch.int32, device=DEV)
    q = write(c, qkv, None, None, cos, sin, pos, 1, slots, status)
    assert status.item() == 1
    assert (q[1:5] == 7.0).all() and not (q[0] == 7.0).any() and not (q[5] == 7.0).any()
    assert (c.k[[1, 2, 3, 4, 6, 7]] == 0xA5).all() and (c.v[[1, 2, 3, 4, 6, 7]] == 0xA5).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("hkv,hd,n", [(1, 16, 1), (3, 48, 7), (8, 128, 181), (5, 80, 600), (1, 256, 1)])
def test_read_is_exact(dt, hkv, hd, n):
    g = gen(n)
    cap = n + 13
    c = Cache(cap, hkv, hd, (0.0123, 3.7e-5))
    c.set("k", randn((cap, hkv, hd), g) * 3)
    c.set("v", randn((cap, hkv, hd), g) * 1e-2)
    slots = torch.randperm(cap, generator=g, device=DEV)[:n].int()
    slots[-1] = slots[0]  # the same slot twice
    for s in (slots, None):
        ko, vo = (torch.empty((n, hkv, hd), dtype=DT[dt], device=DEV) for _ in range(2))
        frt.frt_nvfp4_kvcache_read(*c.args, s, ko, vo)
        idx = s.long() if s is not None else torch.arange(n, device=DEV)
        for which, out in (("k", ko), ("v", vo)):
            assert torch.equal(out, c.values(which)[idx].float().to(DT[dt]))


def test_read_reports_bad_slots():
    c = Cache(8, 2, 32, (1.0, 1.0))
    ko, vo = (torch.full((3, 2, 32), 5.0, dtype=torch.float16, device=DEV) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    frt.frt_nvfp4_kvcache_read(*c.args, torch.tensor([-1, 3, 8], dtype=torch.int32, device=DEV), ko, vo, status=status)
    assert status.item() == 1 and (ko[[0, 2]] == 5.0).all() and (vo[[0, 2]] == 5.0).all()
    assert not (ko[1] == 5.0).any()


# -------------------------------------------------------------- attention --
class Case:
    """Sequences of `tokens` tokens over `lens` positions (kv_len of the last
    token; causal: one less for each token before it), paged or not."""

    def __init__(self, tokens, lens, hq, hkv, hd, dt="bf16", causal=True, window=0, page=0, seed=0, gain=2.0, scale=None,
                 kv_len=None, extra_tokens=0):
        g = gen(1000 + seed)
        self.tokens, self.hq, self.hkv, self.hd, self.dt, self.window, self.page = tokens, hq, hkv, hd, dt, window, page
        b = len(tokens)
        self.m = sum(tokens) + extra_tokens
        self.seq = [i for i in range(b) for _ in range(tokens[i])]
        first = [sum(tokens[:i]) for i in range(b + 1)]
        if kv_len is None:
            kv_len = [max(lens[i] - (tokens[i] - 1 - j if causal else 0), 0) for i in range(b) for j in range(tokens[i])]
        self.lens = kv_len
        self.kv_len = torch.tensor(kv_len + [0] * extra_tokens, dtype=torch.int32, device=DEV)
        self.indptr = torch.tensor(first, dtype=torch.int32, device=DEV)
        longest = max(lens + [1])
        if page:
            need = [-(-n // page) for n in lens]
            order = torch.randperm(sum(need) + 2, generator=torch.Generator().manual_seed(seed)).tolist()
            self.table = torch.full((b, max(need + [1])), -7, dtype=torch.int32, device=DEV)
            at = 0
            for i in range(b):
                for j in range(need[i]):
                    self.table[i, j] = order[at]
                    at += 1
            cap = (sum(need) + 2) * page
        else:
            self.table = None
            cap = longest + 3
        self.longest = longest
        self.cache = Cache(cap, hkv, hd, (0.0019, 0.0022))
        used = cap if page else longest
        self.cache.set("k", randn((used, hkv, hd), g))
        self.cache.set("v", randn((used, hkv, hd), g))
        self.q = (gain * randn((self.m, hq, hd), g)).to(DT[dt])
        self.scale = 1.0 / math.sqrt(hd) if scale is None else scale
        self.kw = {}

    def run(self, **kw):
        out = torch.full(self.q.shape, 9.0, dtype=self.q.dtype, device=DEV)
        a = dict(window=self.window, q_indptr=self.indptr, page_table=self.table, page_size=self.page,
                 max_q_len=max(self.tokens + [1]), max_kv_len=self.longest)
        a.update(self.kw)
        a.update(kw)
        frt.frt_attn_nvfp4_kvcache(self.q, *self.cache.args, self.kv_len, out, self.scale, **a)
        return out

    def slots(self, i, pos):
        if self.table is None:
            return pos
        pages = self.table[self.seq[i]].long()[pos // self.page]
        ok = (pages >= 0) & (pages < self.cache.capacity // self.page)
        return torch.where(ok, pages * self.page + pos % self.page, -1)

    def spans(self):
        return [(max(0, n - self.window) if self.window else 0, n) for n in self.lens]

    def expected(self, rows=None):
        n = sum(self.tokens)
        k, v = self.cache.values("k"), self.cache.values("v")
        q = self.q[:n]
        ref, vmax, smax = P.attention(q, k, v, self.spans(), self.slots, self.scale, lambda h: h // (self.hq // self.hkv))
        return ref, P.attention_bound(ref, vmax, smax, self.longest, self.hd, DT[self.dt])

    def check(self, **kw):
        out = self.run(**kw)
        n = sum(self.tokens)
        ref, tol = self.expected()
        err = (out[:n].double() - ref).abs()
        bad = ~(err <= tol)
        assert not bad.any(), "%d of %d outside, worst %.3g of the bound" % (
            int(bad.sum()), bad.numel(), float((err / tol)[bad].max()) if bad.any() else 0)
        assert (out[n:] == 9.0).all()  # tokens of no sequence
        return out


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,hd", [(1, 1, 16), (3, 1, 32), (2, 2, 48), (8, 2, 64), (5, 1, 80), (8, 8, 96), (6, 2, 112),
                                       (32, 8, 128), (8, 1, 176), (16, 2, 192), (8, 1, 256), (40, 5, 240)])
def test_attn_head_layouts(dt, hq, hkv, hd):
    Case([1], [77], hq, hkv, hd, dt).check()
    Case([3], [130], hq, hkv, hd, dt, seed=1).check()


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 1000])
def test_attn_lengths(n):
    Case([1], [n], 8, 2, 128, seed=n).check()
    Case([2], [n], 2, 1, 256, dt="f16", seed=n).check()
    Case([1], [n], 4, 4, 64, page=4, seed=n).check()


@pytest.mark.parametrize("tokens", [1, 2, 4, 5, 9, 17, 33, 47])
def test_attn_row_counts(tokens):
    """Query rows around every row tile of the kernels for few rows."""
    Case([tokens], [tokens + 90], 4, 2, 128, seed=tokens).check()
    Case([tokens], [tokens + 90], 3, 1, 192, seed=tokens, causal=False).check()


@pytest.mark.parametrize("page", [0, 4, 16, 20, 64])
@pytest.mark.parametrize("window", [0, 1, 5, 40, 4000])
def test_attn_batches(page, window):
    if page == 0:
        Case([3, 1, 0, 7], [60, 60, 60, 60], 8, 2, 64, window=window).check()
        return
    Case([1, 3, 0, 2, 8, 1], [1, 50, 30, 129, 8, 400], 8, 2, 64, page=page, window=window, seed=page).check()
    Case([1] * 9, [9, 200, 33, 64, 1, 2, 3, 4, 700], 4, 1, 96, dt="f16", page=page, window=window, seed=page).check()


def test_attn_empty_rows():
    """Tokens that see nothing give zeros: the first of a sequence longer than its keys, and a batch with none."""
    c = Case([6], [3], 4, 2, 64)
    out = c.check()
    assert (out[:3] == 0).all() and not (out[3:] == 0).all()
    c = Case([2, 1], [0, 0], 4, 2, 64, causal=False)
    assert (c.check() == 0).all()
    c = Case([2], [5], 4, 2, 128, kv_len=[0, 5], window=2)
    assert (c.check()[0] == 0).all()


def test_attn_bidirectional_and_cross():
    """Every token of a sequence sees all of it; queries of one length over a state of another."""
    Case([10], [978], 8, 1, 256, causal=False).check()
    Case([37, 5], [200, 13], 4, 4, 64, causal=False, page=16).check()


def test_attn_tokens_behind_the_last_sequence():
    Case([2, 3], [40, 50], 4, 2, 128, page=16, extra_tokens=4).check()


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-4, 5.0])
def test_attn_scales(scale):
    c = Case([4], [150], 4, 2, 64, scale=scale)
    # the bound holds for any scale; at 5 the softmax takes one key almost alone
    c.check()


def test_attn_default_arguments():
    c = Case([1], [50], 4, 2, 64)
    a = c.run()
    b = torch.empty_like(a)
    frt.frt_attn_nvfp4_kvcache(c.q, *c.cache.args, c.kv_len, b, c.scale)
    ref, tol = c.expected()
    assert ((b.double() - ref).abs() <= tol).all()


def poison(c, which, slot, head=0, block=0):
    sf = getattr(c.cache, which + "sf")
    sf[slot // 4, head, block, slot % 4] = 0xFF if slot % 2 else 0x7F


MANY = dict(tokens=[300], hq=16, hkv=1, hd=64)  # a shape that the kernel for many rows takes (with 1200 keys)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("which", ["k", "v"])
def test_attn_nan_factors(many, which):
    """A NaN factor in a position that a row sees makes the row NaN; in the others' it has no effect."""
    if many:
        c = Case(MANY["tokens"], [1200], MANY["hq"], 1, MANY["hd"])
        at = 1000
    else:
        c = Case([8], [90], 4, 2, 64)
        at = 86
    before = c.run()
    poison(c, which, at)
    out = c.run()
    sees = c.kv_len > at
    group = c.hq // c.hkv
    hit = torch.zeros(c.q.shape[:2], dtype=torch.bool, device=DEV)
    hit[:, :group] = sees.unsqueeze(1)
    assert sees.any() and not sees.all()
    assert torch.isnan(out[hit]).all()
    assert torch.equal(out[~hit], before[~hit])


def test_attn_nan_factors_outside_the_window():
    c = Case([1, 1], [200, 180], 4, 2, 128, window=32, page=16)
    before = c.run()
    for i in range(2):
        n = c.lens[i]
        for p in list(range(0, n - 32)):
            s = int(c.slots(i, torch.tensor([p], device=DEV)))
            for which in ("k", "v"):
                poison(c, which, s, head=p % 2, block=p % 8)
    assert torch.equal(c.run(), before)


def test_attn_reports_lengths():
    c = Case([3], [40], 4, 2, 64)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    c.run(status=status)
    assert status.item() == 0
    good = c.kv_len.clone()
    ref = c.run()
    for bad, clamped in ((-5, 0), (41, 40), (2 ** 31 - 1, 40)):
        status.zero_()
        c.kv_len = good.clone()
        c.kv_len[1] = bad
        out = c.run(status=status)
        assert status.item() == 1
        c.kv_len[1] = clamped
        assert torch.equal(out, c.run())
        assert torch.equal(out[[0, 2]], ref[[0, 2]])
    # a bound above what the cache holds
    c.kv_len = good.clone()
    c.kv_len[1] = 1000
    status.zero_()
    c.cache.set("k", randn((c.cache.capacity, 2, 64), gen(1)))
    c.cache.set("v", randn((c.cache.capacity, 2, 64), gen(2)))
    out = c.run(status=status, max_kv_len=2000)
    assert status.item() == 1
    c.kv_len[1] = c.cache.capacity
    assert torch.equal(out, c.run(max_kv_len=2000))


def test_attn_reports_pages():
    c = Case([1, 2], [100, 90], 4, 2, 64, page=16)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    c.run(status=status)
    assert status.item() == 0
    c.table[0, 2] = -1
    c.table[1, 1] = c.cache.capacity // 16
    c.check(status=status)  # the positions of those pages are left out
    assert status.item() == 1
    status.zero_()
    c.kv_len[0] = 10000  # past the page table
    c.run(status=status, max_kv_len=20000)
    assert status.item() == 1


@pytest.mark.parametrize("indptr", [[0, 5, 3], [-2, 2, 4], [0, 2, 100], [3, 1, 4]])
def test_attn_reports_sequences(indptr):
    c = Case([2, 2], [40, 50], 4, 2, 64, page=16)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    c.run(q_indptr=torch.tensor(indptr, dtype=torch.int32, device=DEV), status=status)
    assert status.item() == 1


def test_attn_sequence_longer_than_its_bound():
    c = Case([4], [40], 4, 2, 64)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    whole = c.run()
    out = c.run(max_q_len=3, status=status)
    assert status.item() == 1 and torch.equal(out[:3], whole[:3]) and (out[3] == 9.0).all()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,hd,tokens,n", [(16, 2, 64, 300, 1200), (5, 5, 80, 700, 1500), (6, 2, 96, 500, 1500),
                                               (16, 8, 128, 200, 900), (7, 1, 192, 300, 900), (8, 1, 256, 200, 900)])
def test_attn_many_rows(dt, hq, hkv, hd, tokens, n):
    Case([tokens], [n], hq, hkv, hd, dt).check()
    Case([tokens], [n], hq, hkv, hd, dt, causal=False, page=20, seed=1).check()


def test_attn_many_rows_masks():
    Case([400, 3, 0, 200], [900, 700, 5, 190], 16, 2, 64, page=16).check()       # rows that see nothing, short sequences
    Case([500], [1200], 16, 2, 64, window=100).check()
    Case([500], [1200], 16, 2, 64, scale=-0.2).check()
    Case([500], [1200], 16, 2, 64, scale=0.0).check()
    Case([300], [1200], 16, 1, 128, page=64, window=33, extra_tokens=5).check()
    c = Case([500], [1200], 16, 2, 64, page=16)
    c.table[0, 3] = -1
    c.table[0, 70] = 10 ** 6
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    c.check(status=status)
    assert status.item() == 1


def test_attn_many_rows_wait_that_runs_out():
    """With no polls allowed the kernel gives its waits up, reports bit 1 and ends; the next call is right."""
    c = Case(MANY["tokens"], [1200], MANY["hq"], 1, MANY["hd"])
    prev = frt.frt_get_wait_polls()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    try:
        frt.frt_set_wait_polls(0)
        c.run(status=status)
        torch.cuda.synchronize()
    finally:
        frt.frt_set_wait_polls(prev)
    assert status.item() & 2
    c.check()


@pytest.mark.parametrize("hq,hkv,hd,n,page", [(8, 1, 64, 60000, 0), (4, 2, 128, 50001, 20), (8, 8, 256, 20011, 16),
                                              (40, 2, 128, 33000, 64)])
def test_attn_long(hq, hkv, hd, n, page):
    """Keys cut into more chunks than a cluster has CTAs (a workspace and a second kernel)."""
    c = Case([1], [n], hq, hkv, hd, page=page)
    assert frt.attn_nvfp4_workspace(c.q, hkv, n) is not None
    c.check()
    # a bound far above the length: chunks without work
    c = Case([2], [100], hq, hkv, hd, page=page, seed=1)
    if page:
        c.table = torch.cat((c.table, torch.full((1, n // page), -1, dtype=torch.int32, device=DEV)), 1).contiguous()
    c.check(max_kv_len=n)


def test_attn_same_bits_every_time():
    for c in (Case([1], [60000], 8, 1, 64), Case([10], [978], 8, 1, 256), Case([300], [1200], 16, 1, 64)):
        first = c.run()
        for _ in range(3):
            assert torch.equal(c.run(), first)


def test_attn_streams_and_graphs():
    """Calls on side streams, and two captured graphs with a workspace each, replayed at once on changed inputs."""
    cases = [Case([1], [60000], 8, 1, 64, seed=s) for s in (1, 2)]
    refs = [c.run() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    for c, st in zip(cases, streams):
        outs.append(c.run(stream=st))                      # the workspace belongs to that stream
    for st in streams:
        st.synchronize()
    # (run() fills `out` on the current stream: wait for it before comparing)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c, st in zip(cases, streams):
        ws = frt.attn_nvfp4_workspace(c.q, 1, c.longest)
        out = torch.empty_like(c.q)
        args = (c.q, *c.cache.args, c.kv_len, out, c.scale)
        kw = dict(max_kv_len=c.longest, workspace=ws)
        with torch.cuda.stream(st):
            frt.frt_attn_nvfp4_kvcache(*args, **kw)
            st.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                frt.frt_attn_nvfp4_kvcache(*args, **kw)
        graphs.append((g, ws))
        outs.append(out)
    for _ in range(5):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        assert torch.equal(o, r)
    # a shorter sequence in a captured graph: lengths are read on the device
    c = cases[0]
    c.kv_len.fill_(777)
    c.lens = [777]
    with torch.cuda.stream(streams[0]):
        graphs[0][0].replay()
    torch.cuda.synchronize()
    ref, tol = c.expected()
    assert ((outs[0].double() - ref).abs() <= tol).all()


# ----------------------------------------------------------------- matvec --
def weights(n, k, g, layout):
    w = randn((n, k), g) / math.sqrt(k)
    scale = (w.abs().amax() / 2688).reshape(1)
    codes, sf = P.quantise(w, scale[0])
    return codes, (P.sf_swizzle(sf) if layout == "swizzled" else sf), scale, P.decode(codes, sf, scale[0])


def matvec_case(m, n, k, fmt, dt="bf16", layout="rows", bias=False, seed=0, x=None, off=0):
    g = gen(seed)
    t = DT[dt]
    wc, wsf, ws, w = weights(n, k, g, layout)
    if x is None:
        x = randn((m, k), g)
        x[:, ::17] *= 40
    xs = xsf = None
    if fmt == "16":
        xd = x.to(t)
        xv = xd.double()
    elif fmt == "nvfp4":
        xs = (x.abs().amax() / 2688).reshape(1)
        xd, sf = P.quantise(x, xs[0])
        xv = P.decode(xd, sf, xs[0])
        xsf = P.sf_swizzle(sf) if layout == "swizzled" else sf
    else:
        nb = -(-k // 128)
        pad = torch.zeros((m, nb * 128), device=DEV)
        pad[:, :k] = x
        pad = pad.view(m, nb, 128)
        xs = (pad.abs().amax(-1) / 448) if fmt == "e4m3_block" else (x.abs().amax() / 448).reshape(1)
        q = (pad / (xs.unsqueeze(-1) if fmt == "e4m3_block" else xs)).clamp(-448, 448).to(torch.float8_e4m3fn)
        xv = (q.double() * (xs.double().unsqueeze(-1) if fmt == "e4m3_block" else xs.double())).flatten(1)[:, :k]
        xd = q.view(torch.uint8).flatten(1)[:, :k].contiguous()
        xs = xs.contiguous()
    b = randn((n,), g).to(t) if bias else None
    raw = torch.full((m * n + off + 8,), 3.0, dtype=t, device=DEV)
    y = raw[off:off + m * n].view(m, n)
    frt.frt_matvec_nvfp4(xd, wc, wsf, ws, y, bias=b, x_format=fmt, x_scales=xs, x_sf=xsf, sf_layout=layout)
    assert (raw[:off] == 3.0).all() and (raw[off + m * n:] == 3.0).all()
    ref = xv @ w.t() + (b.double() if bias else 0.0)
    return y, ref, P.matvec_bound(xv, w, ref, t)


def check_matvec(*a, **kw):
    y, ref, tol = matvec_case(*a, **kw)
    bad = ~((y.double() - ref).abs() <= tol)
    assert not bad.any(), "%d of %d outside" % (int(bad.sum()), bad.numel())


@pytest.mark.parametrize("layout", ["rows", "swizzled"])
@pytest.mark.parametrize("fmt", ["16", "e4m3", "e4m3_block", "nvfp4"])
@pytest.mark.parametrize("k", [16, 32, 48, 64, 112, 128, 144, 160, 272, 512, 528, 1040])
def test_matvec_depths(fmt, layout, k):
    for i, (m, n) in enumerate([(1, 100), (3, 33), (11, 17)]):
        check_matvec(m, n, k, fmt, dt="bf16" if i % 2 else "f16", layout=layout, bias=i == 1, seed=k + i)


@pytest.mark.parametrize("fmt", ["16", "e4m3", "e4m3_block", "nvfp4"])
@pytest.mark.parametrize("m", [1, 2, 5, 7, 8, 9, 15, 16, 17, 31, 32, 33, 41, 48, 49, 63, 64, 65, 130])
def test_matvec_rows(fmt, m):
    check_matvec(m, 200, 272, fmt, layout="swizzled" if m % 2 else "rows", bias=m % 3 == 0, seed=m)
    check_matvec(m, 77, 256, fmt, dt="f16", seed=m + 1)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 130, 2047, 2048, 2568, 40001])
def test_matvec_widths(n):
    check_matvec(1, n, 256, "16", seed=n)
    check_matvec(10, n, 144, "nvfp4", bias=True, layout="swizzled", seed=n)
    check_matvec(40, n, 128, "e4m3_block", dt="f16", seed=n)


@pytest.mark.parametrize("m,n,k,fmt", [(1, 300, 16384, "16"), (8, 64, 20000, "16"), (10, 1024, 4096, "nvfp4"),
                                       (41, 4000, 2048, "e4m3_block"), (64, 64, 8192, "16"), (64, 3000, 8192, "e4m3"),
                                       (17, 40, 12304, "16"), (64, 16, 30000, "e4m3_block")])
def test_matvec_deep(m, n, k, fmt):
    """x that does not fit shared memory at once, k split over warps and the CTAs of a cluster."""
    check_matvec(m, n, k, fmt, seed=m)


@pytest.mark.parametrize("fmt", ["16", "e4m3", "e4m3_block", "nvfp4"])
@pytest.mark.parametrize("m,n,k,layout", [(17, 8200, 2064, "rows"), (24, 4100, 4128, "swizzled"), (32, 37500, 448, "rows"),
                                          (25, 1030, 16384, "swizzled"), (150, 8192, 2048, "rows")])
def test_matvec_many_weights(fmt, m, n, k, layout):
    check_matvec(m, n, k, fmt, dt="f16" if m == 24 else "bf16", layout=layout, bias=m == 32, seed=m)


@pytest.mark.parametrize("off", [1, 2, 4])
def test_matvec_unaligned_output(off):
    check_matvec(3, 64, 128, "16", off=off, bias=True)
    check_matvec(20, 64, 128, "e4m3", off=off)


def test_matvec_wide_range():
    """bf16 rows whose groups and elements differ by many powers of two, zeros, the smallest and largest numbers."""
    g = gen(4)
    x = randn((9, 512), g) * torch.exp2(torch.randint(-60, 60, (9, 512), generator=g, device=DEV).float())
    x[1] = 0
    x[2, :128] = 0
    x[3] *= 2.0 ** -60
    x[4, 100] = 3e38
    x[5] = 1e-38
    x[6, 1:] = 0
    check_matvec(9, 100, 512, "16", x=x)


def test_matvec_nan_and_bits():
    g = gen(5)
    wc, wsf, ws, w = weights(50, 256, g, "rows")
    x = randn((4, 256), g).half()
    y, again = (torch.empty((4, 50), dtype=torch.float16, device=DEV) for _ in range(2))
    frt.frt_matvec_nvfp4(x, wc, wsf, ws, y)
    bad = wsf.clone()
    bad[7, 3] = 0x7F
    frt.frt_matvec_nvfp4(x, wc, bad, ws, again)
    keep = torch.arange(50, device=DEV) != 7
    assert torch.isnan(again[:, 7]).all() and torch.equal(again[:, keep], y[:, keep])
    xn = x.clone()
    xn[2, 9] = float("nan")
    frt.frt_matvec_nvfp4(xn, wc, wsf, ws, again)
    assert torch.isnan(again[2]).all() and torch.equal(again[[0, 1, 3]], y[[0, 1, 3]])


def test_matvec_threads():
    """Calls from several threads at once, whose kernels want different amounts of shared memory."""
    shapes = [(m, n, k) for m in (1, 16, 24) for n, k in ((64, 128), (300, 8192), (64, 2048), (8200, 2064))]

    def work(i, out):
        with torch.cuda.stream(torch.cuda.Stream()):
            for m, n, k in shapes[i:] + shapes[:i]:
                y, ref, tol = matvec_case(m, n, k, "16", seed=i)
                out.append(bool(((y.double() - ref).abs() <= tol).all()))
    outs = [[] for _ in range(4)]
    threads = [threading.Thread(target=work, args=(3 * i, o)) for i, o in enumerate(outs)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert all(len(o) == len(shapes) and all(o) for o in outs)


@pytest.mark.parametrize("dt,k", [("bf16", 144), ("f16", 512), ("f16", 4096)])
def test_matvec_wait_that_runs_out(dt, k):
    """With no polls allowed the kernel of many rows gives its waits up, writes NaN and ends; the next call is right."""
    prev = frt.frt_get_wait_polls()
    try:
        frt.frt_set_wait_polls(0)
        y, _, _ = matvec_case(40, 300, k, "16", dt=dt)
        torch.cuda.synchronize()
    finally:
        frt.frt_set_wait_polls(prev)
    assert torch.isnan(y).all()
    check_matvec(40, 300, k, "16", dt=dt)


# ------------------------------------------------------------ binding, all --
def test_binding_refusals():
    c = Case([1], [50], 4, 2, 64)
    ok = dict(q=c.q, k=c.cache.k, ksf=c.cache.ksf, v=c.cache.v, vsf=c.cache.vsf, s=c.cache.scales, n=c.kv_len,
              out=torch.empty_like(c.q))

    def call(scale=0.1, kw={}, **change):
        a = dict(ok, **change)
        frt.frt_attn_nvfp4_kvcache(a["q"], a["k"], a["ksf"], a["v"], a["vsf"], a["s"], a["n"], a["out"], scale, **kw)
    call()
    for change in (dict(q=c.q.float()), dict(out=torch.empty_like(c.q, dtype=torch.float16)), dict(n=c.kv_len.long()),
                   dict(n=c.kv_len.repeat(2)), dict(k=c.cache.k[:, :1].contiguous()), dict(ksf=c.cache.vsf[:-1]),
                   dict(s=c.cache.scales[:1]), dict(v=c.cache.v.cpu()), dict(v=c.cache.v.transpose(0, 1)),
                   dict(k=c.cache.k.to(torch.int8)), dict(scale=float("nan"))):
        with pytest.raises(frt.FrtError) as e:
            call(**change)
        assert e.value.status == frt.FRT_ERR_INVALID_ARG
    for kw in (dict(page_table=torch.zeros((2, 1), dtype=torch.int32, device=DEV), page_size=16),
               dict(page_table=torch.zeros((1, 1), dtype=torch.int32, device=DEV), page_size=6),
               dict(q_indptr=torch.zeros(1, dtype=torch.int32, device=DEV)), dict(max_q_len=0),
               dict(max_kv_len=100000, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(frt.FrtError):
            call(kw=kw)
    with pytest.raises(frt.FrtError) as e:
        g = torch.zeros((1, 1, 272), dtype=torch.float16, device=DEV)
        z = torch.zeros((4, 1, 136), dtype=torch.uint8, device=DEV)
        f = torch.zeros(frt.nvfp4_kv_sf_shape(4, 1, 272), dtype=torch.uint8, device=DEV)
        frt.frt_attn_nvfp4_kvcache(g, z, f, z, f, c.cache.scales, c.kv_len, torch.empty_like(g), 0.1)
    assert e.value.status == frt.FRT_ERR_UNSUPPORTED


def test_empty_batches():
    c = Cache(8, 2, 64, (1.0, 1.0))
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    i0 = torch.empty((0,), dtype=torch.int32, device=DEV)
    cos, sin = rope_tables(4, 64)
    frt.frt_qkv_norm_rope_nvfp4_kvcache(e.view(0, 4 * 64).expand(0, 256).repeat(1, 2).contiguous(), None, None, cos, sin, i0,
                                        e, *c.args, 4, 2, 64)
    frt.frt_attn_nvfp4_kvcache(e, *c.args, i0, torch.empty_like(e), 0.1)
    k = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    frt.frt_nvfp4_kvcache_read(*c.args, i0, k, k)
    wc, wsf, ws, _ = weights(16, 64, gen(0), "rows")
    frt.frt_matvec_nvfp4(torch.empty((0, 64), dtype=torch.float16, device=DEV), wc, wsf, ws,
                         torch.empty((0, 16), dtype=torch.float16, device=DEV))


def layer(dt, seed):
    """A decoding step of one layer: norm to NVFP4, QKV product, cache write, attention over the cache, output
    product, residual norm to FP8, gate/up product, activation to NVFP4, down product.  Returns its tensors."""
    g = gen(seed)
    t = DT[dt]
    m, d, hq, hkv, hd, inter, past = 5, 256, 8, 2, 64, 512, 70
    wts = {n: weights(o, i, g, "swizzled") for n, (o, i) in
           dict(qkv=((hq + 2 * hkv) * hd, d), o=(d, hq * hd), up=(2 * inter, d), down=(d, inter)).items()}
    x, res = randn((m, d), g).to(t), randn((m, d), g).to(t)
    cos, sin = rope_tables(128, hd)
    c = Cache(128, hkv, hd, (0.002, 0.002))
    c.set("k", randn((past, hkv, hd), g))
    c.set("v", randn((past, hkv, hd), g))
    gs, fs, as_ = (torch.tensor([v], device=DEV) for v in (0.0015, 0.01, 0.002))
    pos = torch.arange(past, past + m, dtype=torch.int32, device=DEV)
    kv_len = pos + 1
    h1, h2 = torch.empty_like(res), torch.empty_like(res)
    n4 = torch.empty((m, d // 2), dtype=torch.uint8, device=DEV)
    n4sf = torch.zeros((frt.nvfp4_sf_bytes(m, d, "swizzled"),), dtype=torch.uint8, device=DEV)
    qkv = torch.empty((m, (hq + 2 * hkv) * hd), dtype=t, device=DEV)
    q, att = (torch.empty((m, hq, hd), dtype=t, device=DEV) for _ in range(2))
    o, dn = (torch.empty((m, d), dtype=t, device=DEV) for _ in range(2))
    q8 = torch.empty((m, d), dtype=torch.uint8, device=DEV)
    gu = torch.empty((m, 2 * inter), dtype=t, device=DEV)
    a4 = torch.empty((m, inter // 2), dtype=torch.uint8, device=DEV)
    a4sf = torch.zeros((frt.nvfp4_sf_bytes(m, inter, "swizzled"),), dtype=torch.uint8, device=DEV)

    def mv(name, x, y, **kw):
        wc, wsf, ws, _ = wts[name]
        frt.frt_matvec_nvfp4(x, wc, wsf, ws, y, sf_layout="swizzled", **kw)

    def step():
        frt.frt_residual_rmsnorm_nvfp4(x, res, h1, None, n4, n4sf, gs, sf_layout="swizzled")
        mv("qkv", n4, qkv, x_format="nvfp4", x_scales=gs, x_sf=n4sf)
        frt.frt_qkv_norm_rope_nvfp4_kvcache(qkv, None, None, cos, sin, pos, q, *c.args, hq, hkv, hd)
        frt.frt_attn_nvfp4_kvcache(q, *c.args, kv_len, att, 1 / math.sqrt(hd), max_kv_len=128)
        mv("o", att.view(m, hq * hd), o)
        frt.frt_residual_rmsnorm_fp8(o, h1, h2, None, q8, static_scale=fs)
        mv("up", q8, gu, x_format="e4m3", x_scales=fs)
        frt.frt_gate_act_nvfp4(gu, a4, a4sf, as_, act="silu", sf_layout="swizzled")
        mv("down", a4, dn, x_format="nvfp4", x_scales=as_, x_sf=a4sf)
    return locals()


def unswizzle(flat, n, c):
    t = flat.view(-(-n // 128), -(-c // 4), 32, 4, 4).permute(0, 3, 2, 1, 4)
    return t.reshape(-(-n // 128) * 128, -1)[:n, :c]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_layer_step(dt):
    """Each operator of a layer's step agrees with its plain form on the inputs that the one before it left, eager
    and replayed from a graph."""
    s = layer(dt, 3)
    t = DT[dt]
    s["step"]()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            s["step"]()
        eager = {n: s[n].clone() for n in ("qkv", "q", "att", "o", "gu", "dn", "h2")}
        for n in eager:
            s[n].zero_()
        graph.replay()
        torch.cuda.synchronize()
    for n, e in eager.items():
        assert torch.equal(s[n], e), n
    m, d, inter = s["m"], s["d"], s["inter"]
    w = {n: v[3] for n, v in s["wts"].items()}

    def close(y, xv, wv):
        ref = xv @ wv.t()
        assert ((y.double() - ref).abs() <= P.matvec_bound(xv, wv, ref, t)).all()
    close(s["qkv"], P.decode(s["n4"], unswizzle(s["n4sf"], m, d // 16), s["gs"][0]), w["qkv"])
    close(s["o"], s["att"].view(m, -1).double(), w["o"])
    close(s["gu"], s["q8"].view(torch.float8_e4m3fn).double() * s["fs"].double(), w["up"])
    close(s["dn"], P.decode(s["a4"], unswizzle(s["a4sf"], m, inter // 16), s["as_"][0]), w["down"])
    k, v = s["c"].values("k"), s["c"].values("v")
    ref, vmax, smax = P.attention(s["q"], k, v, [(0, n) for n in s["kv_len"].tolist()], lambda i, p: p,
                                  1 / math.sqrt(s["hd"]), lambda h: h // 4)
    assert ((s["att"].double() - ref).abs() <= P.attention_bound(ref, vmax, smax, 128, s["hd"], t)).all()


def test_in_bounds():
    """Every operator through the bounds-checked build: no access out of range, the same bits."""
    def attn():
        outs = []
        for c in (Case([1, 3, 0, 2], [1, 50, 30, 129], 8, 2, 64, page=20), Case([2], [77], 5, 5, 80, window=20),
                  Case([1], [30001], 8, 1, 128), Case([3], [401], 6, 2, 192), Case([2], [99], 8, 1, 256),
                  Case([300], [1203], 16, 1, 64, page=4), Case([200], [903], 8, 1, 256), Case([400], [1501], 6, 2, 96)):
            outs.append(c.run())
        return outs

    def cache():
        g = gen(9)
        outs = []
        for m, hq, hkv, hd in ((7, 5, 5, 80), (33, 8, 2, 128), (3, 2, 1, 16)):
            c = Cache(m + 6, hkv, hd, (0.002, 0.002))
            cos, sin = rope_tables(64, hd)
            pos = torch.arange(m, dtype=torch.int32, device=DEV)
            q = write(c, randn((m, (hq + 2 * hkv) * hd), g).half(), None, None, cos, sin, pos, hq, pos.flip(0).contiguous())
            ko, vo = (torch.zeros((m, hkv, hd), dtype=torch.float16, device=DEV) for _ in range(2))
            frt.frt_nvfp4_kvcache_read(*c.args, pos, ko, vo)
            outs += [q, c.k, c.v, c.ksf, c.vsf, ko, vo]
        return outs

    def matvec():
        return [matvec_case(m, n, k, f, layout=lay, bias=True, seed=m)[0]
                for m, n, k, f, lay in ((1, 100, 144, "16", "rows"), (9, 33, 1040, "nvfp4", "swizzled"),
                                        (41, 300, 272, "e4m3_block", "swizzled"), (64, 17, 8192, "16", "rows"),
                                        (10, 1024, 4096, "e4m3", "rows"), (130, 50, 48, "16", "swizzled"),
                                        (20, 8210, 2064, "e4m3", "rows"), (32, 4100, 4128, "16", "swizzled"))]
    for fn in (attn, cache, matvec):
        both_builds(fn)


@pytest.mark.parametrize("hd", [64, 192, 256])
def test_attention_then_output_product(hd):
    """The two kernels that allocate tensor memory, one behind the other on a stream and on two streams at once:
    attention over many rows and the product of its output."""
    cases = [Case([200], [900], 8, 1, hd, seed=s) for s in (1, 2)]
    g = gen(hd)
    wc, wsf, ws, w = weights(512, 8 * hd, g, "rows")
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[(torch.empty_like(c.q), torch.empty((200, 512), dtype=c.q.dtype, device=DEV)) for _ in range(4)] for c in cases]
    torch.cuda.synchronize()
    for i in range(4):
        for c, st, o in zip(cases, streams, outs):
            att, y = o[i]
            frt.frt_attn_nvfp4_kvcache(c.q, *c.cache.args, c.kv_len, att, c.scale, max_kv_len=900, stream=st)
            frt.frt_matvec_nvfp4(att.view(200, 8 * hd), wc, wsf, ws, y, stream=st)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        ref, tol = c.expected()
        x = o[0][0].view(200, -1).double()
        assert ((o[0][0].double() - ref).abs() <= tol).all()
        y = x @ w.t()
        assert ((o[0][1].double() - y).abs() <= P.matvec_bound(x, w, y, c.q.dtype)).all()
        for att, again in o[1:]:
            assert torch.equal(att, o[0][0]) and torch.equal(again, o[0][1])


@pytest.mark.parametrize("m,k", [(1, 2 ** 28 + 4096), (3, 2 ** 28 + 2064), (12, 2 ** 28 + 288)])
def test_matvec_swizzled_factors_past_32_bits(m, k):
    """Swizzled factors of columns behind 2^31 bytes.  x is zero but at some columns of each quarter of K, and the
    factors of all other blocks are zeros."""
    g = gen(m)
    n = 3
    # whole blocks: the first, the last, and both sides of 2^28
    cols = torch.unique(torch.cat([torch.arange(b * 16, b * 16 + 16, device=DEV)
                                   for b in (0, 5, k // 64, k // 32, 2 ** 24 - 1, 2 ** 24, k // 16 - 2, k // 16 - 1)]))
    x = torch.zeros((m, k), dtype=torch.float16, device=DEV)
    xv = randn((m, cols.numel()), g).half()
    x[:, cols] = xv
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    atoms = -(-(k // 16) // 4)
    sf = torch.zeros((atoms * 512,), dtype=torch.uint8, device=DEV)
    blocks = cols[::16] // 16
    factors = torch.randint(40, 80, (n, blocks.numel()), generator=g, device=DEV, dtype=torch.uint8)
    for r in range(n):
        sf[blocks // 4 * 512 + r * 16 + blocks % 4] = factors[r]
    scale = torch.tensor([0.01], device=DEV)
    y = torch.empty((m, n), dtype=torch.float16, device=DEV)
    frt.frt_matvec_nvfp4(x, codes, sf, scale, y, sf_layout="swizzled")
    w = P.decode(codes[:, cols[::2] // 2], factors, scale[0])
    ref = xv.double() @ w.t()
    # products by zero leave the sums as they are: the bound counts the columns that are not
    assert ((y.double() - ref).abs() <= P.matvec_bound(xv.double(), w, ref, torch.float16)).all()


@pytest.mark.parametrize("hq,hkv,hd,q,longest", [(8, 2, 128, 1, 200000), (8, 1, 64, 1, 120000), (8, 1, 256, 41, 30000)])
def test_attn_one_workspace_for_all_lengths(hq, hkv, hd, q, longest):
    """The workspace of the longest call serves every shorter one, whose parts may be more: refused by none, and the
    same bits as with one of its own."""
    c = Case([q], [longest], hq, hkv, hd)
    ws = frt.attn_nvfp4_workspace(c.q, hkv, longest, max_q_len=q)
    for n in (longest, longest - 10584, longest * 9 // 10, longest // 2 + 1, longest // 3, longest // 10, 100):
        c.kv_len = torch.arange(n - q + 1, n + 1, dtype=torch.int32, device=DEV)
        ws.fill_(0xFF)
        assert torch.equal(c.run(workspace=ws, max_kv_len=n), c.run(max_kv_len=n)), n


@pytest.mark.parametrize("hd,power", [(64, 66), (64, 80), (128, 97), (128, -20), (256, -40)])
def test_write_far_from_one(hd, power):
    """bf16 heads whose squares are past fp32's range (above 2^64), and small ones: K's codes bit for bit."""
    hkv, m = 2, 12
    g = gen(hd + power)
    qkv = (randn((m, 3 * hkv * hd), g) * 2.0 ** power).bfloat16()
    kw = (1 + 0.2 * randn((hd,), g)).bfloat16()
    cos, sin = rope_tables(64, hd)
    c = Cache(m, hkv, hd, (0.0019, 0.002))
    pos = torch.arange(m, dtype=torch.int32, device=DEV)
    write(c, qkv, None, kw, cos, sin, pos, hkv)
    k = P.norm_rope(qkv.view(m, 3 * hkv, hd)[:, hkv:2 * hkv], kw, cos[:m], sin[:m], 1e-6).float()
    if power > 0:
        assert (k.abs().amax((1, 2)) > 1).all()  # (normed: of ordinary size)
    codes, sf = P.quantise(k, c.scales[0])
    assert torch.equal(P.sf_rows(c.ksf, m), sf) and torch.equal(c.k, codes)


@pytest.mark.parametrize("m", [4, 14, 40, 100])
@pytest.mark.parametrize("power,shrink", [(-118, 1.0), (-110, 2.0 ** -8), (-90, 2.0 ** -30), (100, 2.0 ** -30)])
def test_matvec_small_rows_and_small_weights(m, power, shrink):
    """bf16 rows and weights whose factors together leave fp32's normal range, though y does not."""
    g = gen(m + power)
    n, k = 70, 272
    wc, wsf, ws, w = weights(n, k, g, "rows")
    ws, w = ws * shrink, w * shrink
    x = (randn((m, k), g) * 2.0 ** power).bfloat16()
    y = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    frt.frt_matvec_nvfp4(x, wc, wsf, ws, y)
    ref = x.double() @ w.t()
    assert (ref.abs().median() > 2.0 ** -126).all()
    assert ((y.double() - ref).abs() <= P.matvec_bound(x.double(), w, ref, torch.bfloat16)).all()


@pytest.mark.parametrize("m", [3, 12, 40])
@pytest.mark.parametrize("beside", [-1e6, -3e38])
def test_matvec_infinity_beside_large_numbers(m, beside):
    """An infinite element of a bf16 row gives infinities of its product's sign (NaN where the weight is zero),
    whatever finite numbers stand beside it."""
    g = gen(m)
    wc, wsf, ws, w = weights(90, 256, g, "rows")
    x = randn((m, 256), g).bfloat16()
    x[1, 7] = float("inf")
    x[1, 8:40] = beside
    x[2, 200] = float("-inf")
    x[2, 190:199] = -beside
    y = torch.empty((m, 90), dtype=torch.bfloat16, device=DEV)
    frt.frt_matvec_nvfp4(x, wc, wsf, ws, y)
    ref = x.double() @ w.t()
    for r in (1, 2):
        assert torch.isinf(ref[r]).any()
        assert torch.equal(torch.isnan(y[r]), torch.isnan(ref[r]))
        fine = ~torch.isnan(ref[r])
        assert torch.equal(y[r][fine].double(), ref[r][fine])
    rest = [r for r in range(m) if r not in (1, 2)]
    assert ((y[rest].double() - ref[rest]).abs() <= P.matvec_bound(x[rest].double(), w, ref[rest], torch.bfloat16)).all()


@pytest.mark.parametrize("m,n,k,tiles", [(16, 64, 4096, False), (17, 64, 4096, True), (32, 4096, 4096, True),
                                         (32, 4112, 4096, False), (33, 4112, 4096, True)])
def test_matvec_which_kernel(m, n, k, tiles):
    """Which kernel a shape takes: the one for many rows gives up its waits without polls and writes NaN, the other
    has none."""
    prev = frt.frt_get_wait_polls()
    try:
        frt.frt_set_wait_polls(0)
        y, ref, tol = matvec_case(m, n, k, "16", dt="f16", seed=m)
        torch.cuda.synchronize()
    finally:
        frt.frt_set_wait_polls(prev)
    if tiles:
        assert torch.isnan(y).all()
    else:
        assert ((y.double() - ref).abs() <= tol).all()
    check_matvec(m, n, k, "16", dt="f16", seed=m)
