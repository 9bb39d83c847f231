"""Host-side refusals of the NVFP4 operators: the C entry points reject bad
arguments before any CUDA call (fake, never-dereferenced pointers), and the
binding rejects tensors that do not fit."""
import os

import pytest
import torch

import memory_bound_non_b200 as frt

A = 0x100000          # a 256-byte aligned fake device address (never dereferenced)
INV, UNSUP, OK = frt.FRT_ERR_INVALID_ARG, frt.FRT_ERR_UNSUPPORTED, frt.FRT_OK


def write_call(M=4, Hq=8, Hkv=2, hd=128, qkv=A, qw=None, kw=None, cos=A, sin=A, pos=A, slots=None, q=A, kc=A, ks=A, vc=A,
               vs=A, gs=A, status=None, max_pos=64, cap=64, dt=1):
    return frt.load().frt_qkv_norm_rope_nvfp4_kvcache(qkv, qw, kw, cos, sin, pos, slots, q, kc, ks, vc, vs, gs, status, M,
                                                      Hq, Hkv, hd, max_pos, cap, 1e-6, dt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INV), (dict(Hq=0), INV), (dict(Hkv=0), INV), (dict(Hq=6, Hkv=4), INV), (dict(hd=0), INV),
    (dict(hd=24), INV), (dict(hd=272), UNSUP), (dict(max_pos=0), INV), (dict(cap=0), INV), (dict(dt=2), INV),
    (dict(qkv=None), INV), (dict(qkv=A + 8), INV), (dict(cos=None), INV), (dict(sin=A + 4), INV), (dict(pos=None), INV),
    (dict(pos=A + 2), INV), (dict(slots=A + 1), INV), (dict(q=None), INV), (dict(q=A + 8), INV), (dict(kc=None), INV),
    (dict(ks=A + 8), INV), (dict(vc=A + 8), INV), (dict(vs=None), INV), (dict(gs=None), INV), (dict(gs=A + 2), INV),
    (dict(qw=A + 8), INV), (dict(kw=A + 2), INV), (dict(status=A + 2), INV), (dict(M=0), OK),
    (dict(M=0, qkv=None, kc=None, gs=None), OK), (dict(M=0, hd=24), INV), (dict(M=0, hd=272), UNSUP),
])
def test_write_host_validation(kw, want):
    assert write_call(**kw) == want


def read_call(n=4, Hkv=2, hd=128, cap=64, kc=A, ks=A, vc=A, vs=A, gs=A, slots=None, ko=A, vo=A, status=None, dt=1):
    return frt.load().frt_nvfp4_kvcache_read(kc, ks, vc, vs, gs, slots, ko, vo, status, n, Hkv, hd, cap, dt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INV), (dict(Hkv=0), INV), (dict(hd=8), INV), (dict(hd=512), UNSUP), (dict(cap=0), INV), (dict(dt=7), INV),
    (dict(kc=None), INV), (dict(vs=A + 4), INV), (dict(gs=None), INV), (dict(slots=A + 2), INV), (dict(ko=None), INV),
    (dict(vo=A + 8), INV), (dict(status=A + 3), INV), (dict(n=0), OK), (dict(n=0, kc=None, ko=None), OK),
])
def test_read_host_validation(kw, want):
    assert read_call(**kw) == want


def attn_call(M=4, n_seqs=1, Hq=8, Hkv=2, hd=128, cap=64, ps=0, mp=0, mq=4, mk=64, window=0, scale=0.1, dt=1, q=A, kc=A,
              ks=A, vc=A, vs=A, gs=A, kl=A, ip=None, pt=None, out=A, ws=None, wb=0, status=None):
    return frt.load().frt_attn_nvfp4_kvcache(q, kc, ks, vc, vs, gs, kl, ip, pt, out, ws, wb, status, M, n_seqs, Hq, Hkv, hd,
                                             cap, ps, mp, mq, mk, window, scale, dt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INV), (dict(n_seqs=0), INV), (dict(n_seqs=2), INV), (dict(Hq=0), INV), (dict(Hq=9), INV),
    (dict(Hkv=0), INV), (dict(hd=0), INV), (dict(hd=40), INV), (dict(hd=272), UNSUP), (dict(cap=0), INV), (dict(mq=0), INV),
    (dict(mk=-1), INV), (dict(mk=0x7FFFFF01), UNSUP), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(dt=3), INV), (dict(q=None), INV), (dict(q=A + 8), INV), (dict(kc=A + 4), INV), (dict(ks=None), INV),
    (dict(vc=None), INV), (dict(vs=A + 8), INV), (dict(gs=A + 1), INV), (dict(kl=None), INV), (dict(kl=A + 2), INV),
    (dict(ip=A + 2), INV), (dict(out=None), INV), (dict(out=A + 8), INV), (dict(status=A + 2), INV),
    (dict(pt=A, ps=0, mp=1), INV), (dict(pt=A, ps=6, mp=1), INV), (dict(pt=A, ps=4, mp=-1), INV),
    (dict(pt=A + 2, ps=4, mp=1), INV), (dict(ip=A, n_seqs=65536), UNSUP), (dict(M=0), OK),
    (dict(M=0, q=None, kl=None, out=None), OK), (dict(M=0, n_seqs=3), INV),
    # a call that needs a workspace: none, too small, misaligned
    (dict(M=1, mq=1, mk=100000, cap=100000), INV), (dict(M=1, mq=1, mk=100000, cap=100000, ws=A, wb=16), INV),
    (dict(M=1, mq=1, mk=100000, cap=100000, ws=A + 8, wb=1 << 30), INV),
])
def test_attn_host_validation(kw, want):
    assert attn_call(**kw) == want


def test_attn_workspace_bytes():
    W = frt.load().frt_attn_nvfp4_workspace_bytes
    assert W(1, 1, 8, 2, 128, 1, 0) == 0 and W(1, 1, 8, 2, 128, 1, 64) == 0
    assert W(-1, 1, 8, 2, 128, 1, 64) == 0 and W(1, 1, 7, 2, 128, 1, 64) == 0    # refused by the call itself
    long = W(1, 1, 8, 2, 128, 1, 200000)
    assert long > 0 and long % 4 == 0
    # it bounds every shorter call of the same shape (a serving program keeps one)
    assert all(W(1, 1, 8, 2, 128, 1, n) <= long for n in (1, 100, 5000, 50000, 199999))


def matvec_call(M=4, N=64, K=128, x=A, xs=None, xsf=None, w=A, wsf=A, ws=A, bias=None, y=A, xfmt=0, lay=0, dt=1):
    return frt.load().frt_matvec_nvfp4(x, xs, xsf, w, wsf, ws, bias, y, M, N, K, xfmt, lay, dt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(K=24), INV), (dict(xfmt=4), INV), (dict(xfmt=-1), INV),
    (dict(lay=2), INV), (dict(dt=2), INV), (dict(x=None), INV), (dict(x=A + 8), INV), (dict(w=A + 8), INV),
    (dict(wsf=None), INV), (dict(wsf=A + 4), INV), (dict(ws=None), INV), (dict(ws=A + 2), INV), (dict(y=None), INV),
    (dict(y=A + 1), INV), (dict(bias=A + 1), INV), (dict(xfmt=1), INV), (dict(xfmt=2), INV), (dict(xfmt=2, xs=A + 2), INV),
    (dict(xfmt=3, xs=A), INV), (dict(xfmt=3, xs=A, xsf=A + 8), INV), (dict(M=0), OK), (dict(M=0, x=None, y=None), OK),
    (dict(M=0, K=8), INV), (dict(N=2**31 - 1), UNSUP), (dict(K=2**31 - 16), UNSUP),
])
def test_matvec_host_validation(kw, want):
    assert matvec_call(**kw) == want


def test_binding_rejects_host_tensors():
    t = torch.zeros((4, 64), dtype=torch.bfloat16)
    u = torch.zeros((4, 32), dtype=torch.uint8)
    with pytest.raises(frt.FrtError) as e:
        frt.frt_matvec_nvfp4(t, u, u, torch.ones(1), t)
    assert e.value.status == INV and "CUDA" in str(e.value)
    with pytest.raises(frt.FrtError):
        frt.frt_matvec_nvfp4(t, u, u, torch.ones(1), t, x_format="int8")
    with pytest.raises(frt.FrtError):
        frt.frt_nvfp4_kvcache_read(u, u, u, u, torch.ones(2), None, t, t)
    with pytest.raises(frt.FrtError):
        frt.frt_qkv_norm_rope_nvfp4_kvcache(t, None, None, t, t, u, t, u, u, u, u, t, 1, 1, 64)
    with pytest.raises(frt.FrtError):
        frt.frt_attn_nvfp4_kvcache(t, u, u, u, u, t, u, t, 0.1)
    with pytest.raises(frt.FrtError):
        frt.frt_matvec_nvfp4(None, u, u, torch.ones(1), t)


def test_kv_sf_shape():
    assert frt.nvfp4_kv_sf_shape(1, 2, 64) == (1, 2, 4, 4)
    assert frt.nvfp4_kv_sf_shape(9, 1, 256) == (3, 1, 16, 4)


def _kernel_text(source):
    """The text of the one kernel of a source file that uses tensor memory."""
    root = os.path.join(os.path.dirname(frt.__file__), "csrc", source)
    with open(root) as f:
        text = f.read()
    return text[text.index("tiles_kernel("):text.index("tc_free<")]


@pytest.mark.parametrize("source", ["attn_nvfp4_tiles.cu", "matvec_nvfp4_tiles.cu"])
def test_tensor_memory_is_never_held_across_a_dependency(source):
    """An allocation of tensor memory blocks without a bound while an SM's columns are taken.  A kernel that held
    columns while it waits for the grid before it, or let the next grid in before it has its own, could block that
    grid for good: the order in the source is wait, allocate, release."""
    body = _kernel_text(source)
    assert "pdl_enter" not in body  # waits and releases at once
    assert body.index("pdl_wait();") < body.index("tc_alloc<") < body.index("pdl_release();")
    assert body.index("tc_alloc<") < body.index("__syncthreads();", body.index("tc_alloc<")) < body.index("pdl_release();")


@pytest.mark.parametrize("m", [2 ** 31 - 65535, 2 ** 31 - 128, 2 ** 31 - 1])
def test_matvec_refuses_rows_at_the_end_of_32_bits(m):
    """The rows are taken 128 at a time by a 32-bit index, which must not run past its end."""
    assert matvec_call(M=m) == UNSUP


@pytest.mark.parametrize("hq,hkv,hd,n_seqs,q", [(8, 2, 128, 1, 1), (8, 2, 128, 3, 1), (32, 8, 128, 1, 1), (8, 1, 64, 1, 1),
                                                (8, 8, 256, 1, 1), (40, 2, 128, 1, 1), (8, 1, 256, 1, 10), (8, 1, 256, 1, 41),
                                                (16, 8, 128, 1, 41), (4, 2, 80, 2, 5), (16, 1, 64, 1, 300), (8, 2, 192, 1, 17)])
def test_attn_workspace_never_falls_with_the_length(hq, hkv, hd, n_seqs, q):
    """A workspace of a program's longest call serves its shorter ones: all tile counts, and more tokens."""
    W = frt.load().frt_attn_nvfp4_workspace_bytes
    last = 0
    for n in list(range(0, 270000, 32)) + [2 ** 20, 2 ** 24, 2 ** 31 - 256]:
        size = W(q * n_seqs, n_seqs, hq, hkv, hd, q, n)
        assert size >= last, n
        last = size
        if n % 4096 == 0:
            assert W(1, n_seqs, hq, hkv, hd, q, n) <= size <= W(2 * q * n_seqs, n_seqs, hq, hkv, hd, q, n)


def test_marshalling_is_built_again_for_another_torch(monkeypatch, tmp_path):
    """_marshal.so holds torch's own layouts: one built against another torch is stale, and is not loaded."""
    from memory_bound_non_b200 import build as B
    B.build_marshal()
    assert not B.marshal_stale()
    tag = tmp_path / "tag"
    monkeypatch.setattr(B, "MARSHAL_TAG", str(tag))
    assert B.marshal_stale()
    tag.write_text("torch 1.0, cpython-312")
    assert B.marshal_stale()
    monkeypatch.setattr(frt, "_native", None)
    monkeypatch.setattr(torch, "__version__", "1.0")
    with pytest.raises(frt.FrtError, match="built against"):
        frt._entry("frt_matvec_nvfp4")
