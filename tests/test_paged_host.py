"""Argument checks of the paged-cache operators (no GPU): every refusal returns its
documented status before anything is launched, and the binding refuses tensors it
cannot describe."""

import ctypes

import pytest
import torch

from rope_context_extension_b200 import jetlong as jl

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, -1, -2, -3, -4
A = 0x10000  # fake, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from rope_context_extension_b200 import build
    build.build()
    return jl.lib()


def _kv(k=A, v=A, num_pages=10, P=16, Hkv=2, D=128, page=None, row=None, head=None):
    head = D if head is None else head
    row = Hkv * D if row is None else row
    page = P * Hkv * D if page is None else page
    return jl._PagedKV(k, v, num_pages, page, row, head, P)


def _norm(lib, q=A, qs=4 * 128, k=A, ks=2 * 128, qw=A, kw=A, eps=1e-6, pos=A, qo=A, ko=A, T=3, Hq=4, Hkv=2, D=128,
          base=1e4):
    return lib.jl_qk_norm_rope(q, qs, k, ks, qw, kw, eps, pos, qo, ko, T, Hq, Hkv, D, base, None, None)


def _append(lib, q=A, qs=4 * 128, k=A, ks=2 * 128, v=A, vs=2 * 128, qw=A, kw=A, eps=1e-6, seq=A, pos=A, qo=A,
            ko=None, kv=None, bt=A, M=4, T=3, B=2, Hq=4, Hkv=2, D=128, base=1e4, cache=True):
    kv = _kv() if kv is None else kv
    return lib.jl_qk_norm_rope_append_paged(q, qs, k, ks, v, vs, qw, kw, eps, seq, pos, qo, ko,
                                            ctypes.byref(kv) if cache else None, bt, M, T, B, Hq, Hkv, D, base, None,
                                            None)


def _decode(lib, q=A, kv=None, bt=A, M=4, lens=A, o=A, lse=None, B=2, Hq=4, Hkv=2, D=128, w0=16, W=64, base=1e4,
            scale=0.0, mode=1, ws=A, ws_bytes=1 << 40):
    kv = _kv() if kv is None else kv
    return lib.jl_bifocal_decode_paged(q, ctypes.byref(kv), bt, M, lens, o, lse, B, Hq, Hkv, D, w0, W, base, scale,
                                       mode, ws, ws_bytes, None, None)


def _sparse(lib, lst=A, n=4, cnt=A, P=16):
    kv = _kv(P=P)
    return lib.jl_bifocal_decode_paged_sparse(A, ctypes.byref(kv), A, 4, A, lst, n, cnt, A, None, 2, 4, 2, 128, 16,
                                              64, 1e4, 0.0, 1, A, 0, None, None)


def _summaries(lib, kv=None, bt=A, M=4, starts=A, lens=A, max_new=1, out=A, B=2, Hkv=2, D=128, base=1e4):
    kv = _kv(v=0) if kv is None else kv
    return lib.jl_page_summaries(ctypes.byref(kv), bt, M, starts, lens, max_new, out, B, Hkv, D, base, None, None)


def _select(lib, q=A, s=A, n=10, P=16, bt=A, M=4, lens=A, sink=1, k=2, lst=A, stride=4, cnt=A, B=2, Hq=4, Hkv=2,
            D=128, w0=16, W=64, base=1e4, mode=1, ws=A, ws_bytes=1 << 40):
    return lib.jl_select_pages(q, s, n, P, bt, M, lens, sink, k, lst, stride, cnt, B, Hq, Hkv, D, w0, W, base, mode,
                               ws, ws_bytes, None, None)


def test_norm_rope_refusals(lib):
    assert _norm(lib, D=96) == UNSUPPORTED
    assert _norm(lib, Hq=3) == INVALID
    assert _norm(lib, T=0) == INVALID
    assert _norm(lib, eps=-1.0) == INVALID and _norm(lib, eps=float("nan")) == INVALID
    assert _norm(lib, base=0.0) == INVALID and _norm(lib, base=float("inf")) == INVALID
    for name in ("q", "k", "pos", "qo", "ko"):
        assert _norm(lib, **{name: None}) == INVALID, name
    assert _norm(lib, qs=4 * 128 - 8) == INVALID and _norm(lib, ks=8) == INVALID
    assert _norm(lib, qs=4 * 128 + 4) == ALIGNMENT
    for name in ("q", "k", "qw", "kw", "qo", "ko"):
        assert _norm(lib, **{name: A + 8}) == ALIGNMENT, name
    assert _norm(lib, pos=A + 2) == ALIGNMENT


def test_append_refusals(lib):
    assert _append(lib, cache=False) == INVALID
    for name in ("v", "seq", "pos", "bt", "q", "k", "qo"):
        assert _append(lib, **{name: None}) == INVALID, name
    assert _append(lib, vs=8) == INVALID and _append(lib, vs=2 * 128 + 4) == ALIGNMENT
    assert _append(lib, v=A + 8) == ALIGNMENT and _append(lib, ko=A + 8) == ALIGNMENT
    assert _append(lib, B=0) == INVALID and _append(lib, M=0) == INVALID
    assert _append(lib, kv=_kv(v=0)) == INVALID


@pytest.mark.parametrize("call", [_append, _decode, _summaries])
def test_cache_refusals(lib, call):
    assert call(lib, kv=_kv(k=0)) == INVALID
    assert call(lib, kv=_kv(num_pages=0)) == INVALID
    assert call(lib, kv=_kv(P=0)) == INVALID
    assert call(lib, kv=_kv(P=24)) == UNSUPPORTED
    assert call(lib, kv=_kv(P=2048)) == UNSUPPORTED
    assert call(lib, kv=_kv(k=A + 8)) == ALIGNMENT
    assert call(lib, kv=_kv(row=2 * 128 + 4)) == ALIGNMENT
    assert call(lib, kv=_kv(row=128)) == INVALID  # rows overlap
    assert call(lib, kv=_kv(head=64)) == INVALID  # heads overlap
    assert call(lib, kv=_kv(page=15 * 2 * 128)) == INVALID  # pages overlap
    assert call(lib, kv=_kv(page=1 << 40)) == UNSUPPORTED
    assert call(lib, M=(1 << 30) // 16 + 1) == UNSUPPORTED


def test_decode_refusals(lib):
    for name in ("q", "bt", "lens", "o"):
        assert _decode(lib, **{name: None}) == INVALID, name
    for name in ("q", "o"):
        assert _decode(lib, **{name: A + 8}) == ALIGNMENT, name
    for name in ("bt", "lens", "lse"):
        assert _decode(lib, **{name: A + 2}) == ALIGNMENT, name
    assert _decode(lib, w0=-1) == INVALID and _decode(lib, W=0) == INVALID and _decode(lib, mode=2) == INVALID
    assert _decode(lib, mode=jl.JL_PREFILL_FP16, ws=None) == WORKSPACE  # ignored, as in the other decode calls
    assert _decode(lib, mode=jl.JL_PREFILL_FP16 | jl.JL_PREFILL_KEYS_IN_KERNEL) == INVALID
    assert _decode(lib, scale=float("nan")) == INVALID
    assert _decode(lib, Hq=18) == UNSUPPORTED  # nine queries per KV head
    assert _decode(lib, B=65536) == UNSUPPORTED
    assert _decode(lib, ws=None) == WORKSPACE and _decode(lib, ws_bytes=64) == WORKSPACE
    assert _decode(lib, ws=A + 8) == ALIGNMENT
    assert _sparse(lib, lst=None) == INVALID and _sparse(lib, cnt=None) == INVALID and _sparse(lib, n=0) == INVALID
    assert _sparse(lib, n=(1 << 30) // 16 + 1) == UNSUPPORTED
    assert _sparse(lib, lst=A + 2) == ALIGNMENT
    assert _sparse(lib) == WORKSPACE


def test_summary_refusals(lib):
    for name in ("bt", "starts", "lens", "out"):
        assert _summaries(lib, **{name: None}) == INVALID, name
    assert _summaries(lib, max_new=0) == INVALID
    assert _summaries(lib, out=A + 8) == ALIGNMENT and _summaries(lib, starts=A + 1) == ALIGNMENT
    assert _summaries(lib, D=32) == UNSUPPORTED


def test_select_refusals(lib):
    for name in ("q", "s", "bt", "lens", "lst", "cnt"):
        assert _select(lib, **{name: None}) == INVALID, name
    assert _select(lib, sink=-1) == INVALID and _select(lib, k=-1) == INVALID and _select(lib, n=0) == INVALID
    assert _select(lib, P=20) == UNSUPPORTED and _select(lib, P=0) == INVALID
    assert _select(lib, stride=3) == INVALID  # 4 pages can be kept
    assert _select(lib, M=100, w0=33, sink=1, k=2, stride=6) == INVALID  # 1 + 2 + ceil(33 / 16) + 1 = 7
    assert _select(lib, Hq=18) == UNSUPPORTED
    assert _select(lib, ws=None) == WORKSPACE and _select(lib, ws_bytes=8) == WORKSPACE
    assert _select(lib, mode=2) == INVALID


def test_workspace_sizes(lib):
    # one counter, two CTA partials and twelve warp partials per CTA, whatever the batch
    small = jl.jl_decode_paged_workspace_bytes(8, 8, 64)
    assert 0 < small < jl.jl_decode_paged_workspace_bytes(32, 8, 128) == jl.jl_decode_paged_workspace_bytes(4, 1, 128)
    assert jl.jl_decode_paged_workspace_bytes(18, 2, 128) == 0
    assert jl.jl_decode_paged_workspace_bytes(3, 2, 128) == 0
    assert jl.jl_select_pages_workspace_bytes(2, 8, 1000) >= 2 * 8 * 1000 * 4
    assert jl.jl_select_pages_workspace_bytes(0, 8, 10) == 0


def test_binding_refuses_host_tensors():
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    k = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        jl.jl_qk_norm_rope(q, k, None, None, pos, q, k, eps=1e-6, rope_base=1e4)
