"""The paged-cache operators on the GPU against plain fp64 forms, at the sizes, masks,
strides and paddings where they can go wrong (tests/paged_helpers.py derives the bounds)."""

import numpy as np
import pytest
import torch

from oracle import jetlong_oracle as jo
from rope_context_extension_b200 import jetlong as jl
from tests import paged_helpers as ph

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF16 = torch.bfloat16
MODES = {jo.MODE_NONE: jl.JL_QSHIFT_NONE, jo.MODE_SELF_EXTEND: jl.JL_QSHIFT_SELF_EXTEND}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from rope_context_extension_b200 import build
    build.build()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(BF16).to(DEV)


def _pool(g, n, P, Hkv, D, layout="rows", fill=None):
    """K and V page pools as [n, P, Hkv, D] views of the given memory order."""
    shape = {"rows": (2, n, P, Hkv, D), "heads": (2, n, Hkv, P, D), "interleaved": (n, 2, P, Hkv, D),
             "beside": (n, P, 2, Hkv, D)}[layout]
    x = _randn(g, *shape) if fill is None else torch.full(shape, fill, dtype=BF16, device=DEV)
    if layout == "rows":
        return x[0], x[1]
    if layout == "heads":
        return x[0].permute(0, 2, 1, 3), x[1].permute(0, 2, 1, 3)
    if layout == "interleaved":
        return x[:, 0], x[:, 1]
    return x[:, :, 0], x[:, :, 1]


def _table(g, lens, P, num_pages, width=None):
    """Block table with pages in a random order and junk behind each sequence's last page."""
    need = [-(-n // P) for n in lens]
    width = max(1, max(need)) if width is None else width
    perm = torch.randperm(num_pages, generator=g).tolist()
    junk = [-1, 1 << 30, -(1 << 31)]
    rows, at = [], 0
    for i, n in enumerate(need):
        rows.append(perm[at:at + n] + [junk[i % 3]] * (width - n))
        at += n
    return _i32(rows)


def _keys(pages, table, b, L, g):
    """fp64 rows 0 .. L - 1 of one KV head of a sequence."""
    P = pages.shape[1]
    ids = table[b, :-(-L // P)].long()
    return _f64(pages[ids, :, g].reshape(-1, pages.shape[3])[:L])


def _stale(k, v, table, lens, value):
    """Every row that no sequence holds becomes `value`."""
    P = k.shape[1]
    used = torch.zeros(k.shape[0], P, dtype=torch.bool, device=DEV)
    for b, n in enumerate(lens):
        for p in range(-(-n // P)):
            used[int(table[b, p]), :min(P, n - p * P)] = True
    k[~used] = value
    v[~used] = value


def _ws(Hq, Hkv, D):
    return torch.zeros(jl.jl_decode_paged_workspace_bytes(Hq, Hkv, D), dtype=torch.uint8, device=DEV)


def _check_decode(o, lse, q, k, v, table, lens, w0, W, base, mode=jo.MODE_SELF_EXTEND, scale=None, lists=None,
                  rows=None):
    B, Hq, D = q.shape
    Hkv, P = k.shape[2], k.shape[1]
    r = Hq // Hkv
    for b, L in enumerate(lens):
        if rows is not None and b not in rows:
            continue
        for g in range(Hkv):
            pos = np.arange(L)
            if lists is not None:
                pos = np.concatenate([np.arange(p * P, min(L, (p + 1) * P)) for p in lists[b][g]] + [[]]).astype(int)
            kk, vv = _keys(k, table, b, L, g)[pos], _keys(v, table, b, L, g)[pos]
            hs = slice(g * r, (g + 1) * r)
            want_o, want_l, err = ph.decode_rows(_f64(q[b, hs]), kk, vv, pos, L, w0, W, base, mode, scale)
            ph.assert_decode(_f64(o[b, hs]), _f64(lse[b, hs]), want_o, want_l, err,
                             np.abs(vv).max() if len(vv) else 0.0, f"sequence {b} ({L}), head {g}")


# ---------------------------------------------------------------- norms + rotation
@pytest.mark.parametrize("T,Hq,Hkv,D,norm", [(1, 32, 8, 128, "both"), (7, 2, 1, 64, "both"), (130, 5, 5, 128, "q"),
                                             (33, 14, 2, 64, "k"), (9, 8, 1, 128, "none"), (600, 16, 8, 128, "both")])
def test_norm_rope(T, Hq, Hkv, D, norm):
    g = torch.Generator().manual_seed(T)
    x = _randn(g, T, Hq + 2 * Hkv, D, scale=3.0)  # a fused projection's rows
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    qw = _randn(g, D) if norm in ("both", "q") else None
    kw = _randn(g, D) if norm in ("both", "k") else None
    pos = torch.randint(0, 1 << 20, (T,), generator=g)
    pos[0] = 0
    pos[-1] = (1 << 31) - 1
    if T > 4:
        pos[3] = -1
    qo = torch.full((T, Hq, D), 7.0, dtype=BF16, device=DEV)
    ko = torch.full((T, Hkv, D), 7.0, dtype=BF16, device=DEV)
    err = _i32([0])
    jl.jl_qk_norm_rope(q, k, qw, kw, pos.to(torch.int32).to(DEV), qo, ko, eps=ph.EPS, rope_base=1e6, dev_error=err)
    assert int(err) == 0
    for src, w, out in ((q, qw, qo), (k, kw, ko)):
        want = ph.norm_rope(_f64(src), None if w is None else _f64(w), pos.numpy(), 1e6)
        tol = ph.norm_rope_tol(want) + (2.0 ** -20 * np.abs(want).max())  # the angle at 2^31 in fp64 on both sides
        live = pos.numpy() != -1
        assert np.all(np.abs(_f64(out) - want)[live] <= tol[live])
        assert np.all(_f64(out)[~live] == 7.0)


@pytest.mark.parametrize("T,Hq,Hkv,D", [(9001, 3, 1, 64), (5000, 40, 8, 128)])
def test_norm_rope_many_tokens(T, Hq, Hkv, D):
    g = torch.Generator().manual_seed(T)
    q, k = _randn(g, T, Hq, D), _randn(g, T, Hkv, D)
    w = _randn(g, D)
    pos = torch.arange(T)
    pos[::7] = -1
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    jl.jl_qk_norm_rope(q, k, w, None, pos.to(torch.int32).to(DEV), qo, ko, eps=ph.EPS, rope_base=1e6)
    for src, ww, out in ((q, w, qo), (k, None, ko)):
        want = ph.norm_rope(_f64(src), None if ww is None else _f64(ww), pos.numpy(), 1e6)
        want[::7] = 7.0
        assert np.all(np.abs(_f64(out) - want) <= ph.norm_rope_tol(want))


def test_norm_rope_of_zero_rows_and_in_place():
    g = torch.Generator().manual_seed(2)
    q, k = _randn(g, 5, 4, 128), _randn(g, 5, 2, 128)
    q[1] = 0
    w = _randn(g, 128)
    pos = _i32([5, 6, 7, 8, 9])
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    jl.jl_qk_norm_rope(q, k, w, w, pos, qo, ko, eps=ph.EPS, rope_base=1e4)
    assert torch.all(qo[1] == 0) and torch.isfinite(qo.float()).all()
    q2, k2 = q.clone(), k.clone()
    jl.jl_qk_norm_rope(q2, k2, w, w, pos, q2, k2, eps=ph.EPS, rope_base=1e4)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


@pytest.mark.parametrize("layout", ["rows", "heads", "interleaved", "beside"])
@pytest.mark.parametrize("D,P,Hq,Hkv", [(128, 16, 8, 2), (64, 48, 3, 3)])
def test_append_writes_its_rows_and_no_others(layout, D, P, Hq, Hkv):
    g = torch.Generator().manual_seed(P)
    lens, n_pages = [3 * P + 5, 1, 2 * P], 9
    k, v = _pool(g, n_pages, P, Hkv, D, layout)
    k0, v0 = k.clone(), v.clone()
    table = _table(g, lens, P, n_pages)
    # a chunk of sequence 0 across a page border, one token each of the others, two padded tokens
    tok = [(0, p) for p in range(P - 3, 2 * P + 2)] + [(1, 0), (2, 2 * P - 1), (7, -1), (-5, -1)]
    T = len(tok)
    q, kr, vr = _randn(g, T, Hq, D), _randn(g, T, Hkv, D), _randn(g, T, Hkv, D)
    w = _randn(g, D)
    qo = torch.full((T, Hq, D), 7.0, dtype=BF16, device=DEV)
    ko = torch.full((T, Hkv, D), 7.0, dtype=BF16, device=DEV)
    err = _i32([0])
    pos = _i32([p for _, p in tok])
    jl.jl_qk_norm_rope_append_paged(q, kr, vr, w, w, _i32([s for s, _ in tok]), pos, table, qo, k, v, eps=ph.EPS,
                                    rope_base=1e4, k_out=ko, dev_error=err)
    assert int(err) == 0
    q2, k2 = torch.full_like(qo, 7.0), torch.full_like(ko, 7.0)
    jl.jl_qk_norm_rope(q, kr, w, w, pos, q2, k2, eps=ph.EPS, rope_base=1e4)
    assert torch.equal(qo, q2) and torch.equal(ko, k2)
    for t, (s, p) in enumerate(tok):
        if p >= 0:
            k0[int(table[s, p // P]), p % P] = ko[t]
            v0[int(table[s, p // P]), p % P] = vr[t]
    assert torch.equal(k, k0) and torch.equal(v, v0)


def test_append_leaves_out_what_is_out_of_range():
    g = torch.Generator().manual_seed(4)
    P, Hkv, D = 16, 2, 64
    k, v = _pool(g, 4, P, Hkv, D)
    k0, v0 = k.clone(), v.clone()
    table = _i32([[0, 1], [2, 99]])
    bad = [(2, 0), (-1, 3), (0, 32), (0, -2), (1, 20)]
    for s, p in bad:
        q, kr, vr = _randn(g, 1, 2, D), _randn(g, 1, Hkv, D), _randn(g, 1, Hkv, D)
        qo = torch.full((1, 2, D), 7.0, dtype=BF16, device=DEV)
        err = _i32([0])
        jl.jl_qk_norm_rope_append_paged(q, kr, vr, None, None, _i32([s]), _i32([p]), table, qo, k, v, eps=0.0,
                                        rope_base=1e4, dev_error=err)
        assert int(err) == 2, (s, p)
        assert torch.all(qo == 7.0)
    assert torch.equal(k, k0) and torch.equal(v, v0)


# ---------------------------------------------------------------- paged decode
@pytest.mark.parametrize("lens,Hq,Hkv,D,P,w0,W,base", [
    ([1], 1, 1, 64, 16, 0, 1, 1e4),
    ([1], 8, 1, 128, 16, 4, 4, 1e4),
    ([2, 0, 15, 16, 17], 4, 2, 128, 16, 0, 4, 1e4),
    ([777], 2, 1, 64, 16, 32, 128, 1e4),
    ([33, 1000, 0, 0, 257], 7, 1, 128, 48, 10, 300, 1e6),
    ([5000, 3], 10, 2, 64, 64, 100, 700, 1e4),
    ([2047, 4096], 16, 8, 128, 32, 4096, 1024, 1e6),
    ([640, 641, 0, 1300], 24, 8, 128, 128, 200, 400, 1e6),
    ([9000], 32, 4, 128, 16, 1, 400, 1e6),  # G 23
    ([3000, 100], 6, 2, 128, 1024, 64, 1000, 1e6),
])
@pytest.mark.parametrize("mode", [jo.MODE_SELF_EXTEND, jo.MODE_NONE])
def test_decode(lens, Hq, Hkv, D, P, w0, W, base, mode):
    g = torch.Generator().manual_seed(sum(lens))
    n = sum(-(-x // P) for x in lens) + 2
    k, v = _pool(g, n, P, Hkv, D)
    table = _table(g, lens, P, n)
    _stale(k, v, table, lens, float("nan"))  # what no sequence holds must not matter
    q = _randn(g, len(lens), Hq, D)
    o = torch.full_like(q, 7.0)
    lse = torch.full((len(lens), Hq), 7.0, device=DEV)
    err, ws = _i32([0]), _ws(Hq, Hkv, D)
    for _ in range(2):  # the second call on the counters that the first left
        jl.jl_bifocal_decode_paged(q, k, v, table, _i32(lens), o, lse, w0=w0, w_pretrained=W, rope_base=base,
                                   mode=MODES[mode], workspace=ws, dev_error=err)
    assert int(err) == 0
    _check_decode(o, lse, q, k, v, table, lens, w0, W, base, mode)


@pytest.mark.parametrize("r", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("layout", ["rows", "heads", "interleaved", "beside"])
def test_decode_ratios_and_layouts(r, layout):
    g = torch.Generator().manual_seed(r)
    lens, P, Hkv, D = [1200, 77], (32, 16, 128, 1024)[r % 4], 3, 128
    n = sum(-(-x // P) for x in lens) + 1
    k, v = _pool(g, n, P, Hkv, D, layout)
    table = _table(g, lens, P, n)
    q = _randn(g, 2, Hkv * r, D)
    o, lse = torch.empty_like(q), torch.empty(2, Hkv * r, device=DEV)
    jl.jl_bifocal_decode_paged(q, k, v, table, _i32(lens), o, lse, w0=50, w_pretrained=400, rope_base=1e6,
                               softmax_scale=0.2, workspace=_ws(Hkv * r, Hkv, D))
    _check_decode(o, lse, q, k, v, table, lens, 50, 400, 1e6, scale=0.2)


def test_sequences_that_share_their_first_pages():
    g = torch.Generator().manual_seed(17)
    lens, P, Hq, Hkv, D = [400, 333, 320], 16, 8, 2, 128
    k, v = _pool(g, 70, P, Hkv, D)
    table = _table(g, lens, P, 70, width=25)
    table[1:, :20] = table[0, :20]  # 320 positions in common
    q = _randn(g, 3, Hq, D)
    o, lse = torch.empty_like(q), torch.empty(3, Hq, device=DEV)
    jl.jl_bifocal_decode_paged(q, k, v, table, _i32(lens), o, lse, w0=30, w_pretrained=100, rope_base=1e6,
                               workspace=_ws(Hq, Hkv, D))
    _check_decode(o, lse, q, k, v, table, lens, 30, 100, 1e6)
    s = torch.zeros(70, Hkv, D, dtype=BF16, device=DEV)
    jl.jl_page_summaries(k, table, _i32([0, 0, 0]), _i32(lens), s, max_new=400, rope_base=1e6)
    alone = torch.zeros_like(s)
    for b in range(3):
        jl.jl_page_summaries(k, table[b:b + 1], _i32([0]), _i32(lens[b:b + 1]), alone, max_new=400, rope_base=1e6)
    assert torch.equal(s, alone)


def test_decode_with_outlier_keys_and_one_dominant_key():
    g = torch.Generator().manual_seed(9)
    lens, P, Hq, Hkv, D = [3000], 16, 8, 2, 128
    k, v = _pool(g, 200, P, Hkv, D)
    table = _table(g, lens, P, 200)
    k[torch.rand(200, P, generator=g).to(DEV) < 0.01] *= 8
    q = _randn(g, 1, Hq, D)
    k[int(table[0, 3]), 5, 0] = q[0, 0] * 2  # the row's softmax is this key's
    o, lse = torch.empty_like(q), torch.empty(1, Hq, device=DEV)
    jl.jl_bifocal_decode_paged(q, k, v, table, _i32(lens), o, lse, w0=100, w_pretrained=1000, rope_base=1e6,
                               workspace=_ws(Hq, Hkv, D))
    _check_decode(o, lse, q, k, v, table, lens, 100, 1000, 1e6)


@pytest.mark.parametrize("qs,ks,share", [(1e-4, 1e4, 1.0), (1e4, 1e-4, 1.0), (1e-2, 2000.0, 0.02), (5e-3, 800.0, 1.0),
                                         (3000.0, 1e-3, 1.0), (1e-9, 1e9, 0.3), (1e-30, 1e30, 1.0)])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 128), (10, 2, 64)])
def test_decode_operands_beyond_half_range(qs, ks, share, Hq, Hkv, D):
    # queries and keys whose products are ordinary and whose own sizes are not: entries above
    # fp16's range in all keys, in some keys of a unit, in the queries, and just below it.  (The
    # smaller side of those that stay in range is above 1e-3, where the bound of 2^-17 holds.)
    g = torch.Generator().manual_seed(int(share * 100) + D)
    lens, P = [1003, 517, 16], 32
    k, v = _pool(g, 60, P, Hkv, D)
    table = _table(g, lens, P, 60)
    k[torch.rand(60, P, generator=g).to(DEV) < share] *= ks
    _stale(k, v, table, lens, float("nan"))
    q = _randn(g, 3, Hq, D) * qs
    o, lse = torch.empty_like(q), torch.empty(3, Hq, device=DEV)
    for w0 in (0, 45):  # 45: units on the band's edge
        jl.jl_bifocal_decode_paged(q, k, v, table, _i32(lens), o, lse, w0=w0, w_pretrained=150, rope_base=1e4,
                                   workspace=_ws(Hq, Hkv, D))
        _check_decode(o, lse, q, k, v, table, lens, w0, 150, 1e4)


@pytest.mark.parametrize("B,Hq,Hkv,D,top,P", [(300, 4, 2, 64, 60, 16), (300, 2, 2, 128, 400, 32), (40, 24, 3, 64, 130, 16),
                                              (700, 1, 1, 64, 17, 16), (97, 32, 8, 128, 300, 48)])
def test_decode_many_short_sequences(B, Hq, Hkv, D, top, P):
    # more items than the work line's runs; sequences that warps take whole, and a mix
    g = torch.Generator().manual_seed(B + top)
    lens = torch.randint(0, top + 1, (B,), generator=g).tolist()
    lens[0], lens[-1] = top, 0
    n = sum(-(-x // P) for x in lens) + 1
    k, v = _pool(g, n, P, Hkv, D)
    table = _table(g, lens, P, n)
    _stale(k, v, table, lens, float("inf"))
    q = _randn(g, B, Hq, D)
    o, lse = torch.full_like(q, 7.0), torch.full((B, Hq), 7.0, device=DEV)
    err, ws = _i32([0]), _ws(Hq, Hkv, D)
    jl.jl_bifocal_decode_paged(q, k, v, table, _i32(lens), o, lse, w0=9, w_pretrained=30, rope_base=1e4, workspace=ws,
                               dev_error=err)
    assert int(err) == 0
    _check_decode(o, lse, q, k, v, table, lens, 9, 30, 1e4)
    assert torch.all(ws[:4 * 148] == 0)  # the tickets are back at zero


@pytest.mark.parametrize("W", [1, 2, 37, 1500, 2999])
def test_decode_group_sizes(W):
    # G = 3000, 1500, 82, 2, 2: how far the keys' turns carry from one unit to the next
    g = torch.Generator().manual_seed(W)
    lens, P, Hq, Hkv, D = [3000, 2999], 32, 4, 1, 128
    k, v = _pool(g, 200, P, Hkv, D)
    table = _table(g, lens, P, 200)
    q = _randn(g, 2, Hq, D)
    o, lse = torch.empty_like(q), torch.empty(2, Hq, device=DEV)
    jl.jl_bifocal_decode_paged(q, k, v, table, _i32(lens), o, lse, w0=33, w_pretrained=W, rope_base=1e6,
                               workspace=_ws(Hq, Hkv, D))
    _check_decode(o, lse, q, k, v, table, lens, 33, W, 1e6)


@pytest.mark.parametrize("at", [5, 990])  # a remote key, a local one
def test_a_nan_key_reaches_its_own_head_only(at):
    g = torch.Generator().manual_seed(at)
    lens, P, Hq, Hkv, D = [1000, 1000], 16, 8, 2, 128
    k, v = _pool(g, 130, P, Hkv, D)
    table = _table(g, lens, P, 130)
    k[int(table[0, at // P]), at % P, 1, 7] = float("nan")
    q = _randn(g, 2, Hq, D)
    o, lse = torch.empty_like(q), torch.empty(2, Hq, device=DEV)
    jl.jl_bifocal_decode_paged(q, k, v, table, _i32(lens), o, lse, w0=100, w_pretrained=300, rope_base=1e6,
                               workspace=_ws(Hq, Hkv, D))
    assert torch.isnan(o[0, 4:]).all() and torch.isnan(lse[0, 4:]).all()
    assert torch.isfinite(o[0, :4]).all() and torch.isfinite(o[1]).all() and torch.isfinite(lse[1]).all()


def test_decode_equals_the_contiguous_varlen_decode():
    from rope_context_extension_b200 import synthetic
    lens = [700, 1999, 2001, 4000]
    q, kc, vc = (t.to(DEV) for t in synthetic.decode_inputs(4, 4096, 8, 2, 128, seed=21, outlier_frac=0.01))
    o1, l1 = torch.empty_like(q), torch.empty(4, 8, device=DEV)
    jl.jl_bifocal_decode_varlen(q, kc, vc, o1, l1, _i32(lens), max_len=4096, w0=150, w_pretrained=1000, rope_base=1e6,
                                workspace=torch.zeros(jl.jl_decode_workspace_bytes(4, 4096, 8, 2, 128),
                                                      dtype=torch.uint8, device=DEV))
    table = torch.arange(4 * 64, dtype=torch.int32, device=DEV).view(4, 64)  # the same cache as pages of 64
    o2, l2 = torch.empty_like(q), torch.empty(4, 8, device=DEV)
    jl.jl_bifocal_decode_paged(q, kc.view(256, 64, 2, 128), vc.view(256, 64, 2, 128), table, _i32(lens), o2, l2,
                               w0=150, w_pretrained=1000, rope_base=1e6, workspace=_ws(8, 2, 128))
    # both carry scores to about 2^-16; the varlen decode's probabilities are bf16 (2^-8 of a value)
    assert (l1 - l2).abs().max() <= 1e-3
    assert (o1.float() - o2.float()).abs().max() <= 2 * 2.0 ** -8 * o1.float().abs().max() + 1e-3


def test_decode_long_offsets():
    # pages whose elements lie behind 2^31 elements and 2^32 bytes of the pool
    P, Hkv, D = 64, 8, 128
    n = (1 << 31) // (P * Hkv * D) + 40
    k = torch.zeros(n, P, Hkv, D, dtype=BF16, device=DEV)
    v = torch.zeros(n, P, Hkv, D, dtype=BF16, device=DEV)
    g = torch.Generator().manual_seed(3)
    lens = [P * 20 + 9]
    table = torch.arange(n - 1, n - 22, -1, dtype=torch.int32, device=DEV)[None].contiguous()
    k[table[0].long()] = _randn(g, 21, P, Hkv, D)
    q = _randn(g, 1, 8, D)
    w = _randn(g, D)
    qo = torch.empty_like(q)
    # the newest token is appended there too, and its page summarised
    kr, vr = _randn(g, 1, Hkv, D), _randn(g, 1, Hkv, D)
    jl.jl_qk_norm_rope_append_paged(q, kr, vr, w, w, _i32([0]), _i32([lens[0] - 1]), table, qo, k, v, eps=ph.EPS,
                                    rope_base=1e6)
    assert torch.equal(v[int(table[0, 20]), 8], vr[0])
    o, lse = torch.empty_like(q), torch.empty(1, 8, device=DEV)
    jl.jl_bifocal_decode_paged(qo, k, v, table, _i32(lens), o, lse, w0=64, w_pretrained=500, rope_base=1e6,
                               workspace=_ws(8, Hkv, D))
    _check_decode(o, lse, qo, k, v, table, lens, 64, 500, 1e6)
    s = torch.zeros(n, Hkv, D, dtype=BF16, device=DEV)
    jl.jl_page_summaries(k, table, _i32([0]), _i32(lens), s, max_new=lens[0], rope_base=1e6)
    want = ph.summary(_keys(k, table, 0, lens[0], 5)[20 * P:], P, 1e6)
    assert np.abs(_f64(s[int(table[0, 20]), 5]) - want).max() <= 2.0 ** -8 * np.abs(want).max()


def test_decode_flags_bad_lengths_and_pages():
    g = torch.Generator().manual_seed(6)
    P, Hq, Hkv, D = 16, 4, 2, 128
    k, v = _pool(g, 8, P, Hkv, D)
    q = _randn(g, 3, Hq, D)
    table = _i32([[0, 1, 2], [3, 4, 5], [6, 7, 0]])
    ws = _ws(Hq, Hkv, D)
    for lens in ([48, -1, 20], [49, 10, 20]):
        o, lse, err = torch.empty_like(q), torch.empty(3, Hq, device=DEV), _i32([0])
        jl.jl_bifocal_decode_paged(q, k, v, table, _i32(lens), o, lse, w0=4, w_pretrained=16, rope_base=1e4,
                                   workspace=ws, dev_error=err)
        assert int(err) == 2
        good = [x if 0 <= x <= 48 else 0 for x in lens]
        _check_decode(o, lse, q, k, v, table, good, 4, 16, 1e4)
    table[1, 1] = 8  # behind the pool: the other pages' keys remain
    o, lse, err = torch.empty_like(q), torch.empty(3, Hq, device=DEV), _i32([0])
    jl.jl_bifocal_decode_paged(q, k, v, table, _i32([40, 40, 40]), o, lse, w0=4, w_pretrained=16, rope_base=1e4,
                               workspace=ws, dev_error=err)
    assert int(err) == 2
    table[1, 1] = 0
    _check_decode(o, lse, q, k, v, table, [40] * 3, 4, 16, 1e4,
                  lists=[[[0, 1, 2]] * 2, [[0, 2]] * 2, [[0, 1, 2]] * 2])


def test_decode_runs_are_equal_bit_for_bit():
    g = torch.Generator().manual_seed(8)
    lens, P, Hq, Hkv, D = [4000, 1, 900, 0, 12000], 16, 32, 8, 128
    k, v = _pool(g, 1100, P, Hkv, D)
    table = _table(g, lens, P, 1100)
    q = _randn(g, 5, Hq, D)
    ws, got = _ws(Hq, Hkv, D), []
    for _ in range(4):
        o, lse = torch.empty_like(q), torch.empty(5, Hq, device=DEV)
        jl.jl_bifocal_decode_paged(q, k, v, table, _i32(lens), o, lse, w0=500, w_pretrained=3000, rope_base=1e6,
                                   workspace=ws)
        got.append((o, lse))
    assert all(torch.equal(o, got[0][0]) and torch.equal(x, got[0][1]) for o, x in got)


@pytest.mark.parametrize("Hq,Hkv,D,lens", [(32, 8, 128, [3000, 2900, 3100, 50]), (8, 8, 64, [5000, 4100, 600, 77]),
                                           (24, 3, 128, [9000, 2000, 4000, 8000]), (6, 2, 64, [20000, 30000, 9, 1000]),
                                           (32, 8, 128, [1500, 1400, 1300, 1200, 1100, 1600, 1700, 1250])])
def test_decode_sums_do_not_depend_on_which_cta_comes_last(Hq, Hkv, D, lens):
    # Items that several CTAs share, most CTAs two of them: which CTA joins what, and
    # whether one joins both its items, changes from run to run; the results do not.
    g = torch.Generator().manual_seed(18)
    P, need = 16, sum((x + 15) // 16 for x in lens) + 8
    k, v = _pool(g, need, P, Hkv, D)
    table = _table(g, lens, P, need)
    q = _randn(g, len(lens), Hq, D)
    ws, n = _ws(Hq, Hkv, D), _i32(lens)
    o = torch.empty(300, *q.shape, dtype=q.dtype, device=DEV)
    lse = torch.empty(300, len(lens), Hq, device=DEV)
    for i in range(300):
        jl.jl_bifocal_decode_paged(q, k, v, table, n, o[i], lse[i], w0=500, w_pretrained=3000, rope_base=1e6,
                                   workspace=ws)
    assert (o == o[0]).all() and (lse == lse[0]).all()


def test_decode_graph_serves_other_lengths_and_streams():
    g = torch.Generator().manual_seed(10)
    P, Hq, Hkv, D = 32, 8, 2, 128
    k, v = _pool(g, 200, P, Hkv, D)
    table = torch.arange(200, dtype=torch.int32, device=DEV).view(4, 50)
    q = _randn(g, 4, Hq, D)
    lens = _i32([1600, 1600, 1600, 1600])
    o, lse, ws = torch.empty_like(q), torch.empty(4, Hq, device=DEV), _ws(Hq, Hkv, D)

    def call():
        jl.jl_bifocal_decode_paged(q, k, v, table, lens, o, lse, w0=40, w_pretrained=500, rope_base=1e6, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for now in ([1600] * 4, [0, 3, 1599, 700], [1, 0, 0, 0]):
        lens.copy_(_i32(now))
        graph.replay()
        torch.cuda.synchronize()
        _check_decode(o, lse, q, k, v, table, now, 40, 500, 1e6)


# ---------------------------------------------------------------- summaries, selection, sparse decode
@pytest.mark.parametrize("lens,starts,Hkv,D,P,layout", [
    ([100, 1, 0, 48], [0, 0, 0, 0], 2, 128, 16, "rows"), ([333, 64], [330, 63], 1, 64, 32, "heads"),
    ([257, 500], [200, 500], 3, 128, 48, "beside"), ([2000], [0], 8, 64, 1024, "interleaved")])
def test_summaries(lens, starts, Hkv, D, P, layout):
    g = torch.Generator().manual_seed(P)
    n = sum(-(-x // P) for x in lens) + 2
    k, v = _pool(g, n, P, Hkv, D, layout)
    table = _table(g, lens, P, n)
    _stale(k, v, table, lens, float("nan"))
    s = torch.full((n, Hkv, D), 7.0, dtype=BF16, device=DEV)
    want = _f64(s)
    err = _i32([0])
    jl.jl_page_summaries(k, table, _i32(starts), _i32(lens), s, max_new=max(x - y for x, y in zip(lens, starts)),
                         rope_base=1e5, dev_error=err)
    assert int(err) == 0
    tol = np.zeros_like(want)
    for b, L in enumerate(lens):
        for p in range(starts[b] // P, -(-L // P) if starts[b] < L else 0):
            for h in range(Hkv):
                keys = _keys(k, table, b, L, h)[p * P:(p + 1) * P]
                want[int(table[b, p]), h] = ph.summary(keys, P, 1e5)
                # fp32 Horner steps: at most P / 4 of them, each 2^-22 of a sum below n max|pair|
                pair = np.hypot(keys[:, :D // 2], keys[:, D // 2:]).max()
                tol[int(table[b, p]), h] = (P // 4 + 8) * 2.0 ** -22 * pair
    assert np.all(np.abs(_f64(s) - want) <= tol + ph.BF16_HALF * np.abs(want) * (tol > 0))


def test_summaries_flag_more_pages_than_the_call_was_sized_for():
    g = torch.Generator().manual_seed(1)
    k, _ = _pool(g, 8, 16, 1, 64)
    table = _i32([[0, 1, 2, 3]])
    for lens, starts, new in (([60], [0], 16), ([65], [60], 1), ([-1], [0], 8), ([10], [-1], 8)):
        s = torch.full((8, 1, 64), 7.0, dtype=BF16, device=DEV)
        err = _i32([0])
        jl.jl_page_summaries(k, table, _i32(starts), _i32(lens), s, max_new=new, rope_base=1e4, dev_error=err)
        assert int(err) == 2 and torch.all(s == 7.0)


def _select(q, s, table, lens, P, w0, W, sink, top_k, base, mode=jo.MODE_SELF_EXTEND, width=None):
    B, Hq, D = q.shape
    Hkv = s.shape[1]
    M = table.shape[1]
    width = max(1, min(M, sink + top_k + -(-w0 // P) + 1)) if width is None else width
    lst = torch.full((B, Hkv, width), 55, dtype=torch.int32, device=DEV)
    cnt = torch.full((B, Hkv), 55, dtype=torch.int32, device=DEV)
    ws = torch.full((jl.jl_select_pages_workspace_bytes(B, Hkv, M),), 255, dtype=torch.uint8, device=DEV)
    err = _i32([0])
    jl.jl_select_pages(q, s, table, _i32(lens), lst, cnt, page_size=P, sink_pages=sink, top_k=top_k, w0=w0,
                       w_pretrained=W, rope_base=base, mode=MODES[mode], workspace=ws, dev_error=err)
    return lst, cnt, int(err)


def _check_lists(lst, cnt, q, s, table, lens, P, w0, W, sink, top_k, base, mode=jo.MODE_SELF_EXTEND):
    Hkv = s.shape[1]
    r = q.shape[1] // Hkv
    got, n = lst.cpu().tolist(), cnt.cpu().tolist()
    kept = []
    for b, L in enumerate(lens):
        kept.append([])
        ids = table[b, :-(-L // P)].long()
        for g in range(Hkv):
            want = ph.select(_f64(q[b, g * r:(g + 1) * r]), _f64(s[ids, g]), L, P, w0, W, sink, top_k, base, mode)
            assert n[b][g] == len(want), (b, g, n[b][g], len(want))
            assert got[b][g] == want + [-1] * (len(got[b][g]) - len(want)), (b, g)
            kept[-1].append(want)
    return kept


@pytest.mark.parametrize("lens,Hq,Hkv,D,P,w0,W,sink,top_k", [
    ([1], 2, 1, 64, 16, 0, 4, 0, 1), ([0, 16, 17, 40], 4, 2, 128, 16, 0, 8, 1, 1),
    ([5000, 900, 0, 33], 8, 2, 128, 16, 100, 1000, 2, 17), ([20000], 32, 8, 128, 16, 1000, 3000, 1, 200),
    ([4000, 4001], 7, 1, 64, 32, 4096, 1000, 0, 5), ([3000], 24, 3, 128, 48, 10, 100, 1, 0),
    ([9999, 10000], 10, 10, 64, 16, 333, 100000, 5, 512), ([70000], 5, 1, 128, 16, 64, 9000, 1, 600)])
@pytest.mark.parametrize("mode", [jo.MODE_SELF_EXTEND, jo.MODE_NONE])
def test_select_and_sparse_decode(lens, Hq, Hkv, D, P, w0, W, sink, top_k, mode):
    g = torch.Generator().manual_seed(sum(lens) + D)
    n = sum(-(-x // P) for x in lens) + 2
    k, v = _pool(g, n, P, Hkv, D)
    table = _table(g, lens, P, n)
    q, s = _randn(g, len(lens), Hq, D), _randn(g, n, Hkv, D, scale=P ** -0.5)
    lst, cnt, err = _select(q, s, table, lens, P, w0, W, sink, top_k, 1e6, mode)
    assert err == 0
    kept = _check_lists(lst, cnt, q, s, table, lens, P, w0, W, sink, top_k, 1e6, mode)
    o, lse = torch.empty_like(q), torch.empty(len(lens), Hq, device=DEV)
    e = _i32([0])
    jl.jl_bifocal_decode_paged_sparse(q, k, v, table, _i32(lens), lst, cnt, o, lse, w0=w0, w_pretrained=W,
                                      rope_base=1e6, mode=MODES[mode], workspace=_ws(Hq, Hkv, D), dev_error=e)
    assert int(e) == 0
    _check_decode(o, lse, q, k, v, table, lens, w0, W, 1e6, mode, lists=kept)


@pytest.mark.parametrize("n", [1000, 5000, 20000])  # one, two and eight CTAs per row
def test_select_ties_go_to_the_lowest_page(n):
    P, D = 16, 64
    s = torch.zeros(n, 2, D, dtype=BF16, device=DEV)  # every score is zero, of either sign
    g = torch.Generator().manual_seed(0)
    q = _randn(g, 1, 4, D)
    table = torch.arange(n, dtype=torch.int32, device=DEV)[None]
    top = 600 * n // 1000
    lst, cnt, err = _select(q, s, table, [P * n], P, 0, 4000, 2, top, 1e4)
    assert err == 0 and cnt.tolist() == [[top + 3, top + 3]]
    assert lst[0, 0].tolist() == list(range(top + 2)) + [n - 1]
    # a NaN summary scores above everything, and in one head only
    s[n - 300, 1, 3] = float("nan")
    lst, cnt, _ = _select(q, s, table, [P * n], P, 0, 4000, 2, top, 1e4)
    assert lst[0, 1].tolist() == list(range(top + 1)) + [n - 300, n - 1]
    assert lst[0, 0].tolist() == list(range(top + 2)) + [n - 1]


@pytest.mark.parametrize("kind", ["plain", "large", "tiny", "equal", "close"])
@pytest.mark.parametrize("pages,Hq,Hkv,D,top_k", [(3000, 4, 1, 128, 100), (70000, 2, 2, 64, 900), (9000, 8, 1, 64, 5)])
def test_select_where_the_error_bound_decides(kind, pages, Hq, Hkv, D, top_k):
    # scores that the first pass tells apart, lengths beyond its range, lengths below it,
    # summaries that are all the same, and summaries one rounding step apart
    g = torch.Generator().manual_seed(pages)
    P, L = 16, 16 * pages
    scale = {"plain": 0.25, "large": 1e6, "tiny": 1e-9}.get(kind, 1.0)
    s = _randn(g, pages, Hkv, D, scale=scale)
    if kind in ("equal", "close"):
        s = s[:1].expand(pages, Hkv, D).contiguous()
    if kind == "close":
        s *= torch.where(torch.rand(pages, Hkv, D, generator=g) < 0.5, 1.0, 1.0 + 2.0 ** -7).to(BF16).to(DEV)
    q = _randn(g, 1, Hq, D)
    table = torch.randperm(pages, generator=g).to(torch.int32).to(DEV)[None]
    # with w_pretrained 8 the pages share few positions, and equal summaries score alike
    W = 8 if kind in ("equal", "close") else L // 5
    lst, cnt, err = _select(q, s, table, [L], P, 200, W, 3, top_k, 1e6)
    assert err == 0
    _check_lists(lst, cnt, q, s, table, [L], P, 200, W, 3, top_k, 1e6)


def test_select_flags_bad_lengths_and_pages():
    g = torch.Generator().manual_seed(5)
    P, D = 16, 128
    s, q = _randn(g, 20, 2, D), _randn(g, 2, 4, D)
    table = torch.arange(20, dtype=torch.int32, device=DEV).view(2, 10)
    lst, cnt, err = _select(q, s, table, [161, 100], P, 0, 50, 0, 3, 1e4)
    assert err == 2 and cnt.tolist()[0] == [0, 0] and torch.all(lst[0] == -1)
    _check_lists(lst, cnt, q, s, table, [0, 100], P, 0, 50, 0, 3, 1e4)
    table[0, 4] = -1  # scores -inf: the last to be taken
    lst, cnt, err = _select(q, s, table, [160, 100], P, 0, 50, 0, 8, 1e4)
    assert err == 2 and lst[0, 0].tolist() == [0, 1, 2, 3, 5, 6, 7, 8, 9]


def test_sparse_decode_lists_in_any_order_and_bad_entries():
    g = torch.Generator().manual_seed(12)
    lens, P, Hq, Hkv, D = [1000, 300], 16, 8, 2, 128
    k, v = _pool(g, 90, P, Hkv, D)
    table = _table(g, lens, P, 90)
    q = _randn(g, 2, Hq, D)
    lists = [[[62, 0, 17, 5], [3]], [[18], []]]
    lst = torch.full((2, Hkv, 6), -1, dtype=torch.int32, device=DEV)
    for b in range(2):
        for h in range(Hkv):
            lst[b, h, :len(lists[b][h])] = _i32(lists[b][h])
    cnt = _i32([[len(x) for x in y] for y in lists])
    ws = _ws(Hq, Hkv, D)
    o, lse, err = torch.empty_like(q), torch.empty(2, Hq, device=DEV), _i32([0])
    jl.jl_bifocal_decode_paged_sparse(q, k, v, table, _i32(lens), lst, cnt, o, lse, w0=40, w_pretrained=200,
                                      rope_base=1e4, workspace=ws, dev_error=err)
    assert int(err) == 0
    _check_decode(o, lse, q, k, v, table, lens, 40, 200, 1e4, lists=lists)
    # entries outside the table, and a count outside the list
    lst[0, 0, 4] = -1
    lst[0, 0, 5] = 63
    cnt[0, 0], cnt[0, 1] = 6, 7
    jl.jl_bifocal_decode_paged_sparse(q, k, v, table, _i32(lens), lst, cnt, o, lse, w0=40, w_pretrained=200,
                                      rope_base=1e4, workspace=ws, dev_error=err)
    assert int(err) == 2
    lists[0][1] = []
    _check_decode(o, lse, q, k, v, table, lens, 40, 200, 1e4, lists=lists)


# ---------------------------------------------------------------- all of them together
def test_prompt_and_decode_steps_across_a_group_border():
    # two prompts, prefilled over contiguous keys and paged at once, then decode steps that cross
    # multiples of w_pretrained: append, summarise, attend densely, select, attend sparsely
    B, Hq, Hkv, D, P, W, w0, base = 2, 8, 2, 128, 16, 128, 40, 1e6
    g = torch.Generator().manual_seed(77)
    lens, M, steps = [250, 383], 26, 10
    k, v = _pool(g, 60, P, Hkv, D, fill=float("nan"))
    s = torch.full((60, Hkv, D), float("nan"), dtype=BF16, device=DEV)
    table = torch.randperm(60, generator=g)[:B * M].view(B, M).to(torch.int32).to(DEV)
    qw, kw = _randn(g, D), _randn(g, D)
    err, ws = _i32([0]), _ws(Hq, Hkv, D)
    T = sum(lens)
    x = _randn(g, T, Hq + 2 * Hkv, D)
    seq = _i32([b for b, n in enumerate(lens) for _ in range(n)])
    pos = _i32([p for n in lens for p in range(n)])
    qo, ko = (torch.empty(T, h, D, dtype=BF16, device=DEV) for h in (Hq, Hkv))
    jl.jl_qk_norm_rope_append_paged(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], qw, kw, seq, pos, table, qo, k, v,
                                    eps=ph.EPS, rope_base=base, k_out=ko, dev_error=err)
    L = lens[0]  # the prefill of the first prompt reads the contiguous copies
    o, lse = torch.empty(1, L, Hq, D, dtype=BF16, device=DEV), torch.empty(1, Hq, L, device=DEV)
    vc = x[:L, Hq + Hkv:].contiguous()[None]
    jl.jl_bifocal_prefill(qo[None, :L], ko[None, :L], vc, o, lse, w0=w0, w_pretrained=W, rope_base=base,
                          workspace=torch.empty(jl.jl_prefill_workspace_bytes(1, L, Hq, Hkv, D), dtype=torch.uint8,
                                                device=DEV), dev_error=err)
    q_last = torch.stack([qo[lens[0] - 1], qo[T - 1]])
    jl.jl_page_summaries(k, table, _i32([0, 0]), _i32(lens), s, max_new=max(lens), rope_base=base, dev_error=err)
    od, ld = torch.empty(B, Hq, D, dtype=BF16, device=DEV), torch.empty(B, Hq, device=DEV)
    jl.jl_bifocal_decode_paged(q_last, k, v, table, _i32(lens), od, ld, w0=w0, w_pretrained=W, rope_base=base,
                               workspace=ws, dev_error=err)
    assert int(err) == 0
    # the prefill's last row is the decode of the last token
    assert (od[0].float() - o[0, L - 1].float()).abs().max() <= 2e-2
    assert (ld[0] - lse[0, :, L - 1]).abs().max() <= 1e-3
    seen = set()
    for _ in range(steps):
        lens = [n + 1 for n in lens]
        seen |= {jo.group_size(n, W) for n in lens}
        x = _randn(g, B, Hq + 2 * Hkv, D)
        new, qs = _i32([n - 1 for n in lens]), torch.empty(B, Hq, D, dtype=BF16, device=DEV)
        jl.jl_qk_norm_rope_append_paged(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], qw, kw, _i32([0, 1]), new,
                                        table, qs, k, v, eps=ph.EPS, rope_base=base, dev_error=err)
        jl.jl_page_summaries(k, table, new, new + 1, s, max_new=1, rope_base=base, dev_error=err)
        jl.jl_bifocal_decode_paged(qs, k, v, table, new + 1, od, ld, w0=w0, w_pretrained=W, rope_base=base,
                                   workspace=ws, dev_error=err)
        _check_decode(od, ld, qs, k, v, table, lens, w0, W, base)
        lst, cnt, e = _select(qs, s, table, lens, P, w0, W, 1, 3, base)
        assert e == 0
        kept = _check_lists(lst, cnt, qs, s, table, lens, P, w0, W, 1, 3, base)
        jl.jl_bifocal_decode_paged_sparse(qs, k, v, table, new + 1, lst, cnt, od, ld, w0=w0, w_pretrained=W,
                                          rope_base=base, workspace=ws, dev_error=err)
        _check_decode(od, ld, qs, k, v, table, lens, w0, W, base, lists=kept)
        assert int(err) == 0
    assert {2, 3, 4} <= seen


def test_a_captured_step_serves_other_lengths():
    # append, summaries, selection and both decodes in one graph, replayed as sequences grow
    # and end; a padded slot carries length 0 and position -1
    B, Hq, Hkv, D, P, M = 3, 8, 2, 64, 16, 30
    W, w0, base = 100, 30, 1e4
    g = torch.Generator().manual_seed(5)
    k, v = _pool(g, B * M, P, Hkv, D)
    table = torch.randperm(B * M, generator=g).view(B, M).to(torch.int32).to(DEV)
    s = _randn(g, B * M, Hkv, D, scale=0.25)
    x, w = _randn(g, B, Hq + 2 * Hkv, D), _randn(g, D)
    seq, pos, lens = _i32([0, 1, 2]), _i32([0, 0, 0]), _i32([1, 1, 1])
    q, od, os_ = (torch.zeros(B, Hq, D, dtype=BF16, device=DEV) for _ in range(3))
    ld, ls = (torch.zeros(B, Hq, device=DEV) for _ in range(2))
    lst, cnt = torch.zeros(B, Hkv, 8, dtype=torch.int32, device=DEV), torch.zeros(B, Hkv, dtype=torch.int32, device=DEV)
    ws, err = _ws(Hq, Hkv, D), _i32([0])
    sel = torch.zeros(jl.jl_select_pages_workspace_bytes(B, Hkv, M), dtype=torch.uint8, device=DEV)
    rule = dict(w0=w0, w_pretrained=W, rope_base=base, dev_error=err)

    def step():
        jl.jl_qk_norm_rope_append_paged(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], w, w, seq, pos, table, q, k, v,
                                        eps=ph.EPS, rope_base=base, dev_error=err)
        jl.jl_page_summaries(k, table, pos.clamp(min=0), lens, s, max_new=1, rope_base=base, dev_error=err)
        jl.jl_select_pages(q, s, table, lens, lst, cnt, page_size=P, sink_pages=1, top_k=4, workspace=sel, **rule)
        jl.jl_bifocal_decode_paged_sparse(q, k, v, table, lens, lst, cnt, os_, ls, workspace=ws, **rule)
        jl.jl_bifocal_decode_paged(q, k, v, table, lens, od, ld, workspace=ws, **rule)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for now in ([450, 1, 300], [451, 0, 301], [16, 17, 479]):
        lens.copy_(_i32(now))
        pos.copy_(_i32([n - 1 for n in now]))
        x.copy_(_randn(g, B, Hq + 2 * Hkv, D))
        graph.replay()
        torch.cuda.synchronize()
        assert int(err) == 0
        _check_decode(od, ld, q, k, v, table, now, w0, W, base)
        kept = _check_lists(lst, cnt, q, s, table, now, P, w0, W, 1, 4, base)
        _check_decode(os_, ls, q, k, v, table, now, w0, W, base, lists=kept)


def test_two_streams_with_their_own_workspaces():
    g = torch.Generator().manual_seed(31)
    P, Hq, Hkv, D = 16, 8, 2, 128
    k, v = _pool(g, 1300, P, Hkv, D)
    cases = []
    for lens in ([9000, 5], [300, 11000]):
        table = _table(g, lens, P, 1300)
        cases.append((lens, table, _randn(g, 2, Hq, D), _i32(lens)))
    want = []
    for lens, table, q, sl in cases:
        o, lse = torch.empty_like(q), torch.empty(2, Hq, device=DEV)
        jl.jl_bifocal_decode_paged(q, k, v, table, sl, o, lse, w0=50, w_pretrained=2000, rope_base=1e6,
                                   workspace=_ws(Hq, Hkv, D))
        want.append((o, lse))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [_ws(Hq, Hkv, D), _ws(Hq, Hkv, D)]
    outs = [(torch.empty_like(c[2]), torch.empty(2, Hq, device=DEV)) for c in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for (lens, table, q, sl), st, ws, (o, lse) in zip(cases, streams, spaces, outs):
            jl.jl_bifocal_decode_paged(q, k, v, table, sl, o, lse, w0=50, w_pretrained=2000, rope_base=1e6,
                                       workspace=ws, stream=st)
    torch.cuda.synchronize()
    for (o, lse), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_outputs_stay_inside_their_buffers():
    # 256-byte margins of a known pattern around every output and the scratch
    g = torch.Generator().manual_seed(15)
    B, Hq, Hkv, D, P, lens = 3, 8, 2, 128, 16, [500, 0, 77]
    pads = []

    def guarded(shape, dtype, zero=False):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        room = -(-n // 256) * 256
        buf = torch.full((room + 512,), 0xA5, dtype=torch.uint8, device=DEV)
        if zero:
            buf[256:256 + n] = 0
        pads.append((buf, n))
        return buf[256:256 + n].view(dtype).view(shape)

    k, v = _pool(g, 60, P, Hkv, D)
    table = _table(g, lens, P, 60)
    k0, v0, t0 = k.clone(), v.clone(), table.clone()
    q = _randn(g, B, Hq, D)
    o, lse = guarded((B, Hq, D), BF16), guarded((B, Hq), torch.float32)
    ws = guarded((jl.jl_decode_paged_workspace_bytes(Hq, Hkv, D),), torch.uint8, zero=True)
    M = table.shape[1]
    lst, cnt = guarded((B, Hkv, M), torch.int32), guarded((B, Hkv), torch.int32)
    sw = guarded((jl.jl_select_pages_workspace_bytes(B, Hkv, M),), torch.uint8)
    s = guarded((60, Hkv, D), BF16)
    sl = _i32(lens)
    jl.jl_page_summaries(k, table, _i32([0, 0, 0]), sl, s, max_new=500, rope_base=1e4)
    jl.jl_select_pages(q, s, table, sl, lst, cnt, page_size=P, sink_pages=1, top_k=5, w0=20, w_pretrained=100,
                       rope_base=1e4, workspace=sw)
    rule = dict(w0=20, w_pretrained=100, rope_base=1e4, workspace=ws)
    jl.jl_bifocal_decode_paged_sparse(q, k, v, table, sl, lst, cnt, o, lse, **rule)
    jl.jl_bifocal_decode_paged(q, k, v, table, sl, o, lse, **rule)
    T = 9
    qo, ko = guarded((T, Hq, D), BF16), guarded((T, Hkv, D), BF16)
    jl.jl_qk_norm_rope(_randn(g, T, Hq, D), _randn(g, T, Hkv, D), None, None, _i32(list(range(T))), qo, ko, eps=0.0,
                       rope_base=1e4)
    torch.cuda.synchronize()
    for buf, n in pads:
        assert torch.all(buf[:256] == 0xA5) and torch.all(buf[256 + n:] == 0xA5)
    assert torch.equal(k, k0) and torch.equal(v, v0) and torch.equal(table, t0)
    _check_decode(o, lse, q, k, v, table, lens, 20, 100, 1e4)


def test_bindings_refuse_what_they_cannot_describe():
    g = torch.Generator().manual_seed(1)
    k, v = _pool(g, 4, 16, 2, 64)
    q, o = _randn(g, 1, 4, 64), torch.empty(1, 4, 64, dtype=BF16, device=DEV)
    table, lens = _i32([[0, 1]]), _i32([20])
    kw = dict(w0=1, w_pretrained=8, rope_base=1e4, workspace=_ws(4, 2, 64))
    for bad in (dict(k=k[:, :, :, ::2]), dict(v=v[:3]), dict(table=table.long()), dict(lens=_i32([1, 2])),
                dict(o=o.float()), dict(q=q.cpu())):
        a = {"q": q, "k": k, "v": v, "table": table, "lens": lens, "o": o, **bad}
        with pytest.raises(ValueError):
            jl.jl_bifocal_decode_paged(a["q"], a["k"], a["v"], a["table"], a["lens"], a["o"], None, **kw)
    with pytest.raises(jl.JetLongError):
        jl.jl_bifocal_decode_paged(q, k, v, table, lens, o, None, **{**kw, "workspace": None})
    x = _randn(g, 3, 8, 64)
    with pytest.raises(ValueError):  # heads apart
        jl.jl_qk_norm_rope(x[:, ::2], x[:, :2], None, None, _i32([0, 1, 2]), torch.empty(3, 4, 64, dtype=BF16, device=DEV),
                           torch.empty(3, 2, 64, dtype=BF16, device=DEV), eps=0.0, rope_base=1e4)
