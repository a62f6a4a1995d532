"""The paged-cache operators' cases: query / key norms with the rotation (and the append to the pages),
paged decode, page summaries, and the sparse decode step over selected pages.

Every case is one call as a serving loop makes it, on Qwen3-shaped or the test suite's tiny head layouts.
"""

import math

import torch

own = False

EPS = 1e-6  # the norms' epsilon (the value these models are configured with)


def _case(name, kind, **kw):
    c = {"name": name, "kind": kind, "B": 1, "L": 1, "Hq": 32, "Hkv": 8, "D": 128, "P": 16, "w0": 4096, "W": 32768,
         "base": 1e6, "ragged": False, "fused": True, "norm": True, "outliers": False, "hnd": False, "step": False,
         "sink": 1, "top_k": 32, "shift": True}
    c.update(kw)
    return c


def listed():
    return [
        # a prompt chunk's fused QKV projection, 8B-shaped layer: norms + rotation before the prefill attention
        _case("norm_rope chunk 8192", "norm_rope", L=8192),
        # small heads, an odd number of tokens, separate projections
        _case("norm_rope 4099 d64", "norm_rope", L=4099, Hq=2, Hkv=1, D=64, base=1e4, fused=False),
        # a whole 128K prompt written into a paged cache
        _case("append prompt 128K", "append", L=131072, P=64),
        # one decode step's new tokens, eight sequences of which one slot is padding (latency)
        _case("append 8 tokens", "append", B=8, L=131072, P=16, step=True),
        # one long sequence, small pages
        _case("decode b1 128K", "decode", L=131072, P=16),
        # the decode workload of the benchmark, paged
        _case("decode b8 128K", "decode", B=8, L=131072, P=64),
        # a continuous batch: 64 sequences of 0 to 8192 keys, padded slots among them, group sizes 1 to 4
        _case("decode b64 ragged", "decode", B=64, L=8192, Hq=16, P=32, w0=256, W=2048, ragged=True),
        # a short sequence on the tiny head layout (latency)
        _case("decode b1 777 d64", "decode", L=777, Hq=2, Hkv=1, D=64, P=16, w0=32, W=128, base=1e4),
        # summaries of a prompt's pages, once after the prefill
        _case("summaries prompt 128K", "summaries", L=131072, P=64),
        # the last pages' summaries after one decode step (latency)
        _case("summaries 8 tokens", "summaries", B=8, L=131072, P=16, step=True),
        # one sparse decode step of eight 128K sequences: select pages, attend to them
        _case("sparse b8 128K", "sparse", B=8, L=131072, P=64),
        # a million tokens, one sequence: 65536 small pages to choose from
        _case("sparse b1 1M", "sparse", L=1048576, P=16, top_k=256),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm_rope", "append", "decode", "decode", "summaries", "sparse", "sparse"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    r = rng.choice([1, 2, 3, 4, 5, 7, 8])
    Hq = Hkv * r
    P = rng.choice([16, 32, 48, 64, 128])
    B = _log_int(rng, 1, 64)
    step = kind in ("append", "summaries") and rng.random() < 0.4
    per_seq = max(64, min(262144, 1048576 // B))
    if kind in ("norm_rope", "append") and not step:
        B = min(B, 8)
        per_seq = max(64, 131072 // B)
        Hq = min(Hq, 32)
        Hq -= Hq % Hkv
    L = _log_int(rng, 1, 64) if rng.random() < 0.15 else _log_int(rng, 64, per_seq)
    W = max(1, _log_int(rng, max(1, L // 8), 2 * L))
    w0 = rng.choice([0, _log_int(rng, 1, L), max(1, L // 32), 4096])
    return _case("", kind, B=B, L=L, Hq=Hq, Hkv=Hkv, D=D, P=P, w0=w0, W=W, base=rng.choice([1e4, 1e6]),
                 ragged=rng.random() < 0.5, fused=rng.random() < 0.7, norm=rng.random() < 0.8,
                 outliers=rng.random() < 0.3, hnd=rng.random() < 0.3, step=step, sink=rng.choice([0, 1, 2]),
                 top_k=_log_int(rng, 1, 512), shift=rng.random() < 0.7)


# ------------------------------------------------------------------ the cases' sizes (the seed plays no part)
def _lens(c):
    """Per-sequence lengths: all L, or spread over 0 .. L (zero: a padded slot of the batch)."""
    if not c["ragged"] or c["B"] == 1:
        return [c["L"]] * c["B"]
    n = [int(c["L"] * ((7 * b + 3) % (2 * c["B"] - 1) + 1) / (2 * c["B"])) for b in range(c["B"])]
    n[0] = c["L"]
    n[c["B"] // 2] = 0 if c["B"] > 2 else max(1, c["L"] // 3)
    return n


def _pages(c, n):
    return -(-n // c["P"])


def _tokens(c):
    """(sequence, position) of every token of a norm_rope / append call."""
    if c["step"]:  # one new token per sequence; a padded slot carries position -1
        return [(b, n - 1) for b, n in enumerate(_lens(c))] if c["B"] < 8 else \
            [(b, -1 if b == c["B"] - 1 else n - 1) for b, n in enumerate(_lens(c))]
    return [(b, i) for b, n in enumerate(_lens(c)) for i in range(n)]


def _token_count(c):
    return c["B"] if c["step"] else sum(_lens(c))


def _kept(c, n):
    """Pages that a sparse step attends to for a sequence of n tokens."""
    if n == 0:
        return 0
    last = (n - 1) // c["P"]
    first = min(max(0, n - c["w0"]) // c["P"], last)
    return min(last + 1, last + 1 - first + min(c["sink"], first) + min(c["top_k"], max(0, first - c["sink"])))


def _list_width(c):
    return max(1, min(_pages(c, c["L"]), c["sink"] + c["top_k"] + _pages(c, c["w0"]) + 1))


def work(c):
    Hq, Hkv, D, P = c["Hq"], c["Hkv"], c["D"], c["P"]
    lens, T = _lens(c), _token_count(c)
    if c["kind"] == "norm_rope":
        return {"bytes": 4 * T * (Hq + Hkv) * D + 4 * T, "flops": 7 * T * (Hq + Hkv) * D}
    if c["kind"] == "append":
        return {"bytes": 4 * T * (Hq + 2 * Hkv) * D + 8 * T, "flops": 7 * T * (Hq + Hkv) * D}
    if c["kind"] == "decode":
        return {"bytes": sum(4 * n * Hkv * D + 4 * _pages(c, n) for n in lens) + 4 * c["B"] * Hq * (D + 1),
                "flops": sum(4 * n * Hq * D for n in lens)}
    if c["kind"] == "summaries":
        keys = sum((n - 1) % P + 1 for n in lens if n) if c["step"] else sum(lens)
        pages = sum(n > 0 for n in lens) if c["step"] else sum(_pages(c, n) for n in lens)
        return {"bytes": 2 * (keys + pages) * Hkv * D, "flops": 7 * keys * Hkv * D}
    cand = sum(max(0, min(max(0, n - c["w0"]) // P, max(0, n - 1) // P) - c["sink"]) for n in lens)
    keys = sum(min(n, _kept(c, n) * P) for n in lens)
    return {"bytes": 2 * cand * Hkv * D + 4 * keys * Hkv * D + 4 * c["B"] * (Hq * (D + 1) + Hkv * _list_width(c)),
            "flops": 2 * cand * Hq * D + 4 * keys * Hq * D}


# ------------------------------------------------------------------ inputs
def _bf16(g, *shape, scale=1.0):
    """N(0, scale^2) in bf16."""
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(scale)


def _pool(c, g, num_pages):
    """One page pool (K or V) as [pages, page_size, Hkv, D]; `hnd` keeps a head's rows of a page together."""
    if c["hnd"]:
        return _bf16(g, num_pages, c["Hkv"], c["P"], c["D"]).permute(0, 2, 1, 3)
    return _bf16(g, num_pages, c["P"], c["Hkv"], c["D"])


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(int(seed) * 1009 + 17)
    B, Hq, Hkv, D, P = c["B"], c["Hq"], c["Hkv"], c["D"], c["P"]
    lens = _lens(c)
    s = {"c": c, "seq_lens": torch.tensor(lens, dtype=torch.int32, device=dev), "keep": {}}
    if c["kind"] in ("norm_rope", "append"):
        if c["step"]:
            tok = torch.tensor(_tokens(c), dtype=torch.int32, device=dev)
            s["seq_ids"], s["positions"] = tok[:, 0].contiguous(), tok[:, 1].contiguous()
        else:
            s["seq_ids"] = torch.repeat_interleave(torch.arange(B, device=dev), s["seq_lens"].long()).to(torch.int32)
            s["positions"] = torch.cat([torch.arange(n, dtype=torch.int32, device=dev) for n in lens])
        T = _token_count(c)
        if c["fused"]:  # views of one projection's rows
            x = _bf16(g, T, Hq + 2 * Hkv, D, scale=2.0)
            s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            s["q"], s["k"], s["v"] = (_bf16(g, T, h, D, scale=2.0) for h in (Hq, Hkv, Hkv))
        s["qw"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16) if c["norm"] else None
        s["kw"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(torch.bfloat16) if c["norm"] else None
        s["q_out"] = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=dev)
        if c["kind"] == "norm_rope":
            s["k_out"] = torch.zeros(T, Hkv, D, dtype=torch.bfloat16, device=dev)
            return s
    # the page pool and the block table: pages in a random order, -1 behind a sequence's last page
    need = [_pages(c, n) for n in lens]
    num_pages, width = sum(need) + 3, max(1, max(need))
    perm = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
    cols = torch.arange(width, device=dev)[None, :]
    need_t = torch.tensor(need, device=dev)[:, None]
    first = torch.cumsum(need_t, 0) - need_t
    s["table"] = torch.where(cols < need_t, perm[(first + cols).clamp(max=num_pages - 1)], -1).to(torch.int32)
    s["spare"] = int(perm[-1])  # a page of the pool that no sequence holds
    s["k_pages"] = _pool(c, g, num_pages)
    if c["kind"] != "summaries":
        s["v_pages"] = _pool(c, g, num_pages)
    if c["outliers"]:  # 1% of the rows eight times as large
        rows = torch.rand(num_pages, P, Hkv, 1, generator=g, device=dev) < 0.01
        s["k_pages"].mul_(torch.where(rows, 8.0, 1.0).to(torch.bfloat16))
    if c["kind"] == "summaries":
        s["starts"] = torch.tensor([max(0, n - 1) if c["step"] else 0 for n in lens], dtype=torch.int32, device=dev)
        s["summaries"] = torch.zeros(num_pages, Hkv, D, dtype=torch.bfloat16, device=dev)
    if c["kind"] in ("decode", "sparse"):
        s["q"] = _bf16(g, B, Hq, D)
        s["o"] = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros(B, Hq, dtype=torch.float32, device=dev)
    if c["kind"] == "sparse":  # the pages' mean keys, as the summaries hold them (spread of a mean of P keys)
        s["summaries"] = _bf16(g, num_pages, Hkv, D, scale=P ** -0.5)
        s["page_list"] = torch.full((B, Hkv, _list_width(c)), -1, dtype=torch.int32, device=dev)
        s["page_counts"] = torch.zeros(B, Hkv, dtype=torch.int32, device=dev)
    return s


# ------------------------------------------------------------------ plain forms
def _theta(c, device):
    t = torch.arange(c["D"] // 2, dtype=torch.float64, device=device)
    return c["base"] ** (-2.0 * t / c["D"])


def _rotate(x, turns, c, dtype=torch.float32):
    """R(turns) x over x's last axis; turns: integers, broadcast against x's other axes."""
    ang = turns.double()[..., None] * _theta(c, x.device)
    cs, sn = torch.cos(ang).to(dtype), torch.sin(ang).to(dtype)
    a, b = x[..., :c["D"] // 2].to(dtype), x[..., c["D"] // 2:].to(dtype)
    return torch.cat([a * cs - b * sn, b * cs + a * sn], -1)


def _norm(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _norm_rope_plain(s):
    c, pos = s["c"], s["positions"][:, None]
    live = (pos >= 0)[..., None]
    q = _rotate(_norm(s["q"], s["qw"]), pos, c).to(torch.bfloat16)
    k = _rotate(_norm(s["k"], s["kw"]), pos, c).to(torch.bfloat16)
    return torch.where(live, q, s["q_out"]), k


def _algebra(c, lens):
    """(G, query position minus its own, all-local) per sequence, int64."""
    n = lens.long().clamp(min=1)
    G = ((n + c["W"] - 1) // c["W"]).clamp(min=1)
    shift = c["w0"] - c["w0"] // G if c["shift"] else torch.zeros_like(G)
    return G, (n - 1) // G + shift - (n - 1), (G == 1) | (n <= c["w0"])


def _attend_plain(s, pages, pos):
    """Attention of s["q"] over keys of `pages` [B, Hkv, M] (page ids) at positions pos [B, Hkv or 1, M P]; entries
    with pos < 0 or behind the sequence take no part."""
    c = s["c"]
    B, Hq, Hkv, D, P = c["B"], c["Hq"], c["Hkv"], c["D"], c["P"]
    lens = s["seq_lens"].long()
    G, dq, local_all = _algebra(c, lens)
    head = torch.arange(Hkv, device=pos.device)[None, :, None]
    safe = pages.clamp(min=0).long()
    k = s["k_pages"].permute(0, 2, 1, 3)[safe, head].reshape(B, Hkv, -1, D).float()
    v = s["v_pages"].permute(0, 2, 1, 3)[safe, head].reshape(B, Hkv, -1, D).float()
    n = lens[:, None, None]
    live = (pos >= 0) & (pos < n)
    local = local_all[:, None, None] | (n - 1 - pos < c["w0"])
    q = s["q"].float()
    qr = _rotate(q, dq[:, None], c).view(B, Hkv, -1, D)
    q = q.view(B, Hkv, -1, D)
    near = torch.matmul(q, k.transpose(-1, -2))
    far = torch.matmul(qr, _rotate(k, pos.clamp(min=0) // G[:, None, None] - pos.clamp(min=0), c).transpose(-1, -2))
    x = torch.where(local[:, :, None], near, far) * D ** -0.5
    x = torch.where(live[:, :, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, torch.where(live[..., None], v, 0.0)) / torch.where(total == 0, 1.0, total)
    lse = (torch.log(total) + m).view(B, Hq)
    return o.view(B, Hq, D).to(torch.bfloat16), lse


def _decode_plain(s):
    c, table = s["c"], s["table"]
    pos = torch.arange(table.shape[1] * c["P"], device=table.device)
    return _attend_plain(s, table[:, None].expand(-1, c["Hkv"], -1), pos.expand(c["B"], 1, -1))


def _select_plain(s):
    """(page_list, page_counts): scores in 64 bits, rounded to fp32; ties to the lowest index."""
    c, table = s["c"], s["table"]
    B, Hkv, D, P = c["B"], c["Hkv"], c["D"], c["P"]
    M = table.shape[1]
    n = s["seq_lens"].long()
    G, dq, _ = _algebra(c, n)
    page = torch.arange(M, device=table.device)
    at = page * P + P // 2
    k = s["summaries"][table.clamp(min=0).long()].permute(0, 2, 1, 3)  # [B, Hkv, M, D]
    k = _rotate(k, (at // G[:, None] - at)[:, None], c, torch.float64)
    q = _rotate(s["q"], dq[:, None], c, torch.float64).view(B, Hkv, -1, D)
    score = torch.matmul(q, k.transpose(-1, -2)).amax(2).float()
    last = (n - 1).clamp(min=0) // P
    first = torch.minimum((n - c["w0"]).clamp(min=0) // P, last)[:, None, None]
    held = (page <= last[:, None, None]) & (n > 0)[:, None, None]
    always = held & ((page >= first) | (page < c["sink"]))
    open_ = held & ~always
    order = torch.sort(torch.where(open_, score, -math.inf), dim=-1, descending=True, stable=True).indices
    best = torch.zeros_like(open_.expand(B, Hkv, M)).scatter(-1, order[..., :c["top_k"]], True)
    kept = always | (open_ & best)
    width = _list_width(c)
    rank = torch.where(kept, page, M).sort(-1).values[..., :width]
    rank = torch.nn.functional.pad(rank, (0, width - rank.shape[-1]), value=M)
    return torch.where(rank < M, rank, -1).to(torch.int32), kept.sum(-1).to(torch.int32)


def _sparse_plain(s):
    c = s["c"]
    page_list, counts = _select_plain(s)
    at = page_list.long()
    pages = torch.gather(s["table"][:, None].expand(-1, c["Hkv"], -1), 2, at.clamp(min=0))
    off = torch.arange(c["P"], device=at.device)
    pos = torch.where(at[..., None] >= 0, at[..., None] * c["P"] + off, -1).flatten(2)
    o, lse = _attend_plain(s, pages, pos)
    return {"page_list": page_list, "page_counts": counts, "o": o, "lse": lse}


def _summaries_plain(s):
    c, table = s["c"], s["table"]
    P = c["P"]
    page = torch.arange(table.shape[1], device=table.device)
    n = (s["seq_lens"].long()[:, None] - page * P).clamp(0, P)
    b, p = torch.nonzero((n > 0) & (page >= s["starts"].long()[:, None] // P), as_tuple=True)
    ids, n = table[b, p].long(), n[b, p]
    off = torch.arange(P, device=table.device)
    k = _rotate(s["k_pages"][ids], (P // 2 - off)[:, None], c)
    k = torch.where((off < n[:, None])[..., None, None], k, 0.0)
    s["summaries"][ids] = (k.sum(1) / n[:, None, None]).to(torch.bfloat16)
    return s["summaries"]


def _append_plain(s):
    c = s["c"]
    q, k = _norm_rope_plain(s)
    pos, seq = s["positions"].long(), s["seq_ids"].long()
    live = pos >= 0
    at = pos.clamp(min=0)
    page = torch.where(live, s["table"][seq, at // c["P"]].long(), s["spare"])
    row = at % c["P"]
    keep = live[:, None, None]
    s["k_pages"][page, row] = torch.where(keep, k, s["k_pages"][page, row])
    s["v_pages"][page, row] = torch.where(keep, s["v"], s["v_pages"][page, row])
    return q


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    c, kind = s["c"], s["c"]["kind"]
    if own:
        return _run_own(s)
    if kind == "norm_rope":
        q, k = _norm_rope_plain(s)
        return {"q": q, "k": k}
    if kind == "append":
        return {"q": _append_plain(s), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if kind == "decode":
        o, lse = _decode_plain(s)
        return {"o": o, "lse": lse}
    if kind == "summaries":
        return {"summaries": _summaries_plain(s)}
    return _sparse_plain(s)


def _run_own(s):
    from rope_context_extension_b200 import jetlong as jl
    c, keep = s["c"], s["keep"]
    kind = c["kind"]
    if kind == "norm_rope":
        jl.jl_qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["positions"], s["q_out"], s["k_out"], eps=EPS,
                           rope_base=c["base"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if kind == "append":
        jl.jl_qk_norm_rope_append_paged(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["seq_ids"], s["positions"],
                                        s["table"], s["q_out"], s["k_pages"], s["v_pages"], eps=EPS,
                                        rope_base=c["base"])
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if kind == "summaries":
        jl.jl_page_summaries(s["k_pages"], s["table"], s["starts"], s["seq_lens"], s["summaries"],
                             max_new=1 if c["step"] else c["L"], rope_base=c["base"])
        return {"summaries": s["summaries"]}
    if not keep:  # scratch that a serving loop keeps from step to step
        keep["decode"] = torch.zeros(jl.jl_decode_paged_workspace_bytes(c["Hq"], c["Hkv"], c["D"]),
                                     dtype=torch.uint8, device=s["q"].device)
        if kind == "sparse":
            keep["select"] = torch.zeros(
                jl.jl_select_pages_workspace_bytes(c["B"], c["Hkv"], s["table"].shape[1]), dtype=torch.uint8,
                device=s["q"].device)
    mode = jl.JL_QSHIFT_SELF_EXTEND if c["shift"] else jl.JL_QSHIFT_NONE
    rule = {"w0": c["w0"], "w_pretrained": c["W"], "rope_base": c["base"], "mode": mode}
    if kind == "decode":
        jl.jl_bifocal_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["seq_lens"], s["o"], s["lse"],
                                   workspace=keep["decode"], **rule)
        return {"o": s["o"], "lse": s["lse"]}
    jl.jl_select_pages(s["q"], s["summaries"], s["table"], s["seq_lens"], s["page_list"], s["page_counts"],
                       page_size=c["P"], sink_pages=c["sink"], top_k=c["top_k"], workspace=keep["select"], **rule)
    jl.jl_bifocal_decode_paged_sparse(s["q"], s["k_pages"], s["v_pages"], s["table"], s["seq_lens"],
                                      s["page_list"], s["page_counts"], s["o"], s["lse"],
                                      workspace=keep["decode"], **rule)
    return {"page_list": s["page_list"], "page_counts": s["page_counts"], "o": s["o"], "lse": s["lse"]}


# ------------------------------------------------------------------ 64-bit values, from the definition
def _turn(x, positions, c):
    """x's rows as complex pairs times e^{i position theta}, in 64 bits (x: [..., D]; positions: [...])."""
    h = c["D"] // 2
    z = torch.complex(x[..., :h].double(), x[..., h:].double())
    theta = torch.tensor([c["base"] ** (-2.0 * t / c["D"]) for t in range(h)], dtype=torch.float64, device=x.device)
    ang = positions.double()[..., None] * theta
    return z * torch.complex(torch.cos(ang), torch.sin(ang))


def _real(z):
    return torch.cat([z.real, z.imag], -1)


def _exact_heads(x, w, pos, c):
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["D"] + EPS) * w.double()
    return _real(_turn(y, pos[:, None].expand(y.shape[:-1]), c))


def _exact_rows(s, b, g, pages, where):
    """o [r, D] and lse [r] of KV head g of sequence b over the page ids `pages` whose first positions are
    `where`: keys taken back to position 0, then placed where the rule says."""
    c = s["c"]
    r, D, P = c["Hq"] // c["Hkv"], c["D"], c["P"]
    L = int(s["seq_lens"][b])
    dev = s["q"].device
    pos = (where[:, None] + torch.arange(P, device=dev)).flatten()
    live = pos < L
    pos = pos[live]
    if pos.numel() == 0:
        return 0.0, -math.inf
    k = s["k_pages"][pages.long(), :, g].reshape(-1, D)[live]
    v = s["v_pages"][pages.long(), :, g].reshape(-1, D)[live].double()
    q = s["q"][b, g * r:(g + 1) * r]
    G = max(1, -(-L // c["W"]))
    here = L - 1
    target = here // G + (c["w0"] - c["w0"] // G if c["shift"] else 0)
    x = q.double() @ k.double().T
    if G > 1 and c["w0"] < L:
        q0 = _real(_turn(_real(_turn(q, torch.full((r,), -here, device=dev), c)), torch.full((r,), target, device=dev), c))
        k0 = _real(_turn(_real(_turn(k, -pos, c)), pos // G, c))
        x = torch.where(here - pos < c["w0"], x, q0 @ k0.T)
    x = x / math.sqrt(D)
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - lse[:, None]) @ v, lse


def exact(case, seed):
    c = case
    B, Hkv, D, P = c["B"], c["Hkv"], c["D"], c["P"]
    s = prepare(c, seed)
    lens = _lens(c)
    if c["kind"] == "norm_rope":
        pos = s["positions"]
        return {"q": _exact_heads(s["q"], s["qw"], pos, c), "k": _exact_heads(s["k"], s["kw"], pos, c)}
    if c["kind"] == "append":
        pos = s["positions"].long()
        live = torch.nonzero(pos >= 0).flatten()
        q = s["q_out"].double()
        q[live] = _exact_heads(s["q"][live], s["qw"], pos[live], c)
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        ids = s["table"][s["seq_ids"][live].long(), pos[live] // P].long()
        kp[ids, pos[live] % P] = _exact_heads(s["k"][live], s["kw"], pos[live], c)
        vp[ids, pos[live] % P] = s["v"][live].double()
        return {"q": q, "k_pages": kp, "v_pages": vp}
    if c["kind"] == "summaries":
        out = s["summaries"].double()
        for b, n in enumerate(lens):
            lo = max(0, n - 1) // P if c["step"] else 0
            full = torch.arange(lo, _pages(c, n), device="cuda")
            for part in torch.split(full, 1024):
                ids = s["table"][b, part].long()
                at = part[:, None] * P + torch.arange(P, device="cuda")
                z = _real(_turn(s["k_pages"][ids], (P // 2 - at % P)[..., None].expand(-1, -1, Hkv), c))
                z = torch.where((at < n)[..., None, None], z, torch.zeros((), dtype=torch.float64, device="cuda"))
                out[ids] = z.sum(1) / (at < n).sum(1)[:, None, None]
        return {"summaries": out}
    r = c["Hq"] // Hkv
    o = torch.zeros(B, c["Hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, c["Hq"], dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        pages = torch.arange(_pages(c, n), device="cuda")
        for h in range(Hkv):
            mine = pages
            if c["kind"] == "sparse" and n:
                G, here = max(1, -(-n // c["W"])), n - 1
                target = here // G + (c["w0"] - c["w0"] // G if c["shift"] else 0)
                first = min(max(0, n - c["w0"]) // P, here // P)
                cand = pages[c["sink"]:first]
                if cand.numel() > c["top_k"]:
                    z = _turn(s["summaries"][s["table"][b, cand].long(), h], (cand * P + P // 2) // G - (cand * P + P // 2), c)
                    q = _turn(s["q"][b, h * r:(h + 1) * r], torch.full((r,), target - here, device="cuda"), c)
                    score = (_real(q) @ _real(z).T).amax(0).float()
                    rank = torch.sort(score, descending=True, stable=True).indices
                    cand = cand[rank[:c["top_k"]].sort().values]
                mine = torch.cat([pages[:min(c["sink"], first)], cand, pages[first:]])
            o[b, h * r:(h + 1) * r], lse[b, h * r:(h + 1) * r] = _exact_rows(s, b, h, s["table"][b, mine], mine * P)
    if c["kind"] == "decode":
        return {"o": o, "lse": lse}
    return {"page_list": None, "page_counts": None, "o": o, "lse": lse}
