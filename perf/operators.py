"""Measured cases of the attention sub-block's serving operators: per-head
query/key norm with rotation, the paged key/value cache (bf16 or e4m3) as it
is written and read back, and the attention of one new token over it.

``run`` computes each operator in plain torch operations, or through the
library where ``own`` is true.  ``exact`` evaluates the definition in 64 bits.

Definitions (d = head size, all per head):
  norm    y = x / sqrt(mean(x^2) + eps) * w
  rotate  the first R of the d elements, in pairs (i, i + R/2), or (2i, 2i+1)
          when interleaved, by the angle position * freq[i]
  e4m3    a row v is kept as codes c and a scale 2^e: e is the smallest
          integer with max|v| <= 448 * 2^e, c = e4m3(v / 2^e)
  attend  s_j = q . k_j * scale; with a cap, s_j = cap * tanh(s_j / cap); with
          slopes, s_j += slope_h * (j - (len - 1)); over j in [lo, len), lo the
          larger of start and len - window; out = softmax(s) v,
          lse = log(sum(exp(s)));
          no visible key: out = 0, lse = -inf
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
SLOT_SPREAD = 3  # the written tokens' cache has this many times their slots


def listed():
    return [
        # one new token of one sequence, its query heads and one key/value row
        # per head put into a bf16 cache: the smallest call of a decode step
        dict(name="append_1_bf16", op="append", T=1, nh=16, nkv=16, d=128, rot=128, inter=False, fmt="bf16", page=16),
        # a decode batch at far positions into an e4m3 cache, with read-back
        dict(name="append_64_e4m3", op="append", T=64, nh=32, nkv=8, d=128, rot=128, inter=False, fmt="e4m3", page=32),
        # a prompt chunk: norm and rotation of all its queries and keys
        dict(name="norm_rope_4096", op="norm_rope", T=4096, nh=48, nkv=8, d=128, rot=128, inter=False),
        # an odd batch, interleaved pairs, half of each head rotated
        dict(name="norm_rope_777_half", op="norm_rope", T=777, nh=16, nkv=16, d=64, rot=32, inter=True),
        # a prompt's keys and values quantised into pages and read back
        dict(name="cache_e4m3_8192", op="cache", T=8192, nkv=8, d=128, fmt="e4m3", page=64),
        # a short prompt of odd length into small pages, wide heads
        dict(name="cache_e4m3_333", op="cache", T=333, nkv=4, d=256, fmt="e4m3", page=8),
        # one sequence at a short context: latency
        dict(name="decode_b1_1000", op="decode", B=1, S=1000, nh=16, nkv=16, d=128, fmt="bf16", page=16, cap=0.0, slopes=False, window=0, starts=False),
        # the decode batch of eight at 4096 tokens of context, one key head per query head
        dict(name="decode_b8_4096", op="decode", B=8, S=4096, nh=16, nkv=16, d=128, fmt="bf16", page=64, cap=0.0, slopes=False, window=0, starts=False),
        # a serving batch with ragged contexts, grouped heads, e4m3 cache
        dict(name="decode_b64_8192_e4m3", op="decode", B=64, S=8192, nh=32, nkv=8, d=128, fmt="e4m3", page=32, cap=0.0, slopes=False, window=0, starts=False),
        # one very long context with one key/value head: all of the work is one row's
        dict(name="decode_b1_200001_mqa", op="decode", B=1, S=200001, nh=16, nkv=1, d=128, fmt="e4m3", page=128, cap=0.0, slopes=False, window=0, starts=False),
        # capped scores within a window, wide heads, documents that begin inside the cache
        dict(name="decode_b24_cap_window", op="decode", B=24, S=6000, nh=16, nkv=8, d=256, fmt="bf16", page=16, cap=50.0, slopes=False, window=4096, starts=True),
        # many short sequences, distance bias, small heads
        dict(name="decode_b200_slopes", op="decode", B=200, S=700, nh=24, nkv=6, d=64, fmt="bf16", page=24, cap=0.0, slopes=True, window=0, starts=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "norm_rope", "cache", "decode", "decode", "decode"])
    d = rng.choice([64, 128, 128, 256])
    nkv = rng.choice([1, 2, 4, 5, 8, 16])
    nh = nkv * rng.choice([1, 2, 3, 4, 7, 8, 12, 16])
    fmt = rng.choice(["bf16", "e4m3"])
    page = rng.choice([1, 8, 16, 24, 32, 64, 100, 128, 256])
    if op in ("append", "norm_rope"):
        nh = min(nh, 64 // nkv * nkv)
        rot = rng.choice([d, d, d // 2, d // 4])
        case = dict(op=op, T=_log_int(rng, 1, 2500), nh=nh, nkv=nkv, d=d, rot=rot, inter=rng.random() < 0.3)
        return case | (dict(fmt=fmt, page=page) if op == "append" else {})
    if op == "cache":
        return dict(op=op, T=_log_int(rng, 1, 8000), nkv=min(nkv, 8), d=min(d, 128), fmt=fmt, page=page)
    B = _log_int(rng, 1, 256)
    # at most a third of the largest listed case's keys
    most = 64 * 8192 * 8 * 128 // (3 * B * nkv * d)
    S = _log_int(rng, 1, max(1, min(100000, most)))
    return dict(op=op, B=B, S=S, nh=nh, nkv=nkv, d=d, fmt=fmt, page=page, cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                slopes=rng.random() < 0.3, window=rng.choice([0, 0, 0, 1, 128, 1000]), starts=rng.random() < 0.3)


def _spans(case):
    """(length, first visible position) of each sequence: a long one of S
    tokens, the others spread over the whole range, a few empty or of one
    token in a larger batch."""
    B, S = case["B"], case["S"]
    frac = (np.arange(B) * 0.6180339887498949) % 1.0
    lens = np.maximum(1, np.ceil(S * (1.0 - frac))).astype(np.int64)
    if B >= 16:
        lens[5], lens[11] = 0, 1
    starts = np.zeros(B, np.int64)
    if case["starts"]:
        starts = (lens * ((np.arange(B) * 0.7548776662466927) % 1.0) * 0.6).astype(np.int64)
        if B >= 16:
            starts[7] = lens[7]  # everything masked
    lo = starts
    if case["window"]:
        lo = np.maximum(lo, lens - case["window"])
    return lens, starts, np.minimum(lo, lens)


def work(case):
    op, d = case["op"], case["d"]
    if op == "decode":
        lens, _, lo = _spans(case)
        keys = int((lens - lo).sum())
        row = 2 * d if case["fmt"] == "bf16" else d + 4
        io = case["B"] * case["nh"] * (4 * d + 4)
        return dict(bytes=2 * keys * case["nkv"] * row + io, flops=4 * keys * case["nh"] * d)
    T, nkv = case["T"], case["nkv"]
    if op == "cache":
        # bf16 rows in, the cache's rows written and read, bf16 rows out
        row = 2 * d if case["fmt"] == "bf16" else d + 4
        return dict(bytes=2 * T * nkv * (2 * d + 2 * row + 2 * d), flops=4 * T * nkv * d)
    n = T * (case["nh"] + nkv)
    bytes_ = n * 4 * d
    if op == "append":
        bytes_ = T * case["nh"] * 4 * d + 2 * T * nkv * (2 * d + (2 * d if case["fmt"] == "bf16" else d + 4 + (d + 4) + 2 * d))
    return dict(bytes=bytes_, flops=8 * n * d)


# ------------------------------------------------------------------ inputs

def _rows(gen, n, heads, d, dev):
    """bf16 rows whose size differs from row to row, as projections give them."""
    x = torch.randn(n, heads, d, generator=gen, device=dev)
    return x * torch.exp(0.5 * torch.randn(n, heads, 1, generator=gen, device=dev))


def _freqs(case):
    R = case["rot"]
    return 10000.0 ** (-np.arange(R // 2, dtype=np.float64) * 2.0 / R)


def _empty_cache(n_pages, page, nkv, d, fmt, dev):
    if fmt == "bf16":
        k = torch.zeros(n_pages, nkv, page, d, dtype=torch.bfloat16, device=dev)
        return [k, torch.zeros_like(k), None, None]
    k = torch.zeros(n_pages, nkv, page, d, dtype=torch.uint8, device=dev)
    s = torch.ones(n_pages, nkv, page, dtype=torch.float32, device=dev)
    return [k, torch.zeros_like(k), s, torch.ones_like(s)]


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, d, nkv = case["op"], case["d"], case["nkv"]
    st = dict(case=case)
    if op == "decode":
        B, page, fmt = case["B"], case["page"], case["fmt"]
        lens, starts, _ = _spans(case)
        width = max(1, -(-int(lens.max()) // page))
        used = (lens + page - 1) // page
        n_pages = int(used.sum()) + 3
        order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
        # a sequence's pages in its row, the rest of the row left at page 0
        first = torch.from_numpy(np.concatenate([[0], np.cumsum(used)[:-1]])).to(dev)
        col = torch.arange(width, device=dev)[None, :]
        mine = col < torch.from_numpy(used).to(dev)[:, None]
        st["table"] = torch.where(mine, order[(first[:, None] + col).clamp(max=n_pages - 1)], torch.zeros((), dtype=torch.int32, device=dev)).contiguous()
        st["lens"] = torch.from_numpy(lens.astype(np.int32)).to(dev)
        st["starts"] = torch.from_numpy(starts.astype(np.int32)).to(dev) if case["starts"] else None
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / case["nh"]) for h in range(case["nh"])], device=dev) if case["slopes"] else None
        st["q"] = (1.5 * torch.randn(B, case["nh"], d, generator=gen, device=dev)).to(torch.bfloat16)
        cache = []
        for _ in range(2):
            if fmt == "bf16":
                cache.append(torch.empty(n_pages, nkv, page, d, dtype=torch.bfloat16, device=dev).normal_(generator=gen))
            else:
                # codes of normal rows whose largest value sits near the top of the format
                x = torch.empty(n_pages, nkv, page, d, dtype=torch.bfloat16, device=dev).normal_(0.0, 100.0, generator=gen)
                cache.append(x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        scales = [None, None]
        if fmt == "e4m3":
            scales = [torch.exp2(torch.randint(-8, -5, (n_pages, nkv, page), generator=gen, device=dev).float()) for _ in range(2)]
        st["cache"] = cache + scales
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(B, case["nh"], dtype=torch.float32, device=dev)
        if own:
            from fp8_routed_expert_gb300 import DecodeAttention, PagedKVCache
            st["attn"] = DecodeAttention(case["nh"], nkv, d)
            st["kv"] = PagedKVCache(*st["cache"])
        return st
    T = case["T"]
    if op != "cache":
        nh = case["nh"]
        # queries, keys and values lie side by side in one projection's rows
        fused = _rows(gen, T, nh + 2 * nkv, d, dev).to(torch.bfloat16)
        st["q"], st["k"], st["v"] = fused[:, :nh], fused[:, nh:nh + nkv], fused[:, nh + nkv:]
        st["wq"] = 1.0 + 0.2 * torch.randn(d, generator=gen, device=dev)
        st["wk"] = 1.0 + 0.2 * torch.randn(d, generator=gen, device=dev)
        st["freqs"] = torch.from_numpy(_freqs(case)).to(dev)
        if op == "append":  # each token belongs to another sequence
            st["pos"] = torch.randint(0, 1 << 20, (T,), generator=gen, device=dev, dtype=torch.int32)
        else:  # a chunk of one sequence
            st["pos"] = (torch.arange(T, device=dev) + torch.randint(0, 1 << 20, (1,), generator=gen, device=dev)).to(torch.int32)
            st["qo"] = torch.empty(T, nh, d, dtype=torch.bfloat16, device=dev)
            st["ko"] = torch.empty(T, nkv, d, dtype=torch.bfloat16, device=dev)
    else:
        nh = nkv
        kv = _rows(gen, T, 2 * nkv, d, dev).to(torch.bfloat16)
        st["k"], st["v"] = kv[:, :nkv], kv[:, nkv:]
    if op != "norm_rope":
        page = case["page"]
        n_pages = -(-T * SLOT_SPREAD // page)
        st["cache"] = _empty_cache(n_pages, page, nkv, d, case["fmt"], dev)
        if op == "append":
            st["slots"] = torch.randperm(n_pages * page, generator=gen, device=dev)[:T].contiguous()
            st["qo"] = torch.empty(T, nh, d, dtype=torch.bfloat16, device=dev)
        else:  # whole pages in an order of their own
            pages = torch.randperm(n_pages, generator=gen, device=dev)
            at = torch.arange(T, device=dev)
            st["slots"] = (pages[at // page] * page + at % page).contiguous()
        st["ko"] = torch.empty(T, nkv, d, dtype=torch.bfloat16, device=dev)
        st["vo"] = torch.empty(T, nkv, d, dtype=torch.bfloat16, device=dev)
    if own:
        from fp8_routed_expert_gb300 import DecodeAttention, PagedKVCache
        rope = dict(rope_freqs=_freqs(case), interleaved=case["inter"]) if op != "cache" else {}
        st["attn"] = DecodeAttention(nh, nkv, d, **rope)
        if op != "norm_rope":
            st["kv"] = PagedKVCache(*st["cache"])
    return st


# -------------------------------------------------------------- plain forms

def _norm_rotate(x, w, pos, freqs, inter):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    R = 2 * freqs.numel()
    angle = pos.double()[:, None, None] * freqs
    cos, sin = angle.cos().float(), angle.sin().float()
    if inter:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., R:]], -1)


def _store(cache, scales, x, slots):
    """Rows x (f32) into their slots."""
    page = cache.shape[2]
    at = (slots // page, slice(None), slots % page)
    if scales is None:
        cache[at] = x.to(cache.dtype)
        return
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), torch.zeros_like(e)).clamp(-126, 127)
    scale = torch.ldexp(torch.ones_like(amax), e)
    cache[at] = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scales[at] = scale


def _load(cache, scales, slots):
    page = cache.shape[2]
    at = (slots // page, slice(None), slots % page)
    if scales is None:
        return cache[at].float()
    return cache[at].view(torch.float8_e4m3fn).float() * scales[at][..., None]


def _gather(cache, scales, table):
    """[pages, heads, page, d] -> f32 [B, heads, width * page, d]."""
    x = cache[table.long()]
    x = x.float() if scales is None else x.view(torch.float8_e4m3fn).float() * scales[table.long()][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _decode_plain(st):
    case = st["case"]
    nkv, d = case["nkv"], case["d"]
    q = st["q"].float()
    B, nh, _ = q.shape
    K = _gather(st["cache"][0], st["cache"][2], st["table"])
    s = torch.matmul(q.view(B, nkv, nh // nkv, d), K.transpose(-1, -2)) / math.sqrt(d)
    del K
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    j = torch.arange(s.shape[-1], device=s.device)[None, :]
    n = st["lens"][:, None]
    if st["slopes"] is not None:
        s = s + st["slopes"].view(1, nkv, -1, 1) * (j - (n - 1)).float()[:, None, None, :]
    seen = j < n
    if st["starts"] is not None:
        seen = seen & (j >= st["starts"][:, None])
    if case["window"]:
        seen = seen & (j >= n - case["window"])
    s = s.masked_fill(~seen[:, None, None, :], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    V = _gather(st["cache"][1], st["cache"][3], st["table"])
    o = torch.matmul(p, V) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.log(total) + top
    return o.reshape(B, nh, d).to(torch.bfloat16), lse.reshape(B, nh)


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        attn = st["attn"]
        if op == "decode":
            out, lse = attn.decode(st["q"], st["kv"], st["table"], st["lens"], softcap=case["cap"], slopes=st["slopes"],
                                   window=case["window"], starts=st["starts"], out=st["out"], lse=st["lse"])
            return dict(out=out, lse=lse)
        if op == "norm_rope":
            q, k = attn.norm_rope(st["q"], st["k"], st["pos"], st["wq"], st["wk"], eps=EPS, q_out=st["qo"], k_out=st["ko"])
            return dict(q=q, k=k)
        if op == "append":
            q = attn.append(st["q"], st["k"], st["v"], st["pos"], st["slots"], st["kv"], st["wq"], st["wk"], eps=EPS, q_out=st["qo"])
            if case["fmt"] == "bf16":
                return dict(q=q, k=st["cache"][0], v=st["cache"][1])
            k, v = attn.read(st["kv"], st["slots"], k_out=st["ko"], v_out=st["vo"])
            return dict(q=q, k=k, v=v)
        attn.write(st["kv"], st["k"], st["v"], st["slots"])
        k, v = attn.read(st["kv"], st["slots"], k_out=st["ko"], v_out=st["vo"])
        return dict(k=k, v=v)
    if op == "decode":
        out, lse = _decode_plain(st)
        return dict(out=out, lse=lse)
    if op == "norm_rope":
        return dict(q=_norm_rotate(st["q"], st["wq"], st["pos"], st["freqs"], case["inter"]).to(torch.bfloat16),
                    k=_norm_rotate(st["k"], st["wk"], st["pos"], st["freqs"], case["inter"]).to(torch.bfloat16))
    kc, vc, ks, vs = st["cache"]
    if op == "append":
        q = _norm_rotate(st["q"], st["wq"], st["pos"], st["freqs"], case["inter"]).to(torch.bfloat16)
        _store(kc, ks, _norm_rotate(st["k"], st["wk"], st["pos"], st["freqs"], case["inter"]), st["slots"])
        _store(vc, vs, st["v"].float(), st["slots"])
        if case["fmt"] == "bf16":
            return dict(q=q, k=kc, v=vc)
        return dict(q=q, k=_load(kc, ks, st["slots"]).to(torch.bfloat16), v=_load(vc, vs, st["slots"]).to(torch.bfloat16))
    _store(kc, ks, st["k"].float(), st["slots"])
    _store(vc, vs, st["v"].float(), st["slots"])
    return dict(k=_load(kc, ks, st["slots"]).to(torch.bfloat16), v=_load(vc, vs, st["slots"]).to(torch.bfloat16))


# ------------------------------------------------- definitions in 64 bits

def _exact_turn(x, w, pos, case):
    """Complex multiplication of the pairs by exp(i * position * freq)."""
    x = x.double()
    y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    R = case["rot"]
    f = torch.from_numpy(_freqs(case)).to(x.device)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos.double()[:, None] * f)[:, None, :]
    i = torch.arange(R // 2, device=x.device)
    first, second = (2 * i, 2 * i + 1) if case["inter"] else (i, i + R // 2)
    z = torch.complex(y[..., first], y[..., second]) * turn
    out = y.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_kept(x, fmt):
    """What the cache holds for rows x (f64), as the values it stands for;
    for bf16 the unrounded values."""
    if fmt == "bf16":
        return x
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.full_like(amax, 448.0)) / 448.0))
    y = x * torch.exp2(-e)
    # the logarithm may be off by one unit at a border
    e = e + (amax * torch.exp2(-e) > 448.0).double() - (amax * torch.exp2(-(e - 1)) <= 448.0).double() * (amax > 0).double()
    y = x * torch.exp2(-e)
    _, b = torch.frexp(y)
    step = torch.exp2((b - 1).clamp(min=-6).double() - 3.0)
    return torch.round(y / step) * step * torch.exp2(e)


def exact(case, seed):
    st = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "norm_rope":
        return dict(q=_exact_turn(st["q"], st["wq"], st["pos"], case), k=_exact_turn(st["k"], st["wk"], st["pos"], case))
    if op in ("append", "cache"):
        k = _exact_turn(st["k"], st["wk"], st["pos"], case) if op == "append" else st["k"].double()
        k, v = _exact_kept(k, case["fmt"]), _exact_kept(st["v"].double(), case["fmt"])
        if op == "cache":
            return dict(k=k, v=v)
        q = _exact_turn(st["q"], st["wq"], st["pos"], case)
        if case["fmt"] == "bf16":
            whole = [c.double() for c in st["cache"][:2]]
            for t, slot in enumerate(st["slots"].tolist()):
                p, r = divmod(slot, case["page"])
                whole[0][p, :, r], whole[1][p, :, r] = k[t], v[t]
            k, v = whole
        return dict(q=q, k=k, v=v)
    nh, nkv, page = case["nh"], case["nkv"], case["page"]
    g = nh // nkv
    lens, _, lo = _spans(case)
    out = torch.zeros(case["B"], nh, d, dtype=torch.float64, device=st["q"].device)
    lse = torch.full((case["B"], nh), -math.inf, dtype=torch.float64, device=out.device)

    def rows(which, pages, a, n):
        x, sc = st["cache"][which], st["cache"][which + 2]
        x = x[pages] if sc is None else x[pages].view(torch.float8_e4m3fn)
        x = x.double() if sc is None else x.float().double() * sc[pages].double()[..., None]
        return x.permute(1, 0, 2, 3).reshape(nkv, -1, d)[:, a:a + n]

    for b in range(case["B"]):
        a, n = int(lo[b]), int(lens[b])
        if a >= n:
            continue
        first = a // page
        pages = st["table"][b, first:-(-n // page)].long()
        K, V = rows(0, pages, a - first * page, n - a), rows(1, pages, a - first * page, n - a)
        s = torch.einsum("cgd,cjd->cgj", st["q"][b].double().view(nkv, g, d), K) * d ** -0.5
        if case["cap"]:
            s = torch.tanh(s / case["cap"]) * case["cap"]
        if st["slopes"] is not None:
            s = s - st["slopes"].double().view(nkv, g, 1) * torch.arange(n - 1 - a, -1, -1, device=s.device, dtype=torch.float64)
        lse[b] = torch.logsumexp(s, -1).reshape(nh)
        out[b] = torch.einsum("cgj,cjd->cgd", torch.softmax(s, -1), V).reshape(nh, d)
    return dict(out=out, lse=lse)
