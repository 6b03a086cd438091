"""Measured cases of the operators around the attention and the MoE of a serving
step: the norm of the hidden states with the residual's addition and 8-bit
output, the product of 8-bit rows with 8-bit weights (a scale for each block of
128), and the attention of whole prompts, packed one after another.

``run`` computes each operator in plain torch operations, or through the
library where ``own`` is true.  ``exact`` evaluates the definition in 64 bits.

Definitions
  norm     with a residual r: r' = bf16(x + r), else r' = x;
           y = r' / sqrt(mean(r'^2) + eps) * w; out = bf16(y);
           quantised: per row and 128 columns scale = max|y| / 448 (1 for zeros),
           code = e4m3(y / scale)
  matmul   out[m, n] = bf16(sum over blocks b of 128 columns of
           sa[m, b] * sw[n / 128, b] * sum_k a[m, k] * w[n, k])
  prefill  sequence with Lq queries and Lk keys, query i at p = i + Lk - Lq:
           s_j = q . k_j * scale; with a cap, s_j = cap * tanh(s_j / cap); with
           slopes, s_j += slope_h * (j - p); over j < Lk, j <= p if causal, and
           j > p - window with a window; out = softmax(s) v,
           lse = log(sum(exp(s))); no visible key: out = 0, lse = -inf
"""
import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # one new token of a decode step: its residual stream, normed and quantised
        dict(name="norm_1_2048", op="norm", T=1, H=2048, residual=True, bf16=False, quant=True),
        # a prompt chunk of the largest hidden size; the router and the experts take the bf16 output too
        dict(name="norm_4096_6144", op="norm", T=4096, H=6144, residual=True, bf16=True, quant=True),
        # an attention output's rows quantised as they are: an odd batch, a last block of 64 columns
        dict(name="norm_777_2880", op="norm", T=777, H=2880, residual=False, bf16=False, quant=True),
        # query, key and value projection of one new token
        dict(name="matmul_1_2048_6144", op="matmul", M=1, K=2048, N=6144),
        # the same of a decode batch, wider hidden size
        dict(name="matmul_64_4096_8192", op="matmul", M=64, K=4096, N=8192),
        # an odd number of rows, ragged blocks of both kinds
        dict(name="matmul_333_2880_1000", op="matmul", M=333, K=2880, N=1000),
        # a prompt chunk's projection at the largest hidden size
        dict(name="matmul_4096_6144_8192", op="matmul", M=4096, K=6144, N=8192),
        # one short prompt: latency
        dict(name="prefill_b1_100", op="prefill", B=1, S=100, past=0, nh=16, nkv=16, d=128, causal=True, window=0, cap=0.0, slopes=False),
        # prompts of different lengths packed into one call, grouped heads
        dict(name="prefill_b12_2048", op="prefill", B=12, S=2048, past=0, nh=32, nkv=8, d=128, causal=True, window=0, cap=0.0, slopes=False),
        # one long prompt
        dict(name="prefill_b1_16384", op="prefill", B=1, S=16384, past=0, nh=32, nkv=8, d=128, causal=True, window=0, cap=0.0, slopes=False),
        # chunks of prompts whose earlier tokens are in the cache: capped scores, a window, wide heads
        dict(name="prefill_b4_chunk_cap", op="prefill", B=4, S=1000, past=5000, nh=16, nkv=8, d=256, causal=True, window=4096, cap=50.0, slopes=False),
        # many short prompts, small heads in odd groups, distance bias
        dict(name="prefill_b60_slopes", op="prefill", B=60, S=700, past=0, nh=21, nkv=7, d=64, causal=True, window=0, cap=0.0, slopes=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "matmul", "matmul", "prefill", "prefill", "prefill"])
    if op == "norm":
        bf16 = rng.random() < 0.5
        return dict(op=op, T=_log_int(rng, 1, 4000), H=8 * _log_int(rng, 16, 768), residual=rng.random() < 0.6,
                    bf16=bf16, quant=not bf16 or rng.random() < 0.5)
    if op == "matmul":
        return dict(op=op, M=_log_int(rng, 1, 4000), K=16 * _log_int(rng, 8, 380), N=8 * _log_int(rng, 8, 1000))
    B, d = _log_int(rng, 1, 64), rng.choice([64, 128, 128, 256])
    nkv = rng.choice([1, 2, 4, 5, 8, 16])
    nh = min(64 // nkv, rng.choice([1, 2, 3, 4, 7, 8, 12, 16])) * nkv
    # at most a quarter of the largest listed case's query-key pairs
    pairs = 16384 * 16384 * 32 * 128 // (8 * B * nh * d)
    S = _log_int(rng, 1, min(12000, int(math.sqrt(pairs))))
    past = rng.choice([0, 0, 0, rng.randrange(1, 4000)])
    if S * past > pairs:
        past = 0
    return dict(op=op, B=B, S=S, past=past, nh=nh, nkv=nkv, d=d, causal=rng.random() < 0.85, window=rng.choice([0, 0, 0, 1, 100, 1024]),
                cap=rng.choice([0.0, 0.0, 30.0]), slopes=rng.random() < 0.25)


def _lengths(case):
    """(queries, keys) of each sequence: a long one of S queries, the others
    spread over the range, one empty in a larger batch; every sequence but the
    first has its own share of earlier keys."""
    B, S, past = case["B"], case["S"], case["past"]
    lens = []
    for b in range(B):
        n = max(1, math.ceil(S * (1.0 - b * 0.6180339887498949 % 1.0)))
        if B >= 12 and b in (5, 9):
            n = 0 if b == 5 else 1
        lens.append((n, n + math.ceil(past * (1.0 - b * 0.7548776662466927 % 1.0))))
    return lens


def _seen(case, n, m):
    """Visible (query, key) pairs of a sequence of n queries and m keys."""
    w = case["window"]
    if not case["causal"]:
        if not w:
            return n * m
        return sum(m - max(0, i + m - n - w + 1) for i in range(n))
    last = [i + m - n + 1 for i in range(n)]
    return sum(min(t, w) if w else t for t in last)


def work(case):
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        row = 2 * H + 4 * H * case["residual"] + 2 * H * case["bf16"] + (H + 4 * -(-H // 128)) * case["quant"]
        return dict(bytes=T * row + 4 * H, flops=6 * T * H)
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        blocks = -(-K // 128)
        return dict(bytes=M * K + N * K + 4 * blocks * (M + -(-N // 128)) + 2 * M * N, flops=2 * M * N * K)
    nh, nkv, d = case["nh"], case["nkv"], case["d"]
    lens = _lengths(case)
    q, k = sum(n for n, _ in lens), sum(m for n, m in lens if n)
    return dict(bytes=q * nh * (4 * d + 4) + k * nkv * 4 * d, flops=4 * d * nh * sum(_seen(case, n, m) for n, m in lens))


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * scale

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=dev)

    op = case["op"]
    st = dict(case=case)
    if op == "norm":
        T, H = case["T"], case["H"]
        # rows of different sizes, a few columns much larger than the others, as hidden states have them
        column = torch.where(torch.rand(H, generator=gen, device=dev) < 0.005, 30.0, 1.0)
        st["x"] = (randn(T, H) * torch.exp(0.5 * randn(T, 1)) * column).to(torch.bfloat16)
        st["weight"] = 1.0 + randn(H, scale=0.2)
        if case["residual"]:
            st["residual"] = (randn(T, H, scale=2.0) * column).to(torch.bfloat16)
            st["sum"] = empty(T, H)
        if case["bf16"]:
            st["out"] = empty(T, H)
        if case["quant"]:
            st["codes"] = empty(T, H, dtype=torch.uint8)
            st["scales"] = empty(-(-H // 128), T, dtype=torch.float32).t()
    elif op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        blocks = -(-K // 128)
        # codes of rows whose largest value sits near the top of the format, as quantised activations are
        st["a"] = randn(M, K, scale=120.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        st["sa"] = (0.01 * torch.exp(0.5 * randn(blocks, M))).t()
        st["w"] = randn(N, K, scale=120.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        st["sw"] = 0.0002 * torch.exp(0.2 * randn(-(-N // 128), blocks))
        st["out"] = empty(M, N)
    else:
        nh, nkv, d = case["nh"], case["nkv"], case["d"]
        lens = _lengths(case)
        Tq, Tk = sum(n for n, _ in lens), sum(m for _, m in lens)
        if case["past"]:  # keys and values read back from a cache
            st["q"] = randn(Tq, nh, d, scale=1.5).to(torch.bfloat16)
            st["k"], st["v"] = randn(Tk, nkv, d).to(torch.bfloat16), randn(Tk, nkv, d).to(torch.bfloat16)
        else:  # queries, keys and values lie side by side in one projection's rows
            fused = randn(Tq, nh + 2 * nkv, d).to(torch.bfloat16)
            st["q"], st["k"], st["v"] = fused[:, :nh], fused[:, nh:nh + nkv], fused[:, nh + nkv:]
        starts = torch.tensor([[0, 0]] + [list(x) for x in lens]).cumsum(0).to(torch.int32)
        st["q_starts"], st["k_starts"] = starts[:, 0].contiguous().to(dev), starts[:, 1].contiguous().to(dev)
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / nh) for h in range(nh)], device=dev) if case["slopes"] else None
        st["out"], st["lse"] = empty(Tq, nh, d), empty(Tq, nh, dtype=torch.float32)
        st["lens"] = lens
    if own:
        from fp8_routed_expert_gb300 import DecodeAttention, Projection
        if op == "prefill":
            st["attn"] = DecodeAttention(case["nh"], case["nkv"], case["d"])
        else:
            st["proj"] = Projection()
    return st


# -------------------------------------------------------------- plain forms

def _blocks(x):
    """f32 [T, H] as [T, blocks, 128], zeros behind the last column."""
    T, H = x.shape
    x = torch.nn.functional.pad(x, (0, -H % 128))
    return x.view(T, -1, 128)


def _norm_plain(st):
    case = st["case"]
    res = {}
    x = st["x"]
    if case["residual"]:
        x = (x.float() + st["residual"].float()).to(torch.bfloat16)
        res["residual"] = x
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * st["weight"]
    if case["bf16"]:
        res["out"] = y.to(torch.bfloat16)
    if case["quant"]:
        b = _blocks(y)
        amax = b.abs().amax(-1)
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        codes = (b / scale[..., None]).to(torch.float8_e4m3fn)
        res["codes"], res["scales"] = codes.view(y.shape[0], -1)[:, :y.shape[1]], scale
    return res


def _matmul_plain(st):
    K = st["a"].shape[1]
    a = st["a"].view(torch.float8_e4m3fn).float() * st["sa"].repeat_interleave(128, 1)[:, :K]
    sw = st["sw"].repeat_interleave(128, 0)[:st["w"].shape[0]].repeat_interleave(128, 1)[:, :K]
    return (a @ (st["w"].view(torch.float8_e4m3fn).float() * sw).t()).to(torch.bfloat16)


def _prefill_plain(st):
    case = st["case"]
    nh, nkv, d = case["nh"], case["nkv"], case["d"]
    g = nh // nkv
    q, k, v = (st[n].float().transpose(0, 1) for n in "qkv")
    slopes = None if st["slopes"] is None else st["slopes"].view(nkv, g, 1, 1)
    out = torch.empty(nkv, g, q.shape[1], d, dtype=torch.bfloat16, device=q.device)
    lse = torch.empty(nkv, g, q.shape[1], device=q.device)
    q0 = k0 = 0
    for n, m in st["lens"]:
        step = max(1, (1 << 28) // (nh * max(m, 1)))  # queries at a time: about 1 GB of scores
        for a in range(0, n, step):
            e = min(n, a + step)
            # keys that any of these queries sees
            hi = max(0, min(m, e + m - n)) if case["causal"] else m
            lo = max(0, a + m - n - case["window"] + 1) if case["window"] else 0
            lo = min(lo, hi)
            s = torch.matmul(q[:, q0 + a:q0 + e].reshape(nkv, g * (e - a), d), k[:, k0 + lo:k0 + hi].transpose(1, 2)) / math.sqrt(d)
            s = s.view(nkv, g, e - a, hi - lo)
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            j = torch.arange(lo, hi, device=s.device)[None, :]
            p = torch.arange(a + m - n, e + m - n, device=s.device)[:, None]
            if slopes is not None:
                s = s + slopes * (j - p).float()
            hidden = torch.zeros(e - a, hi - lo, dtype=torch.bool, device=s.device)
            if case["causal"]:
                hidden |= j > p
            if case["window"]:
                hidden |= j <= p - case["window"]
            s = s.masked_fill(hidden, -math.inf)
            top = s.amax(-1, keepdim=True) if hi > lo else torch.full_like(s[..., :1].sum(-1, keepdim=True), -math.inf)
            ref = torch.where(top == -math.inf, torch.zeros_like(top), top)
            w = torch.exp(s - ref)
            total = w.sum(-1, keepdim=True)
            o = torch.matmul(w.view(nkv, g * (e - a), hi - lo), v[:, k0 + lo:k0 + hi]).view(nkv, g, e - a, d)
            out[:, :, q0 + a:q0 + e] = (o / torch.where(total > 0, total, torch.ones_like(total))).to(torch.bfloat16)
            lse[:, :, q0 + a:q0 + e] = (torch.log(total) + ref)[..., 0]
        q0, k0 = q0 + n, k0 + m
    return out.view(nh, -1, d).transpose(0, 1), lse.view(nh, -1).t()


def run(st):
    case = st["case"]
    op = case["op"]
    if op == "norm":
        if not own:
            return _norm_plain(st)
        residual = {}
        if case["residual"]:
            residual = dict(residual=st["residual"], residual_out=st["sum"])
        if case["quant"]:
            codes, scales = st["proj"].norm_quant(st["x"], st["weight"], eps=EPS, codes=st["codes"], scales=st["scales"],
                                                  out=st.get("out"), **residual)
            res = dict(codes=codes.view(torch.float8_e4m3fn), scales=scales)
            if case["bf16"]:
                res["out"] = st["out"]
        else:
            res = dict(out=st["proj"].norm(st["x"], st["weight"], eps=EPS, out=st["out"], **residual))
        if case["residual"]:
            res["residual"] = st["sum"]
        return res
    if op == "matmul":
        if own:
            return dict(out=st["proj"].matmul(st["a"], st["sa"], st["w"], st["sw"], out=st["out"]))
        return dict(out=_matmul_plain(st))
    if own:
        out, lse = st["attn"].prefill(st["q"], st["k"], st["v"], st["q_starts"], st["k_starts"], causal=case["causal"], softcap=case["cap"],
                                      slopes=st["slopes"], window=case["window"], out=st["out"], lse=st["lse"])
    else:
        out, lse = _prefill_plain(st)
    return dict(out=out, lse=lse)


# ------------------------------------------------- definitions in 64 bits

def _exact_prefill(st):
    case = st["case"]
    nh, nkv, d, w = case["nh"], case["nkv"], case["d"], case["window"]
    g = nh // nkv
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device=out.device)
    q0 = k0 = 0
    for n, m in st["lens"]:
        for c in range(nkv):
            K, V = st["k"][k0:k0 + m, c].double(), st["v"][k0:k0 + m, c].double()
            for h in range(c * g, c * g + g):
                for i0 in range(0, n, 4096):
                    i = torch.arange(i0, min(n, i0 + 4096), device=out.device)
                    # key j at distance p - j >= 0 from the query in the causal case
                    top = min(m, int(i[-1]) + m - n + 1) if case["causal"] else m
                    first = max(0, i0 + m - n - w + 1) if w else 0
                    if first >= top:
                        continue
                    dist = (i + (m - n))[:, None] - torch.arange(first, top, device=out.device)[None, :]
                    rows = st["q"][q0 + i0:q0 + i0 + len(i), h].double()
                    s = torch.einsum("id,jd->ij", rows, K[first:top]) * d ** -0.5
                    if case["cap"]:
                        s = torch.tanh(s / case["cap"]) * case["cap"]
                    if st["slopes"] is not None:
                        s = s - st["slopes"][h].double() * dist
                    if case["causal"]:
                        s[dist < 0] = -math.inf
                    if w:
                        s[dist >= w] = -math.inf
                    z = torch.logsumexp(s, 1)
                    lse[q0 + i, h] = z
                    p = torch.exp(s - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
                    out[q0 + i, h] = p @ V[first:top]
        q0, k0 = q0 + n, k0 + m
    return dict(out=out, lse=lse)


def exact(case, seed):
    # about 20 seconds of 64-bit products
    if work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    if case["op"] == "prefill":
        return _exact_prefill(st)
    if case["op"] == "matmul":
        out = torch.zeros(case["M"], case["N"], dtype=torch.float64, device=st["a"].device)
        a, w = st["a"].view(torch.float8_e4m3fn).to(torch.float64), st["w"].view(torch.float8_e4m3fn).to(torch.float64)
        rows = torch.arange(case["N"], device=a.device) // 128
        for b in range(-(-case["K"] // 128)):
            c = slice(128 * b, min(128 * b + 128, case["K"]))
            out += (a[:, c] * st["sa"][:, b:b + 1].double()) @ (w[:, c] * st["sw"][rows, b].double()[:, None]).t()
        return dict(out=out)
    res = {}
    x = st["x"].double()
    if case["residual"]:
        x = x + st["residual"].double()
        res["residual"] = x
        x = x.to(torch.bfloat16).double()
    y = st["weight"].double() * x / ((x * x).sum(1, keepdim=True) / case["H"] + EPS).sqrt()
    if case["bf16"]:
        res["out"] = y
    if case["quant"]:
        codes, scales = torch.empty_like(y), []
        for c in range(0, case["H"], 128):
            part = y[:, c:c + 128]
            s = part.abs().max(1).values / 448.0
            s = torch.where(s == 0, torch.ones_like(s), s)
            codes[:, c:c + 128] = part / s[:, None]
            scales.append(s)
        res["codes"], res["scales"] = codes, torch.stack(scales, 1)
    return res
