"""Norm, quantisation and 8-bit products on the GPU against the f64 oracle.

Tolerances, from the arithmetic (u = 2^-24, half a step of f32):
  * norm: the mean of H squares is off by at most 32 + 5 + 16 additions' u, halved by
    the root, and about four more roundings: 32 u of |y|; bf16 outputs half a step,
    2^-8 |y|, more;
  * scales: 34 u of the block's largest value (one division more);
  * codes: half a step of e4m3 about the quotient of the exact value and the scale
    that was written, and the value's 34 u: 2^-4 of the value, or 2^-10 below the
    normal range;
  * products: f32 sums of exact products, 32 at a time on the matrix unit (each step
    charged 8 u of the magnitudes), then a product and a sum per block of 128 and per
    CTA of a cluster: (K / 4 + K / 64 + 24) u of the magnitudes, half a step 2^-8 of
    the output.
"""
import ctypes

import numpy as np
import pytest
import torch

from fp8_routed_expert_gb300 import DecodeAttention, MoELayer, Projection
from harness import check_output
from oracle import E4M3_TABLE, moe_forward
from oracle import projection as P
from test_gpu_prefill import check as check_prompts

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEV = torch.device("cuda", 0)
TABLE = np.asarray(E4M3_TABLE, np.float64)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def proj(_built):
    return Projection()


def f64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def rows(g, T, H, size=1.0):
    x = torch.randn(T, H, generator=g, device=DEV) * torch.exp(torch.randn(T, 1, generator=g, device=DEV)) * size
    return x.to(torch.bfloat16)


def close(got, want, tol):
    got = f64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4], tol[bad][:4])


def check_codes(codes, scales, y):
    """codes and scales against exact values y (f64)."""
    want = P.block_scales(y)
    close(scales, want, 34 * U * want)
    s = P.spread(f64(scales), y.shape[1])
    c = TABLE[codes.cpu().numpy()]
    close(torch.from_numpy(c), y / s, np.maximum(2.0 ** -4 * np.abs(y / s), 2.0 ** -10) + 36 * U * np.abs(y / s))
    top = np.stack([np.abs(c[:, i:i + 128]).max(1) for i in range(0, y.shape[1], 128)], 1)
    assert (top[np.abs(want - 1) > 1e-9] > 430).all() or (want <= 2.0 ** -125).any()


@pytest.mark.parametrize("T,H", [(1, 8), (1, 128), (3, 136), (1, 2048), (2, 1000), (33, 256), (7, 2880), (130, 1024), (5, 4104),
                                 (64, 6144), (3, 8192), (2, 8200), (2, 16384), (1500, 512), (2049, 2048)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(proj, T, H, residual):
    g = gen(T + H)
    x, r = rows(g, T, H), rows(g, T, H)
    w = torch.randn(H, generator=g, device=DEV)
    s = (x.float() + r.float()).to(torch.bfloat16) if residual else x
    y = P.norm(f64(s), f64(w), 1e-5)
    ro = torch.empty_like(x) if residual else None
    kw = dict(residual=r, residual_out=ro) if residual else {}
    out = proj.norm(x, w, eps=1e-5, **kw)
    close(out, y, (2.0 ** -8 + 32 * U) * np.abs(y))
    if residual:
        assert torch.equal(ro, s)
    both = torch.empty_like(x)
    codes, scales = proj.norm_quant(x, w, eps=1e-5, out=both, **kw)
    assert torch.equal(both, out) and scales.shape == (T, -(-H // 128))
    check_codes(codes, scales, y)
    # quantised as they are
    codes, scales = proj.norm_quant(x, **kw)
    check_codes(codes, scales, f64(s))
    assert proj.status() == 0


def test_norm_in_place_and_strided(proj):
    g = gen(2)
    wide = rows(g, 40, 3 * 1000)
    x, r = wide[:, :1000], wide[:, 1000:2000]
    w = torch.randn(1000, generator=g, device=DEV)
    ro = torch.empty(40, 1000, dtype=torch.bfloat16, device=DEV)
    want = proj.norm(x.contiguous(), w, residual=r.contiguous(), residual_out=ro)
    keep = wide.clone()
    scales = torch.full((40, 20), -1.0, device=DEV)
    codes = torch.zeros(40, 1200, dtype=torch.uint8, device=DEV)
    c0, s0 = proj.norm_quant(x, w, residual=r, residual_out=ro)
    c1, s1 = proj.norm_quant(x, w, residual=r, codes=codes[:, 96:1096], scales=scales[:, 1:17:2], out=x)  # over x and r
    assert torch.equal(x, want) and torch.equal(r, ro) and torch.equal(wide[:, 2000:], keep[:, 2000:])
    assert torch.equal(c0, c1) and torch.equal(s0, s1)
    assert (scales[:, ::2] == -1).all() and (codes[:, :96] == 0).all() and (codes[:, 1096:] == 0).all()


@pytest.mark.parametrize("H", [64, 1000, 4096, 16384])
def test_norm_special_rows(proj, H):
    """Rows whose squares leave f32, beside ordinary ones of the same CTA; zeros;
    infinities and NaN stay within their row and their block's code."""
    x = torch.ones(12, H, dtype=torch.bfloat16, device=DEV)
    x[0], x[1], x[2], x[3] = 1e30, 3e38, 1e-25, 0.0
    x[4, 5], x[5, 5] = float("nan"), float("inf")
    x[6] = -2e18
    x[7] = 1e-38
    w = torch.ones(H, device=DEV)
    y = f64(proj.norm(x, w, eps=0.0))
    for t, v in ((0, 1), (1, 1), (2, 1), (6, -1), (7, 1), (8, 1), (11, 1)):
        assert (y[t] == v).all(), t
    assert np.isnan(y[3]).all() and np.isnan(y[4]).all()
    y = f64(proj.norm(x, w, eps=1e-6))
    assert (y[3] == 0).all() and np.abs(y[2]).max() < 1e-20 and (y[0] == 1).all()
    codes, scales = proj.norm_quant(x)
    c = codes.cpu().numpy()
    assert (c[4, 5] & 0x7F) == 0x7F and (c[5, 5] & 0x7F) == 0x7F and (c[4, :5] == 0x7E).all() and (c[5, :5] == 0x7E).all()
    assert (c[3] == 0).all() and (f64(scales)[3] == 1).all() and (c[1] == 0x7E).all() and (c[7] != 0).all()


def e4m3(g, *shape):
    return (torch.randn(*shape, generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def make(g, M, N, K, pad=0):
    kb, up = -(-K // 128), -(-K // 16) * 16 + pad
    a, w = e4m3(g, M, up)[:, :K], e4m3(g, N, up)[:, :K]
    sa = torch.exp(torch.randn(kb, M, generator=g, device=DEV)).t()
    sw = torch.exp(torch.randn(-(-N // 128), kb, generator=g, device=DEV)) * 1e-4
    return a, sa, w, sw


def check_matmul(proj, a, sa, w, sw, out=None):
    got = proj.matmul(a, sa, w, sw, out=out)
    K = a.shape[1]
    want, size = P.matmul(a.cpu().numpy(), f64(sa), w.cpu().numpy(), f64(sw))
    close(got, want, 2.0 ** -8 * np.abs(want) + (K / 4 + K / 64 + 24) * U * size)
    assert proj.status() == 0
    return got


@pytest.mark.parametrize("M,N,K", [
    (1, 128, 128), (1, 8, 16), (1, 1, 1), (3, 129, 130), (16, 256, 2048), (8, 1000, 2880), (1, 6144, 2048), (31, 64, 640), (64, 4096, 1024),
    (127, 200, 384), (128, 130, 256), (129, 257, 500), (333, 1000, 2880), (2, 20000, 256), (700, 640, 128), (1025, 4000, 300),
    (2500, 2500, 700), (4097, 2056, 1100), (1, 16, 65536)])
def test_matmul(proj, M, N, K):
    check_matmul(proj, *make(gen(M + N + K), M, N, K))


@pytest.mark.parametrize("seed", range(30))
def test_matmul_drawn(proj, seed):
    """Sizes over every way of splitting: few rows, clusters, tiles of each width."""
    rng = np.random.default_rng(seed)
    M = int(np.exp(rng.uniform(0, np.log([20, 70, 300, 1500][seed % 4]))))
    N, K = int(np.exp(rng.uniform(np.log(8), np.log(5000)))), int(np.exp(rng.uniform(np.log(16), np.log(4000))))
    few = Projection(max_sms=int(rng.choice([1, 5, 40]))) if seed % 5 == 0 else proj
    a, sa, w, sw = make(gen(seed), M, N, K, pad=int(rng.choice([0, 0, 32])))
    got = check_matmul(few, a, sa, w, sw)
    assert torch.equal(few.matmul(a, sa, w, sw), got)


@pytest.mark.parametrize("M", [1, 31, 32, 33, 64, 65, 128, 129])
def test_matmul_rows_at_the_borders(proj, M):
    g = gen(M)
    a, sa, w, sw = make(g, M, 520, 1100)
    wide = torch.full((M + 2, 528), 9.0, dtype=torch.bfloat16, device=DEV)
    check_matmul(proj, a, sa, w, sw, wide[1:-1, :520])
    assert (wide[0] == 9).all() and (wide[-1] == 9).all() and (wide[:, 520:] == 9).all()


@pytest.mark.parametrize("M,N", [(1300, 2100), (1281, 2049), (1313, 2064), (2000, 2239), (4000, 257)])
def test_matmul_outputs_of_wide_tiles_stay_in_their_rows(proj, M, N):
    """Tiles of 256 columns whose last rows and columns lie outside, within wider rows."""
    a, sa, w, sw = make(gen(M), M, N, 300)
    wide = torch.full((M + 2, -(-N // 8) * 8 + 24), 9.0, dtype=torch.bfloat16, device=DEV)
    got = check_matmul(proj, a, sa, w, sw, wide[1:-1, 8:8 + N])
    assert (wide[0] == 9).all() and (wide[-1] == 9).all() and (wide[:, :8] == 9).all() and (wide[:, 8 + N:] == 9).all()
    assert torch.equal(proj.matmul(a, sa, w, sw), got)


def test_matmul_strides(proj):
    """Rows within wider ones, scales in either order, output within wider rows."""
    g = gen(5)
    a, sa, w, sw = make(g, 77, 200, 300, pad=64)
    out = torch.full((77, 256), 5.0, dtype=torch.bfloat16, device=DEV)
    got = check_matmul(proj, a, sa, w, sw, out[:, 8:208])
    assert (out[:, :8] == 5).all() and (out[:, 208:] == 5).all()
    assert torch.equal(proj.matmul(a, sa.contiguous(), w, sw), got)
    big = torch.zeros(77, 9, device=DEV)
    big[:, 1:7:2] = sa
    assert torch.equal(proj.matmul(a, big[:, 1:7:2], w, sw), got)


def test_matmul_nan_stays_in_its_row(proj):
    a, sa, w, sw = make(gen(6), 130, 300, 400)
    want = proj.matmul(a, sa, w, sw).clone()
    a = a.clone().contiguous()
    a2 = torch.zeros(130, 400, dtype=torch.uint8, device=DEV)
    a2.copy_(a)
    a2[129, 7] = 0x7F
    got = proj.matmul(a2, sa, w, sw)
    assert torch.isnan(got[129]).all() and torch.equal(got[:129], want[:129])
    sa2 = sa.clone()
    sa2[3, 1] = float("inf")
    got = proj.matmul(a, sa2, w, sw)
    assert not torch.isfinite(got[3]).any() and torch.equal(got[4:], want[4:])


def test_matmul_of_nothing(proj):
    g = gen(1)
    a, sa, w, sw = make(g, 5, 40, 64)
    assert proj.matmul(a[:0], sa[:0], w, sw).shape == (0, 40) and proj.matmul(a, sa, w[:0], sw[:0]).shape == (5, 0)
    out = torch.full((5, 48), 3.0, dtype=torch.bfloat16, device=DEV)
    proj.matmul(a[:, :0], sa[:, :0], w[:, :0], sw[:, :0], out=out[:, :40])
    assert (out[:, :40] == 0).all() and (out[:, 40:] == 3).all()
    x = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    assert proj.norm(x).shape == (0, 256) and proj.norm_quant(x)[1].shape == (0, 2)
    assert proj.status() == 0


@pytest.mark.parametrize("M,N,K", [(1, 512, 2048), (200, 1000, 1500), (3000, 3000, 256)])
def test_same_bits_in_a_graph_on_a_stream_and_with_others_in_flight(proj, M, N, K):
    a, sa, w, sw = make(gen(M), M, N, K)
    want = proj.matmul(a, sa, w, sw).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(want) for _ in range(4)]
    for i, o in enumerate(outs):  # two streams, one context
        proj.matmul(a, sa, w, sw, out=o, stream=side if i % 2 else None)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        proj.matmul(a, sa, w, sw, out=outs[0])
        proj.norm(outs[0], out=outs[1])
    outs[0].zero_()
    g.replay()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_few_sms(proj):
    a, sa, w, sw = make(gen(9), 300, 700, 900)
    few = Projection(max_sms=4)
    check_matmul(few, a, sa, w, sw)
    x = rows(gen(3), 900, 640)
    assert torch.equal(few.norm(x), proj.norm(x))


def test_projections_of_a_block(proj):
    """Norm, projection, prompt attention, output projection, norm, and the experts: as
    they are used together, against the same steps in 64 bits."""
    g = gen(40)
    T, H, nh, nkv, d, I = 150, 512, 4, 2, 128, 256
    x, res = rows(g, T, H), rows(g, T, H)
    w1 = torch.rand(H, generator=g, device=DEV) + 0.5
    wq = e4m3(g, (nh + 2 * nkv) * d, H)
    sq = torch.full((-(-wq.shape[0] // 128), H // 128), 0.0004, device=DEV)
    wo = e4m3(g, H, nh * d)
    so = torch.full((H // 128, nh * d // 128), 0.0004, device=DEV)
    starts = torch.tensor([0, 90, 150], dtype=torch.int32, device=DEV)
    attn = DecodeAttention(nh, nkv, d)
    c, s = proj.norm_quant(x, w1, residual=res)
    qkv = proj.matmul(c, s, wq, sq).view(T, -1, d)
    o = attn.prefill(qkv[:, :nh], qkv[:, nh:nh + nkv], qkv[:, nh + nkv:], starts)
    co, so2 = proj.norm_quant(o.view(T, -1))
    y = proj.matmul(co, so2, wo, so)
    both = torch.empty_like(y)
    proj.norm_quant(y, w1, residual=res, out=both)
    layer = MoELayer(T, H, 8, I, 2, 0)
    z = layer.forward(both, torch.randn(8, H, generator=g, device=DEV), None, e4m3(g, 8, 2 * I, H),
                      torch.full((8, 2 * I // 128, H // 128), 0.01, device=DEV), e4m3(g, 8, H, I),
                      torch.full((8, H // 128, I // 128), 0.01, device=DEV), 2)
    # every step from what the step before it gave
    want, size = P.matmul(c.cpu().numpy(), f64(s), wq.cpu().numpy(), f64(sq))
    close(qkv.reshape(T, -1), want, 2.0 ** -8 * np.abs(want) + (H / 4 + H / 64 + 24) * U * size)
    want, size = P.matmul(co.cpu().numpy(), f64(so2), wo.cpu().numpy(), f64(so))
    close(y, want, 2.0 ** -8 * np.abs(want) + (H / 4 + H / 64 + 24) * U * size)
    yn = P.norm(f64(res), f64(w1), 1e-6)
    close(both, yn, (2.0 ** -8 + 32 * U) * np.abs(yn))
    assert torch.isfinite(z).all() and attn.status() == 0 and proj.status() == 0 and layer.status() == 0


def test_refusals(proj):
    x = rows(gen(1), 4, 256)
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(weight=torch.ones(255, device=DEV)), dict(residual=x[:3]),
                dict(out=x[:, :128]), dict(x=x.t())):
        with pytest.raises(ValueError):
            proj.norm(**{**dict(x=x), **bad})
    for bad in (dict(eps=-1.0), dict(x=x[:, :100]), dict(x=x[:, 4:12])):
        with pytest.raises(RuntimeError):
            proj.norm(**{**dict(x=x), **bad})
    a, sa, w, sw = make(gen(2), 4, 256, 256)
    for bad in (dict(codes=x), dict(scales=sa[:3]), dict(w=w[:, :128]), dict(w_scale=sw.t()[:, :1]), dict(out=x[:, :4]),
                dict(w_scale=sw.repeat(1, 2)[:, ::2])):
        with pytest.raises(ValueError):
            proj.matmul(**{**dict(codes=a, scales=sa, w=w, w_scale=sw), **bad})
    with pytest.raises(RuntimeError):
        proj.matmul(a[:, 1:129], sa[:, :1], w[:, 1:129], sw[:, :1].contiguous())
    p = Projection()
    p.close()
    with pytest.raises(ValueError):
        p.norm(x)


@pytest.mark.parametrize("T,H,size", [(300, 1000, 1.0), (40, 6144, 3.0), (1, 2048, 1e3), (65, 16384, 1e-4), (900, 136, 1e-33), (50, 512, 1e-36), (50, 512, 1e-38),
                                      (70, 256, 1e35)])
def test_codes_are_those_of_the_quotient(proj, T, H, size):
    """Rows quantised as they are: scale and quotient are one f32 division each, and the code the
    quotient's nearest, so every bit follows."""
    x = rows(gen(T), T, H, size)
    x[0, 5], x[-1, 7] = 0.0, -0.0
    codes, scales = proj.norm_quant(x)
    y = x.float().cpu().numpy()
    s = np.stack([np.abs(y[:, c:c + 128]).max(1) for c in range(0, H, 128)], 1) / np.float32(448)
    s = np.where(s == 0, np.float32(1), np.maximum(s, np.float32(2.0 ** -126)))
    assert s.dtype == np.float32 and (scales.cpu().numpy() == s).all()
    want = torch.from_numpy(y / P.spread(s, H)).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(codes.cpu(), want)


@pytest.mark.parametrize("H", [64, 1000, 4096])
def test_norm_with_weights_far_from_one(proj, H):
    """Rows and weights whose products are ordinary numbers, though 1 / rms times a weight is not
    one; eps 0."""
    g = gen(H)
    for size, weight in ((1e-12, 1e30), (1e15, 1e-30), (1e-30, 1e20), (1e25, 1e-20)):
        x = (torch.randn(9, H, generator=g, device=DEV) * size).to(torch.bfloat16)
        w = (torch.rand(H, generator=g, device=DEV) + 0.5) * weight
        y = P.norm(f64(x), f64(w), 0.0)
        close(proj.norm(x, w, eps=0.0), y, (2.0 ** -8 + 32 * U) * np.abs(y))


@pytest.mark.parametrize("M,N,K", [(5, 300, 700), (50, 200, 300), (200, 130, 640), (300, 1100, 400), (1500, 1500, 300)])
def test_matmul_scales_at_the_ends_of_f32(proj, M, N, K):
    """A block's two scales multiply to normal f32 numbers, down to the smallest and up to where the
    results end, though one of them or both are far outside.  Half a step of results below bf16's
    normal ones is 2^-134."""
    def check(a, sa, w, sw):
        want, size = P.matmul(a.cpu().numpy(), f64(sa), w.cpu().numpy(), f64(sw))
        close(proj.matmul(a, sa, w, sw), want, 2.0 ** -8 * np.abs(want) + (K / 4 + K / 64 + 24) * U * size + 2.0 ** -134)
        assert proj.status() == 0 and np.abs(want).max() < 3e38

    g = gen(M)
    a, sa, w, sw = make(g, M, N, K)
    sa, sw = sa.clamp(0.5, 2.0), (sw * 1e4).clamp(0.5, 2.0)
    a[(a & 0x7F) == 0] = 0x38
    # 2^-124 / 4 is the smallest normal number; subnormal scales on either side
    for da, dw in ((2.0 ** -62, 2.0 ** -62), (2.0 ** -140, 2.0 ** 16), (2.0 ** 20, 2.0 ** -144), (2.0 ** -124, 1.0), (2.0 ** 100, 2.0 ** -60), (2.0 ** 50, 2.0 ** 50)):
        check(a, sa * da, w, sw * dw)
    # zeros and scales that are not finite stay in their rows
    s0 = sa.clone()
    s0[0], s0[1] = 0.0, float("inf")
    got = proj.matmul(a, s0, w, sw)
    assert (got[0] == 0).all() and not torch.isfinite(got[1]).any() and torch.equal(got[2:], proj.matmul(a, sa, w, sw)[2:])


def grids(run):
    """CTAs of the kernels that `run` launches, as a graph that captures them has them."""
    class Params(ctypes.Structure):
        _fields_ = [("func", ctypes.c_void_p), *((n, ctypes.c_uint) for n in ("gx", "gy", "gz", "bx", "by", "bz", "shared")),
                    *((n, ctypes.c_void_p) for n in ("params", "extra", "kern", "ctx"))]

    run()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        run()
    cuda, handle, n = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(g.raw_cuda_graph()), ctypes.c_size_t()
    assert cuda.cuGraphGetNodes(handle, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cuda.cuGraphGetNodes(handle, nodes, ctypes.byref(n)) == 0
    found = []
    for node in nodes:
        kind, p = ctypes.c_int(-1), Params()
        assert cuda.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:  # a kernel
            assert cuda.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
            found.append(p.gx * p.gy * p.gz)
    return found


@pytest.mark.parametrize("limit", [1, 5, 40])
def test_a_limit_on_the_sms_is_one_of_ctas(proj, limit):
    few, g = Projection(max_sms=limit), gen(limit)
    for T, H in ((900, 640), (4000, 2048), (3, 64), (2000, 16384)):
        x = rows(g, T, H)
        n = grids(lambda: few.norm(x))
        assert len(n) == 1 and 1 <= n[0] <= limit, n
        assert torch.equal(few.norm(x), proj.norm(x))
    for M, N, K in ((1, 4096, 2048), (33, 6000, 1000), (64, 700, 4000), (100, 512, 2048), (333, 1000, 2880), (2000, 2048, 512)):
        args = make(g, M, N, K)
        n = grids(lambda: few.matmul(*args))
        assert len(n) == 1 and 1 <= n[0] <= limit, (M, N, K, n)
        check_matmul(few, *args)
    attn = DecodeAttention(8, 2, 128, max_sms=limit)
    for Tq, Tk in ((1, 3000), (700, 700), (1000, 5000)):
        q, k = rows(g, Tq, 1024).view(Tq, 8, 128), rows(g, Tk, 256).view(Tk, 2, 128)
        starts = [torch.tensor([0, t], dtype=torch.int32, device=DEV) for t in (Tq, Tk)]
        n = grids(lambda: attn.prefill(q, k, k, *starts))
        assert len(n) == 1 and 1 <= n[0] <= limit, (Tq, Tk, n)


def test_a_block_step_by_step():
    """The same steps, each against its oracle on what the step before it gave: both residual sums, the codes of
    both norms and of the attention's output, the attention, the projections, the norms' bf16 rows and the experts."""
    g, proj = gen(41), Projection()
    T, H, nh, nkv, d, I = 170, 512, 4, 2, 128, 256
    x, res = rows(g, T, H), rows(g, T, H, 0.5)
    w1, w2 = (torch.rand(H, generator=g, device=DEV) + 0.5 for _ in range(2))
    wq, wo = e4m3(g, (nh + 2 * nkv) * d, H), e4m3(g, H, nh * d)
    sq = torch.rand(nh + 2 * nkv, H // 128, generator=g, device=DEV) * 0.0008
    so = torch.rand(H // 128, nh * d // 128, generator=g, device=DEV) * 0.02
    starts = np.array([0, 90, 170], np.int32)

    def product(got, c, s, w, sw):
        want, size = P.matmul(c.cpu().numpy(), f64(s), w.cpu().numpy(), f64(sw))
        k = c.shape[1]
        close(got, want, 2.0 ** -8 * np.abs(want) + (k / 4 + k / 64 + 24) * U * size)

    total = (x.float() + res.float()).to(torch.bfloat16)
    c, s = proj.norm_quant(x, w1, residual=res)
    assert torch.equal(res, total)
    check_codes(c, s, P.norm(f64(total), f64(w1), 1e-6))
    qkv = proj.matmul(c, s, wq, sq)
    product(qkv, c, s, wq, sq)
    q, k, v = qkv.view(T, -1, d).split([nh, nkv, nkv], dim=1)
    o, _ = check_prompts(q, k, v, starts, starts)
    co, s_o = proj.norm_quant(o.view(T, -1))
    check_codes(co, s_o, f64(o.view(T, -1)))
    y = proj.matmul(co, s_o, wo, so)
    product(y, co, s_o, wo, so)
    total = (y.float() + res.float()).to(torch.bfloat16)
    assert not torch.equal(total, res)  # the projection matters
    h = proj.norm(y, w2, residual=res)
    assert torch.equal(res, total)
    want = P.norm(f64(total), f64(w2), 1e-6)
    close(h, want, (2.0 ** -8 + 32 * U) * np.abs(want))
    router, w13, w2e = torch.randn(8, H, generator=g, device=DEV), e4m3(g, 8, 2 * I, H), e4m3(g, 8, H, I)
    s13 = torch.rand(8, 2 * I // 128, H // 128, generator=g, device=DEV) * 0.001
    s2 = torch.rand(8, H // 128, I // 128, generator=g, device=DEV) * 0.01
    layer = MoELayer(T, H, 8, I, 2, 0)
    z = layer.forward(h, router, None, w13, s13, w2e, s2, 2)
    host = [t.cpu().numpy() for t in (router, w13, s13, w2e, s2)]
    ref = moe_forward(h.view(torch.int16).cpu().numpy().view(np.uint16), host[0], None, *host[1:], 2)
    check_output(z.view(torch.int16).cpu().numpy().view(np.uint16), ref)
    assert proj.status() == 0 and layer.status() == 0
