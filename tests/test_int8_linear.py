"""8-bit integer rows and products against their definitions in 64 bits (and whole numbers)."""
import pytest
import torch

from paged_kv_chunk_gb300 import build, capi

import e4m3_ref as ref

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 2.0 ** -100


def rows(x):
    """x8 and scale by the definition: the three fp32 operations written out (each a 64-bit one of
    operands of 24 bits, rounded), the scale in 64 bits."""
    m = x.float().abs().amax(1).clamp(min=TINY)
    f = ((1.0 / m.double()).float().double() * 127.0).float()
    q = torch.round((x.float().double() * f.double()[:, None]).float())
    return q.to(torch.int8), m.double() / 127.0


def product(x8, xs, w8, ws, bias, dtype):
    """out in 64 bits and its elementwise bound.  The integer sum is exact where it stays below 2^24
    however it is added up; above, each of K / 16 additions may drop one step of fp32 (2^-23).  Two
    scalings, the bias and the result are rounded once each, to half a step."""
    s = x8.double() @ w8.double().t()
    mag = x8.double().abs() @ w8.double().abs().t()
    K = x8.shape[1]
    few = x8.shape[0] <= 8
    ds = torch.where((mag < 2.0 ** 24) | few, 0.0, mag * (K / 16) * 2.0 ** -23)
    ds = ds + (s.abs() * 2.0 ** -24 if few else 0)           # the exact integer to fp32
    sc = xs.double()[:, None] * ws.double()
    y = s * sc
    out = y if bias is None else y + bias.double()
    r = ref.BF16 if dtype == torch.bfloat16 else 0
    tol = (ds * sc + 2 * 2.0 ** -24 * y.abs() + 2.0 ** -24 * out.abs()) * 1.01 + r * out.abs() * 1.01 + 1e-36
    return out, tol


def integers(g, *shape, top=127):
    return torch.randint(-top, top + 1, shape, generator=g).to(torch.int8)


def close(got, want):
    out, tol = want
    err = (got.double().cpu() - out).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


# ------------------------------------------------------------------- CPU

@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


FAKE = 1 << 20


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), capi.OASR_ERR_INVALID_ARG), (dict(M=0), capi.OASR_ERR_INVALID_ARG),
    (dict(K=24), capi.OASR_ERR_UNSUPPORTED), (dict(dt=2), capi.OASR_ERR_UNSUPPORTED),
    (dict(x8=FAKE + 8), capi.OASR_ERR_INVALID_ARG),
])
def test_quantize_refusals(lib, kw, expect):
    a = dict(x=FAKE, x8=FAKE, s=FAKE, M=4, K=64, dt=capi.OASR_BF16)
    a.update(kw)
    assert lib.oasr_quantize_rows(*a.values(), None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(w=None), capi.OASR_ERR_INVALID_ARG), (dict(N=0), capi.OASR_ERR_INVALID_ARG),
    (dict(K=72), capi.OASR_ERR_UNSUPPORTED), (dict(K=65552), capi.OASR_ERR_UNSUPPORTED),
    (dict(dt=2), capi.OASR_ERR_UNSUPPORTED), (dict(out=FAKE + 4), capi.OASR_ERR_INVALID_ARG),
    (dict(bias=FAKE + 2), capi.OASR_ERR_INVALID_ARG), (dict(M=2 ** 31 - 255), capi.OASR_ERR_UNSUPPORTED),
    (dict(N=2 ** 31 - 1), capi.OASR_ERR_UNSUPPORTED),
])
def test_linear_refusals(lib, kw, expect):
    a = dict(x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, bias=None, out=FAKE, M=4, N=64, K=64, dt=capi.OASR_F32)
    a.update(kw)
    assert lib.oasr_linear_w8a8(*a.values(), None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(b=None), capi.OASR_ERR_INVALID_ARG), (dict(rel=FAKE + 8), capi.OASR_ERR_INVALID_ARG),
    (dict(M=0), capi.OASR_ERR_INVALID_ARG), (dict(R=-1), capi.OASR_ERR_INVALID_ARG),
    (dict(d=96), capi.OASR_ERR_UNSUPPORTED), (dict(H=3), capi.OASR_ERR_UNSUPPORTED),
    (dict(dt=4), capi.OASR_ERR_UNSUPPORTED), (dict(d=16448, H=257), capi.OASR_ERR_UNSUPPORTED),
    (dict(M=2 ** 31 - 1), capi.OASR_ERR_UNSUPPORTED), (dict(R=2 ** 31 - 1), capi.OASR_ERR_UNSUPPORTED),
])
def test_project_refusals(lib, kw, expect):
    a = dict(x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, b=FAKE, p=FAKE, ps=FAKE, wp=FAKE, wps=FAKE, q=FAKE, k=FAKE, v=FAKE,
             rel=FAKE, M=4, R=9, d=128, H=2, dt=capi.OASR_BF16)
    a.update(kw)
    assert lib.oasr_project_qkv_pos_w8a8(*a.values(), None) == expect


# ------------------------------------------------------------------- GPU

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 1024), (7, 48), (9, 512), (300, 256), (5, 1040), (3, 8192), (2, 8208),
                                 (2, 20000)])
def test_quantize_rows(M, K, dtype):
    g = torch.Generator().manual_seed(M + K)
    x = (torch.randn(M, K, generator=g) * 2.0 ** torch.randint(-20, 20, (M, 1), generator=g)).to(DT[dtype])
    x[0] = 0 if M > 1 else x[0]
    x[-1, K // 2] = 5e30
    x8, scale = capi.oasr_quantize_rows(x.cuda())
    q, s = rows(x)
    assert torch.equal(x8.cpu(), q)
    assert bool(((scale.double().cpu() - s).abs() <= s * 2.0 ** -24).all())
    assert int(x8[-1, K // 2]) == 127


@pytest.mark.gpu
def test_quantize_rows_ties_tiny_and_bad():
    x = torch.zeros(5, 32)
    x[0, :5] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5])       # the factor is one: ties to even
    x[1, 0] = 2.0 ** -130                                       # below the least maximum
    x[2, 3] = float("nan")
    x[3, 31] = float("-inf")
    x[4, 0] = 3.0e38
    x8, scale = capi.oasr_quantize_rows(x.cuda())
    assert x8[0, :5].tolist() == [127, 0, 2, 2, 0] and float(scale[0]) == 1.0
    assert not x8[1:4].any() and torch.equal(scale[1].cpu(), torch.tensor(TINY) / 127)
    assert scale[2:4].isnan().all() and int(x8[4, 0]) == 127 and bool(scale[4].isfinite())
    w8 = torch.ones(24, 32, dtype=torch.int8, device="cuda")
    out = capi.oasr_linear_w8a8(x8, scale, w8, torch.ones(24, device="cuda"))
    assert out[2:4].isnan().all() and out[[0, 1, 4]].isfinite().all()


SHAPES = [  # M, N, K
    (1, 1, 16), (1, 2048, 512), (2, 37, 80), (4, 64, 1024), (5, 33, 4096), (8, 1000, 528),
    (9, 1, 16), (17, 40, 64), (128, 32, 48), (129, 100, 256), (200, 129, 1024), (1000, 513, 272),
    (64, 4096, 2048), (4096, 640, 128), (2500, 2000, 1024), (130, 72, 4112),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K, dtype):
    g = torch.Generator().manual_seed(M * 7 + N + K)
    x8, w8 = integers(g, M, K), integers(g, N, K)
    x8[0, 0] = -128                      # not made by quantize_rows, but an 8-bit integer
    xs, ws = torch.rand(M, generator=g) + 0.1, torch.rand(N, generator=g) * 1e-3
    bias = torch.randn(N, generator=g).to(DT[dtype])
    for b in (bias, None):
        out = capi.oasr_linear_w8a8(x8.cuda(), xs.cuda(), w8.cuda(), ws.cuda(), None if b is None else b.cuda(),
                                    out_dtype=DT[dtype])
        close(out, product(x8, xs, w8, ws, b, DT[dtype]))
    assert capi.oasr_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(9, 37, 528), (16, 3, 2064), (33, 130, 4112), (128, 70, 1040), (100, 513, 80), (17, 4096, 1024),
                                   (127, 501, 2048), (31, 512, 512)])
def test_some_rows(M, N, K, dtype):
    """Batches of a few dozen tokens: rows and columns that end inside a block, K that ends inside a round."""
    g = torch.Generator().manual_seed(M * 5 + N + K)
    x8, w8 = integers(g, M, K), integers(g, N, K)
    xs, ws = torch.rand(M, generator=g) + 0.1, torch.rand(N, generator=g) * 1e-3
    bias = torch.randn(N, generator=g).to(DT[dtype])
    # a guard behind the last row stays as it was
    out = torch.full((M + 1, N), 7.0, dtype=DT[dtype], device="cuda")
    for b in (bias, None):
        capi.oasr_linear_w8a8(x8.cuda(), xs.cuda(), w8.cuda(), ws.cuda(), None if b is None else b.cuda(), out=out[:M])
        close(out[:M], product(x8, xs, w8, ws, b, DT[dtype]))
        assert bool((out[M] == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 8, 9, 140])
def test_sums_are_the_integers(M):
    """The largest sums K = 1024 can have, and alternating ones, bit for bit."""
    K, N = 1024, 96
    x8 = torch.full((M, K), 127, dtype=torch.int8)
    x8[-1] = -128
    w8 = torch.full((N, K), 127, dtype=torch.int8)
    w8[1] = -128
    w8[2, ::2] = -127
    w8[3, 1:] = 0
    w8[4:] = integers(torch.Generator().manual_seed(M), N - 4, K)
    one = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    out = capi.oasr_linear_w8a8(x8.cuda(), one[0], w8.cuda(), one[1], out_dtype=torch.float32)
    assert torch.equal(out.double().cpu(), x8.double() @ w8.double().t())


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(64, 4096, 1024), (1000, 513, 272), (3000, 700, 1008), (2600, 1100, 1024), (8191, 4096, 48),
                                   (4100, 1000, 208), (257, 9000, 512), (2600, 1101, 1024), (5000, 2302, 64), (1000, 503, 64)])
def test_tiles_of_every_shape_bit_for_bit(M, N, K):
    """Several tiles per CTA, last tiles of a row or column, a CTA pair whose second half has no row; the same
    sums at every repetition."""
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    x8, w8 = (torch.randint(-128, 128, (n, K), generator=g, device="cuda", dtype=torch.int8) for n in (M, N))
    want = (x8.double() @ w8.double().t()).float()   # integers below 2^24
    one = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    for _ in range(20):
        assert torch.equal(capi.oasr_linear_w8a8(x8, one[0], w8, one[1], out_dtype=torch.float32), want)
    assert capi.oasr_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(2600, 1100, 512), (300, 700, 512), (40, 500, 2048)])
def test_captured_products_side_by_side(M, N, K):
    """Two graphs of the same products on two streams at once, replayed over and over with new rows."""
    w8 = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda")
    ws = torch.rand(N, device="cuda")
    jobs = []
    for _ in range(2):
        x8, xs = torch.zeros(M, K, dtype=torch.int8, device="cuda"), torch.rand(M, device="cuda")
        out = capi.oasr_linear_w8a8(x8, xs, w8, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                capi.oasr_linear_w8a8(x8, xs, w8, ws, out=out)
        jobs.append((x8, xs, out, graph, torch.cuda.Stream()))
    for _ in range(5):
        for x8, xs, _, _, _ in jobs:
            x8.copy_(torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda"))
        torch.cuda.synchronize()
        for _, _, _, graph, stream in jobs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for x8, xs, out, _, _ in jobs:
            assert torch.equal(out, capi.oasr_linear_w8a8(x8, xs, w8, ws))
    assert capi.oasr_device_status() == 0


@pytest.mark.gpu
def test_longest_rows():
    g = torch.Generator().manual_seed(2)
    for M in (3, 20):
        x8, w8 = integers(g, M, 65536, top=60), integers(g, 40, 65536, top=60)
        one = torch.ones(M), torch.ones(40)
        out = capi.oasr_linear_w8a8(x8.cuda(), one[0].cuda(), w8.cuda(), one[1].cuda(), out_dtype=torch.float32)
        close(out, product(x8, *one[:1], w8, one[1], None, torch.float32))


@pytest.mark.gpu
@pytest.mark.parametrize("M,R,H,dtype", [(1, 31, 1, "bf16"), (5, 1, 3, "f32"), (200, 287, 4, "bf16"),
                                         (1030, 95, 8, "bf16"), (300, 130, 5, "f32")])
def test_project(M, R, H, dtype):
    d = 64 * H
    g = torch.Generator().manual_seed(M + R)
    x8, w8, p8, wp8 = (integers(g, n, d) for n in (M, 3 * d, R, d))
    xs, ws, ps, wps = (torch.rand(n, generator=g) * 0.01 + 0.001 for n in (M, 3 * d, R, d))
    bias = torch.randn(3 * d, generator=g).to(DT[dtype])
    q, k, v, rel = capi.oasr_project_qkv_pos_w8a8(*(t.cuda() for t in (x8, xs, w8, ws, bias, p8, ps, wp8, wps)), H)
    want, tol = product(torch.cat([x8, x8[:0]]), xs, w8, ws, bias, DT[dtype])
    # the one-launch call accumulates in fp32 whatever the row count; d <= 1024: exact
    for i, t in enumerate((q, k, v)):
        close(t.reshape(M, d), (want[:, i * d:(i + 1) * d], tol[:, i * d:(i + 1) * d]))
    close(rel.reshape(R, d), product(p8, ps, wp8, wps, None, DT[dtype]))


@pytest.mark.gpu
def test_the_8_bit_step_together():
    """Quantised activations -> projections -> step over the 8-bit cache -> commit, as a layer runs
    them, captured as one graph and replayed for three chunks, against 64 bits on the library's own
    projections."""
    B, H, T, bs, window = 3, 4, 16, 16, 64
    d, M, R = 64 * H, B * T, window + 16 + 2 * T - 1
    g = torch.Generator().manual_seed(3)
    w8, ws = capi.oasr_quantize_rows((torch.randn(3 * d, d, generator=g) * d ** -0.5).cuda())
    wp8, wps = capi.oasr_quantize_rows((torch.randn(d, d, generator=g) * d ** -0.5).cuda())
    bias = (torch.randn(3 * d, generator=g) * 0.1).bfloat16().cuda()
    p8, ps = capi.oasr_quantize_rows(torch.randn(R, d, generator=g).bfloat16().cuda())
    u, vb = (torch.randn(2, H, 64, generator=g) * 0.2).bfloat16().cuda()
    c = ref.Cache(B, H, bs, 6, 4)
    pools = c.cuda()
    lens = torch.tensor([0, 16, 32], dtype=torch.int32).cuda()
    pre = torch.randn(B, 32, H, 64, generator=g).bfloat16()
    capi.oasr_paged_append_e4m3(pre.cuda(), pre.cuda(), *pools, torch.zeros(B, dtype=torch.int32).cuda())
    x = torch.randn(M, d, generator=g).bfloat16().cuda()
    keep = {}

    def layer():
        x8, xs = capi.oasr_quantize_rows(x)
        q, k, v, rel = capi.oasr_project_qkv_pos_w8a8(x8, xs, w8, ws, bias, p8, ps, wp8, wps, H)
        q, k, v = (t.view(B, T, H, 64) for t in (q, k, v))
        out = capi.oasr_chunk_step_paged_e4m3(q, k, v, *pools[:3], pools[3], lens, u, vb, rel)
        keep.update(q=q, k=k, v=v, rel=rel, out=out)
        capi.oasr_window_commit(pools[3], lens, T, bs, window)

    saved = lens.clone(), pools[3].clone()
    layer()                                     # warm-up, undone below
    lens.copy_(saved[0])
    pools[3].copy_(saved[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    past = [[(pre[b, t], pre[b, t]) for t in range(int(saved[0][b]))] for b in range(B)]
    for n in range(5):
        x.copy_(torch.randn(M, d, generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        host = {name: t.cpu() for name, t in keep.items()}
        for b in range(B):
            C = len(past[b])
            past[b] += [(host["k"][b, t], host["v"][b, t]) for t in range(T)]
            hist = [ref.values(*ref.quantise(torch.stack([p[i] for p in past[b]]))) for i in range(2)]
            want, tol = ref.attention(host["q"][b], u.cpu(), vb.cpu(), host["rel"], hist, C, 0.125, torch.bfloat16)
            err = (host["out"][b].double() - want).abs()
            assert bool((err <= tol).all()), (n, b, float((err / tol).max()))
            past[b] = past[b][len(past[b]) - int(lens[b]):]
    assert capi.oasr_device_status() == 0


@pytest.mark.gpu
def test_same_bits_on_two_streams():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(700, 512, generator=g).bfloat16().cuda()
    w8, ws = capi.oasr_quantize_rows(torch.randn(1000, 512, generator=g).cuda())
    first = capi.oasr_linear_w8a8(*capi.oasr_quantize_rows(x), w8, ws)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(capi.oasr_linear_w8a8(*capi.oasr_quantize_rows(x), w8, ws))
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)


@pytest.mark.gpu
def test_binding_refusals():
    x = torch.randn(4, 64, device="cuda")
    x8, xs = capi.oasr_quantize_rows(x)
    w8, ws = capi.oasr_quantize_rows(torch.randn(8, 64, device="cuda"))
    for a in ((x, xs, w8, ws), (x8, xs[:3], w8, ws), (x8, xs, w8[:, :48], ws), (x8, xs, w8, ws.double()),
              (x8.cpu(), xs, w8, ws), (x8, xs, w8, ws, torch.zeros(7, device="cuda")),
              (x8, xs, w8, ws, torch.zeros(8, device="cuda")),       # bias is not of the output's type
              (x8[:, :48], xs, w8[:, :48], ws)):                     # not contiguous
        with pytest.raises(ValueError):
            capi.oasr_linear_w8a8(*a)
    with pytest.raises(TypeError):
        capi.oasr_quantize_rows(x.half())
    with pytest.raises(capi.OasrError):
        capi.oasr_quantize_rows(torch.randn(4, 40, device="cuda"))
    with pytest.raises(ValueError):
        capi.oasr_quantize_rows(x.t())
