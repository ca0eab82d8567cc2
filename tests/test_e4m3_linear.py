"""e4m3 rows with a scale for each block of 128 and their products, against their definitions in 64 bits."""
import pytest
import torch

from paged_kv_chunk_gb300 import build, capi

import e4m3_ref as ref

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
FAKE = 1 << 20


def power(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def blocks(x):
    """Values [M, K] (64 bits, scaled) and scale bytes by the definition."""
    M, K = x.shape
    out, byte = torch.empty(M, K, dtype=torch.float64), torch.empty(M, -(-K // 128), dtype=torch.uint8)
    for b in range(byte.shape[1]):
        v = x[:, 128 * b:128 * b + 128].double()
        most = v.abs().amax(1)
        e = torch.where(most > 0, torch.ceil(torch.log2(most / 448.0)), -100.0).clamp(min=-100)
        y = v * power(-e)[:, None]
        step = power((torch.frexp(y)[1] - 1).clamp(min=-6) - 3)
        out[:, 128 * b:128 * b + 128] = torch.round(y / step) * step
        byte[:, b] = (e + 127).to(torch.uint8)
    return out, byte


def values(x8, scale):
    """What e4m3 rows and their scales stand for, in 64 bits."""
    K = x8.shape[1]
    return x8.double() * power(scale.long() - 127).repeat_interleave(128, 1)[:, :K]


def product(x8, xs, w8, ws, bias, dtype):
    """out in 64 bits and its elementwise bound.  Products are exact; each of at most K additions of fp32 numbers may
    lose a step (2^-23, as a truncation does) of the running sum, at most the sum of magnitudes; the bias and the
    result are rounded once."""
    x, w = values(x8, xs), values(w8, ws)
    y, mag = x @ w.t(), x.abs() @ w.abs().t()
    out = y if bias is None else y + bias.double()
    r = ref.BF16 if dtype == torch.bfloat16 else 2.0 ** -24
    return out, x8.shape[1] * 2.0 ** -23 * mag * 1.01 + 2.0 ** -24 * out.abs() + r * out.abs() * 1.01 + 1e-38


def close(got, want):
    out, tol = want
    err = (got.double().cpu() - out).abs()
    assert bool((err <= tol).all()), float((err / tol).nan_to_num(9e9).max())


def matrix(g, M, K, loud=True):
    """Rows whose blocks' magnitudes lie some octaves apart."""
    x = torch.randn(M, K, generator=g)
    if loud:
        x *= 2.0 ** torch.randint(-6, 7, (M, -(-K // 128)), generator=g).repeat_interleave(128, 1)[:, :K]
    return x


# ------------------------------------------------------------------- CPU

@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), capi.OASR_ERR_INVALID_ARG), (dict(M=0), capi.OASR_ERR_INVALID_ARG),
    (dict(K=24), capi.OASR_ERR_UNSUPPORTED), (dict(dt=2), capi.OASR_ERR_UNSUPPORTED),
    (dict(x8=FAKE + 8), capi.OASR_ERR_INVALID_ARG), (dict(s=None), capi.OASR_ERR_INVALID_ARG),
])
def test_quantize_refusals(lib, kw, expect):
    a = dict(x=FAKE, x8=FAKE, s=FAKE, M=4, K=64, dt=capi.OASR_BF16)
    a.update(kw)
    assert lib.oasr_quantize_blocks(*a.values(), None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(w=None), capi.OASR_ERR_INVALID_ARG), (dict(N=0), capi.OASR_ERR_INVALID_ARG),
    (dict(K=72), capi.OASR_ERR_UNSUPPORTED), (dict(K=65552), capi.OASR_ERR_UNSUPPORTED),
    (dict(dt=2), capi.OASR_ERR_UNSUPPORTED), (dict(out=FAKE + 4), capi.OASR_ERR_INVALID_ARG),
    (dict(bias=FAKE + 2), capi.OASR_ERR_INVALID_ARG), (dict(M=2 ** 31 - 255), capi.OASR_ERR_UNSUPPORTED),
    (dict(N=2 ** 31 - 1), capi.OASR_ERR_UNSUPPORTED), (dict(ws=None), capi.OASR_ERR_INVALID_ARG),
])
def test_linear_refusals(lib, kw, expect):
    a = dict(x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, bias=None, out=FAKE, M=4, N=64, K=64, dt=capi.OASR_F32)
    a.update(kw)
    assert lib.oasr_linear_e4m3(*a.values(), None) == expect


def test_binding_refusals():
    x, e4, u8 = torch.zeros(4, 256), torch.float8_e4m3fn, torch.uint8
    x8, s = torch.zeros(4, 256, dtype=u8).view(e4), torch.zeros(4, 2, dtype=u8)
    with pytest.raises(ValueError, match="CUDA"):
        capi.oasr_quantize_blocks(x)
    with pytest.raises(ValueError, match="scale"):
        capi.oasr_quantize_blocks(x, scale=s[:, :1])
    with pytest.raises(ValueError, match="x8's scale"):
        capi.oasr_linear_e4m3(x8, s[:, :1], x8, s)
    with pytest.raises(ValueError, match="shapes"):
        capi.oasr_linear_e4m3(x8, s, x8[:, :240], s)
    with pytest.raises(ValueError, match="bias"):
        capi.oasr_linear_e4m3(x8, s, x8, s, bias=torch.zeros(3, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        capi.oasr_quantize_blocks(x.half())


# ------------------------------------------------------------------- GPU

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (7, 48), (9, 512), (300, 256), (5, 1040), (2, 8192),
                                 (3, 65536), (5000, 272)])
def test_quantize_blocks(M, K, dtype):
    g = torch.Generator().manual_seed(M + K)
    x = (matrix(g, M, K) * 2.0 ** torch.randint(-20, 20, (M, 1), generator=g)).to(DT[dtype])
    if M > 1:
        x[0] = 0
    x8, scale = capi.oasr_quantize_blocks(x.cuda())
    want, byte = blocks(x)
    assert torch.equal(scale.cpu(), byte)
    assert torch.equal(x8.cpu().double(), want)
    # what it stands for, quantised again, keeps its bytes (a block whose largest value fell below the last octave's
    # border aside: its scale may be one step lower, its values are the same)
    back = values(x8.cpu(), scale.cpu()).to(DT[dtype])
    again8, again = capi.oasr_quantize_blocks(back.cuda())
    assert torch.equal(values(again8.cpu(), again.cpu()), values(x8.cpu(), scale.cpu()))


@pytest.mark.gpu
def test_quantize_the_longest_row():
    """A row of 2^31 - 16 values, its last block of 112: the same bytes as its blocks by themselves."""
    K = 2 ** 31 - 16
    x = torch.randn(1, 1 << 20, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda().repeat(1, 2048)[:, 16:].contiguous()
    x8, scale = capi.oasr_quantize_blocks(x)
    whole = K // 128 * 128
    for part, rows in ((slice(0, whole), -1), (slice(whole, K), 1)):
        y = x[0, part].contiguous().view(rows, 128 if rows < 0 else 112)
        y8, s = capi.oasr_quantize_blocks(y)
        assert torch.equal(x8.view(torch.uint8)[0, part], y8.view(torch.uint8).view(-1))
        assert torch.equal(scale[0, part.start // 128:-(-part.stop // 128)], s.view(-1))
    assert capi.oasr_device_status() == 0


@pytest.mark.gpu
def test_quantize_blocks_edges():
    """Ties to even, magnitudes at 448's border, below the least scale, the largest, and values that are not finite."""
    x = torch.zeros(7, 272)
    x[0, :6] = torch.tensor([448.0, 17.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10])
    x[1, 0], x[1, 1], x[1, 130] = 449.0, 448.0, 448.0
    x[2, 5] = 2.0 ** -140
    x[3, 200] = 3.0e38
    x[4, 3], x[4, 200] = float("nan"), 1.0
    x[5, 260] = float("-inf")
    x8, scale = capi.oasr_quantize_blocks(x.cuda())
    v, byte = x8.cpu().float(), scale.cpu()
    assert v[0, :6].tolist() == [448, 16, 20, -16, 0, 2.0 ** -8] and byte[0].tolist() == [127, 27, 27]
    assert byte[1].tolist() == [128, 127, 27] and v[1, 0] == 224 and v[1, 130] == 448
    assert byte[2, 0] == 27 and not v[2].any() and not v[6].any()
    assert byte[3, 1] == blocks(x[3:4])[1][0, 1] and v[3, 200] == blocks(x[3:4])[0][0, 200]
    assert byte[4].tolist() == [255, blocks(x[6:7] + x[4, 200])[1][0, 1].item(), 27] and v[4, :128].isnan().all()
    assert v[4, 128:].isfinite().all() and byte[5, 2] == 255 and v[5, 256:].isnan().all()
    w8, ws = capi.oasr_quantize_blocks(torch.randn(24, 272, device="cuda"))
    for rows in (slice(0, 7), None):      # few rows, and many
        a8, a = (x8, scale) if rows else (x8.view(torch.uint8).repeat(40, 1).view(torch.float8_e4m3fn), scale.repeat(40, 1))
        out = capi.oasr_linear_e4m3(a8, a, w8, ws).view(-1, 7, 24)
        assert out[:, 4:6].isnan().all() and out[:, [0, 1, 2, 6]].isfinite().all()


SHAPES = [  # M, N, K
    (1, 1, 16), (1, 2048, 512), (2, 37, 80), (4, 64, 1024), (5, 33, 4096), (8, 1000, 528),
    (9, 1, 16), (17, 40, 64), (128, 32, 48), (129, 100, 256), (200, 129, 1024), (1000, 513, 272),
    (64, 4096, 2048), (4096, 640, 128), (2500, 2000, 1024), (130, 72, 4112), (16, 512, 4096), (100, 192, 640),
    (700, 1030, 528), (33, 385, 144), (50001, 700, 400), (140000, 450, 512), (60000, 1024, 128),
]


@pytest.mark.gpu
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K, dtype, bias):
    g = torch.Generator().manual_seed(M + N + K)
    x8, xs = (t.cpu() for t in capi.oasr_quantize_blocks(matrix(g, M, K).cuda()))
    w8, ws = (t.cpu() for t in capi.oasr_quantize_blocks(matrix(g, N, K).cuda()))
    b = torch.randn(N, generator=g).to(DT[dtype]) if bias else None
    keep = torch.full((M * N + 64,), 7.0, dtype=DT[dtype], device="cuda")
    out = keep[:M * N].view(M, N)
    got = capi.oasr_linear_e4m3(x8.cuda(), xs.cuda(), w8.cuda(), ws.cuda(), None if b is None else b.cuda(), out=out)
    assert got is out and bool((keep[M * N:] == 7.0).all())
    if M > 5000:     # every row on the GPU, in 64 bits
        x8, xs, w8, ws, b = (None if t is None else t.cuda() for t in (x8, xs, w8, ws, b))
        want = product(x8, xs, w8, ws, b, DT[dtype])
        assert bool(((out.double() - want[0]).abs() <= want[1]).all())
    else:
        close(out, product(x8, xs, w8, ws, b, DT[dtype]))
    assert capi.oasr_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(9, 512, 2048), (64, 100, 1552), (200, 70, 4096), (128, 64, 2064), (129, 65, 1424),
                                   (10, 41, 16384), (300, 520, 2560), (17, 64, 65536)])
def test_blocks_shared_by_a_cluster(M, N, K, dtype, bias):
    test_linear(M, N, K, dtype, bias)


@pytest.mark.gpu
def test_each_block_of_a_cluster_counts_once():
    """Rows that are zero but for one block, in every share of K, the last shorter block among them; captured, twice the
    same bits."""
    g = torch.Generator().manual_seed(4)
    M, N, K = 70, 100, 2064
    x, w = matrix(g, M, K), matrix(g, N, K).cuda()
    w8, ws = capi.oasr_quantize_blocks(w)
    for b in range(17):
        y = torch.zeros_like(x)
        y[:, 128 * b:128 * b + 128] = x[:, 128 * b:128 * b + 128]
        x8, xs = capi.oasr_quantize_blocks(y.cuda())
        out = capi.oasr_linear_e4m3(x8, xs, w8, ws, out_dtype=torch.float32)
        close(out, product(x8.cpu(), xs.cpu(), w8.cpu(), ws.cpu(), None, torch.float32))
    again = torch.zeros_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        capi.oasr_linear_e4m3(x8, xs, w8, ws, out=again)
    for _ in range(5):
        again.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, again)
    assert capi.oasr_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 300])
def test_each_scale_reaches_its_block(M):
    """One block of one row at a time stands out, in x and in w."""
    N, K = 200, 1200
    kb = -(-K // 128)
    one = torch.full((max(M, N), K), 1.0).to(torch.float8_e4m3fn)
    g = torch.Generator().manual_seed(1)
    xs, ws = (torch.randint(117, 138, (n, kb), generator=g).to(torch.uint8) for n in (M, N))
    out = capi.oasr_linear_e4m3(one[:M].cuda(), xs.cuda(), one[:N].cuda(), ws.cuda(), out_dtype=torch.float32)
    n = torch.tensor([min(128, K - 128 * b) for b in range(kb)], dtype=torch.float64)
    want = (power(xs.long() - 127) * n) @ power(ws.long() - 127).t()
    err = (out.double().cpu() - want).abs() / want
    assert float(err.max()) <= K * 2.0 ** -23


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 2, 3, 9, 200])
def test_scales_whose_product_alone_is_in_range(M, dtype):
    """A block's sum times one of its two scales is past fp32's range, or below it, where the product of all three is
    not: large activations by small weights, and scales of 2^-126 by 2^127."""
    g = torch.Generator().manual_seed(M)
    N, K = 40, 400
    x, w = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g)
    x[:, 200], w[:, 128:256] = 3.0e38, w[:, 128:256].clamp(-3, 3)
    x[:, 128:200], x[:, 201:256], w[:, 200] = 0, 0, 0.5
    w[0, 201] = 3
    x8, xs = (t.cpu() for t in capi.oasr_quantize_blocks(x.cuda()))
    w8, ws = (t.cpu() for t in capi.oasr_quantize_blocks(w.cuda()))
    assert int(xs[0, 1]) - 127 == 120 and 1.0e38 < float(values(x8, xs)[0] @ values(w8, ws)[0]) < 2.0e38
    out = capi.oasr_linear_e4m3(x8.cuda(), xs.cuda(), w8.cuda(), ws.cuda(), out_dtype=DT[dtype])
    close(out, product(x8, xs, w8, ws, None, DT[dtype]))
    xs[:], ws[:] = 1, 254
    out = capi.oasr_linear_e4m3(x8.cuda(), xs.cuda(), w8.cuda(), ws.cuda(), out_dtype=DT[dtype])
    close(out, product(x8, xs, w8, ws, None, DT[dtype]))
    xs[:], ws[:] = 254, 1
    out = capi.oasr_linear_e4m3(x8.cuda(), xs.cuda(), w8.cuda(), ws.cuda(), out_dtype=DT[dtype])
    close(out, product(x8, xs, w8, ws, None, DT[dtype]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(20001, 1024, 16), (19969, 1032, 128), (40033, 512, 16)])
def test_full_tiles_before_one_of_few_rows(M, N, K, dtype):
    """CTAs that take a last row tile of 1, 33 or 97 rows after full ones: warps without rows there leave the tile that
    is still on its way to memory alone.  Short K, so that little time lies between; the same bits every time."""
    g = torch.Generator().manual_seed(K)
    x8, xs = capi.oasr_quantize_blocks(matrix(g, M, K).cuda())
    w8, ws = capi.oasr_quantize_blocks(matrix(g, N, K).cuda())
    want = product(x8, xs, w8, ws, None, DT[dtype])
    first = capi.oasr_linear_e4m3(x8, xs, w8, ws, out_dtype=DT[dtype])
    assert bool(((first.double() - want[0]).abs() <= want[1]).all())
    for _ in range(30):
        assert torch.equal(capi.oasr_linear_e4m3(x8, xs, w8, ws, out_dtype=DT[dtype]), first)
    assert capi.oasr_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(3, 77, 512), (4, 2050, 1024), (5, 512, 512), (5, 100, 1024), (6, 33, 512), (6, 1000, 144),
                                   (7, 512, 512), (8, 100, 16)])
def test_rows_around_the_border_of_the_forms(M, N, K, dtype, bias):
    """Every instance of the form without tiles (1, 2, 3 to 4, 5 to 6 rows) and the first sizes that tiles take."""
    test_linear(M, N, K, dtype, bias)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 2, 4, 5, 6, 40])
def test_blocks_that_stand_for_nan(M, dtype):
    """A scale of 255, of x or of w, makes its row's or its column's results NaN and no other."""
    g = torch.Generator().manual_seed(M)
    N, K = 24, 272
    x, w = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g)
    x[M // 2, 260], w[5, 3], w[9, 200] = float("inf"), float("nan"), float("-inf")
    x8, xs = capi.oasr_quantize_blocks(x.cuda())
    w8, ws = capi.oasr_quantize_blocks(w.cuda())
    assert xs[M // 2].tolist()[2] == 255 and ws[5].tolist()[0] == 255 and ws[9].tolist()[1] == 255
    out = capi.oasr_linear_e4m3(x8, xs, w8, ws, out_dtype=DT[dtype]).cpu()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[M // 2], bad[:, 5], bad[:, 9] = True, True, True
    assert torch.equal(out.isnan(), bad)
    rows, cols = [i for i in range(M) if i != M // 2], [j for j in range(N) if j not in (5, 9)]
    x8, xs, w8, ws = x8.cpu().float()[rows], xs.cpu()[rows], w8.cpu().float()[cols], ws.cpu()[cols]
    if rows:
        close(out[rows][:, cols], product(x8, xs, w8, ws, None, DT[dtype]))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(300, 500, 512), (2, 700, 256)])
def test_same_bits_captured_and_beside_others(M, N, K):
    g = torch.Generator().manual_seed(3)
    sets = []
    for _ in range(3):
        x, w = matrix(g, M, K).to(torch.bfloat16).cuda(), matrix(g, N, K).cuda()
        sets.append((x, *capi.oasr_quantize_blocks(w)))
    run = lambda s, **kw: capi.oasr_linear_e4m3(*capi.oasr_quantize_blocks(s[0], stream=kw.get("stream")), s[1], s[2], **kw)
    want = [run(s) for s in sets]
    outs = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            run(sets[i], out=outs[i])
    for _ in range(20):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        with torch.cuda.stream(streams[2]):
            run(sets[2], out=outs[2])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.gpu
def test_tensors_past_4_gb():
    """Outputs whose byte offsets pass 2^32."""
    M, N, K = 300_000, 4096, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    x8, xs = capi.oasr_quantize_blocks(torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16))
    w8, ws = capi.oasr_quantize_blocks(torch.randn(N, K, generator=g, device="cuda"))
    out = capi.oasr_linear_e4m3(x8, xs, w8, ws, out_dtype=torch.float32)
    for rows in (slice(0, 3), slice(M // 2 - 100, M // 2 + 100), slice(M - 130, M)):
        close(out[rows], product(x8[rows].cpu(), xs[rows].cpu(), w8.cpu(), ws.cpu(), None, torch.float32))
