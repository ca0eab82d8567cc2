"""The 8-bit cache: append, read-back and attention against their definitions in 64 bits."""
import pytest
import torch

from paged_kv_chunk_gb300 import build, capi

import e4m3_ref as ref

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def normal(g, *shape, dtype="bf16", std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(DT[dtype])


def make(B, H, T, Cs, bs, dtype, seed, mbps=None, R=None, std=1.0, fill=True):
    """A cache holding each stream's history, the next chunk and the attention's other inputs."""
    g = torch.Generator().manual_seed(seed)
    need = max(1, -(-(max(Cs) + T) // bs))
    c = ref.Cache(B, H, bs, need if mbps is None else mbps, seed + 1)
    if fill:
        for b in range(B):
            if Cs[b]:
                one = ref.Cache.__new__(ref.Cache)
                one.__dict__.update(c.__dict__, B=1, table=c.table[b:b + 1])
                louder = 2.0 ** torch.randint(-3, 4, (1, Cs[b], H, 1), generator=g)
                one.append(torch.randn(1, Cs[b], H, 64, generator=g) * louder,
                           torch.randn(1, Cs[b], H, 64, generator=g) * louder, [0])
    R = max(Cs) + 2 * T - 1 if R is None else R
    x = dict(q=normal(g, B, T, H, 64, dtype=dtype, std=std), k_new=normal(g, B, T, H, 64, dtype=dtype),
             v_new=normal(g, B, T, H, 64, dtype=dtype), u=normal(g, H, 64, dtype=dtype, std=0.25),
             vb=normal(g, H, 64, dtype=dtype, std=0.25), rel=normal(g, R, H, 64, dtype=dtype, std=0.5))
    return c, x, torch.tensor(Cs, dtype=torch.int32)


def step(c, x, lens, pools=None, fused=True, scale=None):
    k, v, s, table = c.cuda() if pools is None else pools
    d = {n: t.cuda() for n, t in x.items()}
    lens = lens.cuda()
    if fused:
        out = capi.oasr_chunk_step_paged_e4m3(d["q"], d["k_new"], d["v_new"], k, v, s, table, lens, d["u"],
                                              d["vb"], d["rel"], scale=scale)
    else:
        capi.oasr_paged_append_e4m3(d["k_new"], d["v_new"], k, v, s, table, lens)
        out = capi.oasr_chunk_relattn_paged_e4m3(d["q"], k, v, s, table, lens, d["u"], d["vb"], d["rel"],
                                                 scale=scale)
    return out, (k, v, s, table)


def check(c, x, lens, out, dtype, scale=0.125, streams=None):
    """c: the cache after the chunk was appended."""
    T = x["q"].shape[1]
    cap = c.mbps * c.bs
    for b in range(c.B) if streams is None else streams:
        C = int(lens[b])
        K = min(C + T, cap)
        want, tol = ref.attention(x["q"][b], x["u"], x["vb"], x["rel"], c.history(b, K), C, scale, DT[dtype], K)
        err = (out[b].double().cpu() - want).abs()
        assert bool((err <= tol).all()), (b, float((err / tol).max()), float(err.max()))


# ------------------------------------------------------------------- CPU

@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


FAKE = 1 << 20


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), capi.OASR_ERR_INVALID_ARG), (dict(sc=None), capi.OASR_ERR_INVALID_ARG),
    (dict(D=128), capi.OASR_ERR_UNSUPPORTED), (dict(T=0), capi.OASR_ERR_INVALID_ARG),
    (dict(dt=3), capi.OASR_ERR_UNSUPPORTED), (dict(vp=FAKE + 8), capi.OASR_ERR_INVALID_ARG),
    (dict(sc=FAKE + 8), capi.OASR_ERR_INVALID_ARG),
    (dict(T=1 << 27), capi.OASR_ERR_UNSUPPORTED), (dict(B=1 << 28, T=64), capi.OASR_ERR_UNSUPPORTED),
])
def test_append_refusals(lib, kw, expect):
    a = dict(k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, sc=FAKE, nb=16, bs=16, bt=FAKE, mbps=8, cs=FAKE, B=2, T=16, H=4,
             D=64, dt=capi.OASR_BF16)
    a.update(kw)
    assert lib.oasr_paged_append_e4m3(*a.values(), None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), capi.OASR_ERR_INVALID_ARG), (dict(L=0), capi.OASR_ERR_INVALID_ARG),
    (dict(D=32), capi.OASR_ERR_UNSUPPORTED), (dict(dt=2), capi.OASR_ERR_UNSUPPORTED),
    (dict(k=FAKE + 4), capi.OASR_ERR_INVALID_ARG), (dict(L=1 << 28), capi.OASR_ERR_UNSUPPORTED),
])
def test_read_refusals(lib, kw, expect):
    a = dict(kp=FAKE, vp=FAKE, sc=FAKE, nb=16, bs=16, bt=FAKE, mbps=8, cs=FAKE, st=None, k=FAKE, v=FAKE, B=2, L=16,
             H=4, D=64, dt=capi.OASR_BF16)
    a.update(kw)
    assert lib.oasr_paged_read_e4m3(*a.values(), None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), capi.OASR_ERR_INVALID_ARG), (dict(sc=None), capi.OASR_ERR_INVALID_ARG),
    (dict(D=32), capi.OASR_ERR_UNSUPPORTED), (dict(T=65), capi.OASR_ERR_UNSUPPORTED),
    (dict(bs=24), capi.OASR_ERR_UNSUPPORTED), (dict(bs=4), capi.OASR_ERR_UNSUPPORTED),
    (dict(bs=512), capi.OASR_ERR_UNSUPPORTED), (dict(mbps=513), capi.OASR_ERR_UNSUPPORTED),
    (dict(nb=1 << 25), capi.OASR_ERR_UNSUPPORTED), (dict(rel=FAKE + 8), capi.OASR_ERR_INVALID_ARG),
    (dict(R=0), capi.OASR_ERR_INVALID_ARG), (dict(dt=9), capi.OASR_ERR_UNSUPPORTED),
    (dict(k=None), capi.OASR_ERR_INVALID_ARG),
])
def test_step_refusals(lib, kw, expect):
    a = dict(q=FAKE, k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, sc=FAKE, nb=16, bs=16, bt=FAKE, mbps=8, cs=FAKE, u=FAKE,
             vb=FAKE, rel=FAKE, R=95, out=FAKE, B=2, T=16, H=4, D=64, scale=0.125, dt=capi.OASR_BF16)
    a.update(kw)
    assert lib.oasr_chunk_step_paged_e4m3(*a.values(), None) == expect
    if "k" not in kw:
        del a["k"], a["v"]
        assert lib.oasr_chunk_relattn_paged_e4m3(*a.values(), None) == expect


def test_reference_format():
    """The 64-bit definition on rows whose result is known by hand."""
    row = torch.zeros(6, 64, dtype=torch.float64)
    row[1, 0] = 448.0
    row[2, 0] = 449.0                       # one octave up: 449/2 -> 224 (step 16)
    row[3, :3] = torch.tensor([1.0, 1.0625, 2.0 ** -20])   # scale 2^-8: 256, 272 -> tie to 256, subnormal step
    row[4, 0] = 2.0 ** -140
    row[5, 7] = float("inf")
    q, byte = ref.quantise(row)
    assert byte.tolist() == [27, 127, 128, 119, 27, 255]
    assert q[1, 0] == 448 and q[2, 0] == 224 and q[3, 0] == 256 and q[3, 1] == 256 and q[3, 2] == 0
    assert q[4, 0] == 0 and q[5].isnan().all()
    x = torch.randn(200, 64, generator=torch.Generator().manual_seed(0)) * 37
    q, byte = ref.quantise(x)
    again = ref.quantise(ref.values(q, byte))
    assert torch.equal(ref.values(*again), ref.values(q, byte))
    # a rounding of half a step of the value, or of the smallest step for the small ones
    err = (ref.values(q, byte) - x.double()).abs()
    assert bool((err <= torch.maximum(x.double().abs() * 2.0 ** -4, torch.ldexp(torch.tensor(2.0 ** -10, dtype=torch.float64), byte.int() - 127)[:, None])).all())


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the refusal of CPU tensors")
def test_cpu_tensors_are_refused(lib):
    c, x, lens = make(1, 2, 2, [3], 8, "bf16", 0)
    k, v = c.k.view(torch.float8_e4m3fn), c.v.view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        capi.oasr_paged_append_e4m3(x["k_new"], x["v_new"], k, v, c.scale, c.table, lens)
    with pytest.raises(ValueError):
        capi.oasr_paged_read_e4m3(k, v, c.scale, c.table, lens, 0)


# ------------------------------------------------------------------- GPU

@pytest.mark.gpu
@pytest.mark.parametrize("B,H,T,Cs,bs,dtype", [
    (1, 1, 1, [0], 8, "bf16"), (2, 4, 16, [64, 64], 16, "f32"), (3, 3, 7, [5, 0, 30], 8, "bf16"),
    (2, 8, 64, [1, 130], 128, "f32"), (5, 2, 33, [10, 11, 12, 13, 14], 32, "bf16"), (2, 5, 3, [254, 2], 256, "bf16"),
    (3, 2, 9, [6, 13, 20], 10, "f32"),   # a page size that is no power of two
])
def test_append_writes_the_definition(B, H, T, Cs, bs, dtype):
    c, x, lens = make(B, H, T, Cs, bs, dtype, 10 * T + B)
    # rows of every kind: zeros, one value, tiny, subnormal, huge, a row at the edge of an octave
    x["k_new"][0, 0, 0] = 0
    x["v_new"][0, 0, 0] = 0
    x["v_new"][0, 0, 0, 5] = -448
    x["k_new"][-1, -1, -1] *= 2.0 ** -120
    x["v_new"][-1, -1, -1] *= 2.0 ** 120
    k, v, s, table = c.cuda()
    capi.oasr_device_status()
    capi.oasr_paged_append_e4m3(x["k_new"].cuda(), x["v_new"].cuda(), k, v, s, table, lens.cuda())
    c.append(x["k_new"], x["v_new"], lens)
    assert c.same(k, v, s)
    assert capi.oasr_device_status() == 0


@pytest.mark.gpu
def test_append_of_nan_and_infinite_rows():
    c, x, lens = make(2, 2, 4, [3, 9], 8, "f32", 3)
    x["k_new"][0, 1, 1, 63] = float("nan")
    x["v_new"][1, 2, 0, 0] = float("-inf")
    k, v, s, table = c.cuda()
    capi.oasr_paged_append_e4m3(x["k_new"].cuda(), x["v_new"].cuda(), k, v, s, table, lens.cuda())
    c.append(x["k_new"], x["v_new"], lens)
    assert c.same(k, v, s)
    back, _ = capi.oasr_paged_read_e4m3(k, v, s, table, lens.cuda() + 4, 13, dtype=torch.float32)
    assert back[0, 4, 1].isnan().all() and back[0, 4, 0].isfinite().all() and back[0, 5, 1].isfinite().all()
    # the attention of every query that sees the row is NaN, of other heads and streams it is not
    out = capi.oasr_chunk_relattn_paged_e4m3(x["q"].bfloat16().cuda(), k, v, s, table, lens.cuda(),
                                             x["u"].bfloat16().cuda(), x["vb"].bfloat16().cuda(),
                                             x["rel"].bfloat16().cuda())
    assert out[0, :, 1].isnan().all() and out[1, :, 0].isnan().all()
    assert out[0, :, 0].isfinite().all() and out[1, :, 1].isfinite().all()


@pytest.mark.gpu
def test_append_drops_bad_rows_and_says_so():
    c, x, lens = make(3, 2, 6, [5, 20, 4], 8, "bf16", 4, mbps=3)
    c.table[0, 1] = c.nb              # the second page of stream 0 names no block
    k, v, s, table = c.cuda()
    capi.oasr_device_status()
    lens = torch.tensor([5, 20, -2], dtype=torch.int32)   # past the table; a negative length
    capi.oasr_paged_append_e4m3(x["k_new"].cuda(), x["v_new"].cuda(), k, v, s, table, lens.cuda())
    assert capi.oasr_device_status() == capi.STATUS_BOUNDS_BIT
    c.append(x["k_new"], x["v_new"], lens)
    assert c.same(k, v, s)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bs,L,start", [(8, 40, None), (16, 1, None), (32, 77, [0, 3, 60]), (10, 33, [5, 0, 1])])
def test_read_back(dtype, bs, L, start):
    c, x, lens = make(3, 3, 1, [70, 0, 61], bs, dtype, 5)
    k, v, s, table = c.cuda()
    capi.oasr_device_status()
    st = None if start is None else torch.tensor(start, dtype=torch.int32).cuda()
    got = capi.oasr_paged_read_e4m3(k, v, s, table, lens.cuda(), L, start=st, dtype=DT[dtype])
    for b in range(3):
        first = 0 if start is None else start[b]
        want = c.history(b, int(lens[b]))
        for g, w in zip(got, want):
            w = w[first:first + L]
            assert torch.equal(g[b, :w.shape[0]].double().cpu(), w)    # exact in bf16 too
            assert bool((g[b, w.shape[0]:] == 0).all())
    assert capi.oasr_device_status() == 0
    # written again, the rows keep their bytes
    if start is None and L >= 40 and dtype == "bf16":
        capi.oasr_paged_append_e4m3(got[0][:1, :40].contiguous(), got[1][:1, :40].contiguous(), k, v, s, table[:1],
                                    torch.zeros(1, dtype=torch.int32, device="cuda"))
        assert c.same(k, v, s)


@pytest.mark.gpu
def test_read_back_of_bad_rows():
    c, x, lens = make(2, 2, 1, [30, 12], 8, "bf16", 6)
    c.table[0, 1] = -1
    k, v, s, table = c.cuda()
    capi.oasr_device_status()
    got = capi.oasr_paged_read_e4m3(k, v, s, table, lens.cuda(), 30)
    assert capi.oasr_device_status() == capi.STATUS_BOUNDS_BIT
    assert torch.equal(got[0][0].double().cpu(), c.history(0, 30)[0])      # zeros in the page
    got = capi.oasr_paged_read_e4m3(k, v, s, table[1:].contiguous(), lens[1:].cuda(), 5,
                                    start=torch.tensor([-3], dtype=torch.int32, device="cuda"))
    assert capi.oasr_device_status() == capi.STATUS_BOUNDS_BIT
    assert bool((got[0][0, :3] == 0).all())
    assert torch.equal(got[0][0, 3:].double().cpu(), c.history(1, 2)[0])
    got = capi.oasr_paged_read_e4m3(k, v, s, table, torch.tensor([1000, 12], dtype=torch.int32, device="cuda"), 9,
                                    start=torch.tensor([900, 12], dtype=torch.int32, device="cuda"))
    assert capi.oasr_device_status() == capi.STATUS_BOUNDS_BIT and not got[0].any() and not got[1].any()


SHAPES = [
    # B, H, T, Cs, bs
    (1, 1, 1, [0], 8), (1, 1, 1, [1], 8), (2, 2, 1, [63, 64], 16), (2, 4, 16, [64, 64], 16),
    (3, 3, 5, [0, 7, 200], 8), (2, 2, 15, [31, 33], 32), (2, 2, 17, [40, 0], 16), (1, 3, 32, [100], 64),
    (2, 2, 33, [5, 70], 16), (2, 1, 48, [129, 64], 128), (1, 2, 64, [300], 256), (2, 2, 64, [0, 65], 8),
    (1, 1, 16, [575], 16), (1, 1, 16, [576], 16), (1, 1, 16, [577], 16), (1, 2, 32, [1155], 32),   # table segments
    (1, 1, 1, [2047], 16), (1, 2, 16, [1500], 8), (1, 1, 64, [1300], 32),                           # keys over a cluster
    (40, 8, 3, [17] * 40, 16), (170, 2, 2, list(range(170)), 16),                                   # more CTAs than SMs
]


@pytest.mark.gpu
@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("B,H,T,Cs,bs", SHAPES)
def test_attention_bf16(B, H, T, Cs, bs, fused):
    c, x, lens = make(B, H, T, Cs, bs, "bf16", 100 + T)
    capi.oasr_device_status()
    out, pools = step(c, x, lens, fused=fused)
    assert capi.oasr_device_status() == 0
    c.append(x["k_new"], x["v_new"], lens)
    assert c.same(*pools[:3])
    check(c, x, lens, out, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("B,H,T,mode", [(300, 2, 3, "uneven"), (300, 2, 16, "even"), (110, 2, 40, "uneven"),
                                        (90, 3, 64, "even"), (600, 1, 2, "uneven"), (250, 2, 1, "one long")])
def test_many_items_per_cta(B, H, T, mode, fused):
    """More (stream, head, query tile) items than the GPU holds at once, in streams of equal and of
    unequal lengths (which are handed out longest first up to 512 streams)."""
    g = torch.Generator().manual_seed(B + T)
    Cs = [23] * B if mode == "even" else torch.randint(0, 90, (B,), generator=g).tolist()
    if mode == "one long":
        Cs = [3] * B
        Cs[77] = 900
    c, x, lens = make(B, H, T, Cs, 16, "bf16", B * T)
    capi.oasr_device_status()
    out, pools = step(c, x, lens, fused=fused)
    assert capi.oasr_device_status() == 0
    c.append(x["k_new"], x["v_new"], lens)
    assert c.same(*pools[:3])
    check(c, x, lens, out, "bf16", streams=range(B) if T < 16 else list(range(0, B, 7)) + [B - 1])


@pytest.mark.gpu
@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("B,H,T,Cs,bs", SHAPES[:12] + [(1, 1, 1, [700], 16)])
def test_attention_f32(B, H, T, Cs, bs, fused):
    c, x, lens = make(B, H, T, Cs, bs, "f32", 200 + T)
    capi.oasr_device_status()
    out, pools = step(c, x, lens, fused=fused)
    assert capi.oasr_device_status() == 0
    c.append(x["k_new"], x["v_new"], lens)
    assert c.same(*pools[:3])
    check(c, x, lens, out, "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_longer_tables_and_scales(dtype):
    """Spare table pages and rel rows, negative, zero and sharp score scales."""
    for scale, std in ((0.125, 1.0), (-0.3, 1.0), (0.0, 1.0), (1.0, 0.5)):
        c, x, lens = make(2, 2, 6, [50, 21], 16, dtype, 7, mbps=20, R=500, std=std)
        out, _ = step(c, x, lens, scale=scale)
        c.append(x["k_new"], x["v_new"], lens)
        check(c, x, lens, out, dtype, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 20, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_far_magnitudes(T, dtype):
    """Scales far from one on both sides; K small enough for finite scores, V near the type's ends."""
    for kmag, vmag in ((2.0 ** -60, 2.0 ** 100), (2.0 ** -90, 2.0 ** -90), (2.0 ** 5, 2.0 ** 60)):
        c, x, lens = make(1, 2, T, [0], 8, dtype, 8)
        x["k_new"], x["v_new"] = x["k_new"] * kmag, x["v_new"] * vmag
        out, pools = step(c, x, lens)
        c.append(x["k_new"], x["v_new"], lens)
        assert c.same(*pools[:3])
        check(c, x, lens, out, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 20])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_mixed_magnitudes(T, dtype):
    """Zero rows and rows many octaves apart in one stream, in every order: none may disturb the sums
    of the others."""
    C = 70
    for seed, mags in enumerate(((0.0, 1.0), (1.0, 0.0), (2.0 ** 60, 0.0, 1.0), (0.0, 2.0 ** -70, 2.0 ** 90),
                                 (2.0 ** -110, 2.0 ** 30), (2.0 ** 12, 2.0 ** -12, 1.0))):
        c, x, lens = make(1, 2, T, [C], 16, dtype, 30 + seed, fill=False)
        g = torch.Generator().manual_seed(seed)
        # runs of 16 keys (a slice of one warp) first, then key by key
        size = torch.tensor([mags[(j // 16 if j < 48 else j) % len(mags)] for j in range(C + T)])[None, :, None, None]
        k, v = torch.randn(1, C + T, 2, 64, generator=g), torch.randn(1, C + T, 2, 64, generator=g) * size
        c.append(k[:, :C].to(DT[dtype]), v[:, :C].to(DT[dtype]), [0])
        x["k_new"], x["v_new"] = k[:, C:].to(DT[dtype]).contiguous(), v[:, C:].to(DT[dtype]).contiguous()
        out, pools = step(c, x, lens)
        c.append(x["k_new"], x["v_new"], lens)
        assert c.same(*pools[:3])
        check(c, x, lens, out, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 20])
def test_rows_of_far_queries(T):
    """Query rows of magnitudes far from one, each scaled into fp16 by its own power of two."""
    c, x, lens = make(1, 2, T, [70], 16, "bf16", 40)
    mags = torch.tensor([2.0 ** e for e in (-60, 0, 8, -20, 3)])[torch.arange(T) % 5][None, :, None, None]
    x["q"] = (x["q"].float() * mags).bfloat16()
    x["u"], x["vb"] = x["u"] * 2.0 ** -12, x["vb"] * 2.0 ** -12
    for scale in (0.125, 2.0 ** -9):
        out, _ = step(c, x, lens, scale=scale)
        cc, _, _ = make(1, 2, T, [70], 16, "bf16", 40)
        cc.append(x["k_new"], x["v_new"], lens)
        check(cc, x, lens, out, "bf16", scale)


@pytest.mark.gpu
@pytest.mark.parametrize("T,C", [(4, 40), (16, 700), (40, 40)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fused", [True, False])
def test_bad_block_ids_read_as_zero_rows(T, C, dtype, fused):
    c, x, lens = make(3, 2, T, [C, C, C], 16, dtype, 9)
    c.table[0, 1] = c.nb + 5
    c.table[1, (C + 1) // 16] = -7          # a page the chunk lands in
    capi.oasr_device_status()
    out, pools = step(c, x, lens, fused=fused)
    assert capi.oasr_device_status() == capi.STATUS_BOUNDS_BIT
    c.append(x["k_new"], x["v_new"], lens)
    assert c.same(*pools[:3])
    check(c, x, lens, out, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fused", [True, False])
def test_lengths_past_the_table(dtype, fused):
    """Keys past the table are dropped; the distances still count from the stream's position."""
    c, x, lens = make(3, 2, 6, [20, 24, 17], 8, dtype, 11, mbps=3, R=64)
    capi.oasr_device_status()
    out, pools = step(c, x, lens, fused=fused)
    assert capi.oasr_device_status() == capi.STATUS_BOUNDS_BIT
    c.append(x["k_new"], x["v_new"], lens)
    assert c.same(*pools[:3])
    check(c, x, lens, out, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rel_table_too_short(dtype):
    c, x, lens = make(2, 2, 6, [40, 3], 8, dtype, 12, R=30)
    capi.oasr_device_status()
    out, _ = step(c, x, lens)
    assert capi.oasr_device_status() == capi.STATUS_BOUNDS_BIT
    c.append(x["k_new"], x["v_new"], lens)
    check(c, x, lens, out, dtype)


@pytest.mark.gpu
def test_uninitialised_rows_do_not_leak():
    """Everything past each stream's keys holds NaN bytes and NaN scales; no output is NaN."""
    for T, Cs in ((3, [1, 62, 100]), (30, [5, 6, 7])):
        c, x, lens = make(3, 2, T, Cs, 32, "bf16", 13)
        for fused in (True, False):
            out, _ = step(c, x, lens, fused=fused)
            assert out.isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,C,B", [(16, 256, 3), (1, 3000, 1), (64, 200, 2)])
def test_same_bits_every_time_and_permuted_blocks(T, C, B):
    c, x, lens = make(B, 2, T, [C] * B, 16, "bf16", 14)
    first, _ = step(c, x, lens)
    again, _ = step(c, x, lens)
    assert torch.equal(first, again)
    perm = torch.randperm(c.nb, generator=torch.Generator().manual_seed(1))
    inv = torch.argsort(perm)
    c.k, c.v, c.scale = c.k[inv], c.v[inv], c.scale[inv]      # block i moves to perm[i]
    c.table = perm[c.table.long()].to(torch.int32)
    moved, _ = step(c, x, lens)
    assert torch.equal(first, moved)


@pytest.mark.gpu
def test_sessions_with_eviction():
    """Steps and commits as a session runs them, every output against the stream's own history."""
    B, H, T, bs, window = 3, 2, 8, 8, 24
    g = torch.Generator().manual_seed(15)
    c, x, _ = make(B, H, T, [0] * B, bs, "bf16", 15, mbps=5, R=64)
    pools = c.cuda()
    lens = torch.tensor([0, 8, 16], dtype=torch.int32).cuda()
    pre = torch.randn(B, 16, H, 64, generator=g).bfloat16()
    capi.oasr_paged_append_e4m3(pre.cuda(), pre.cuda(), *pools, torch.zeros(B, dtype=torch.int32).cuda())
    past = [[(pre[b, t], pre[b, t]) for t in range(int(lens[b]))] for b in range(B)]
    for n in range(9):
        x["q"], x["k_new"], x["v_new"] = (normal(g, B, T, H, 64) for _ in range(3))
        out, _ = step(c, x, lens, pools=pools)
        for b in range(B):
            C = len(past[b])
            assert C == int(lens[b])
            past[b] += [(x["k_new"][b, t], x["v_new"][b, t]) for t in range(T)]
            hist = [ref.values(*ref.quantise(torch.stack([p[i] for p in past[b]]))) for i in range(2)]
            want, tol = ref.attention(x["q"][b], x["u"], x["vb"], x["rel"], hist, C, 0.125, torch.bfloat16)
            assert bool(((out[b].double().cpu() - want).abs() <= tol).all())
        capi.oasr_window_commit(pools[3], lens, T, bs, window)
        for b in range(B):
            past[b] = past[b][len(past[b]) - int(lens[b]):]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_steps_and_streams(dtype):
    """A captured step replays on new inputs; two streams at once do not disturb each other."""
    cases = [make(2, 2, 16, [40, 90], 16, dtype, 16), make(1, 2, 1, [2500], 16, dtype, 17)]
    runs = []
    for c, x, lens in cases:
        d = {n: t.cuda() for n, t in x.items()}
        pools, ln = c.cuda(), lens.cuda()
        out = torch.empty_like(d["q"])
        runs.append((d, pools, ln, out, torch.cuda.Stream(), torch.cuda.CUDAGraph()))

    def call(r):
        d, (k, v, s, table), ln, out = r[:4]
        capi.oasr_chunk_step_paged_e4m3(d["q"], d["k_new"], d["v_new"], k, v, s, table, ln, d["u"], d["vb"],
                                        d["rel"], out=out)

    for r in runs:
        call(r)
    torch.cuda.synchronize()
    for r in runs:
        with torch.cuda.graph(r[5], stream=r[4]):
            call(r)
    for r, (c, x, lens) in zip(runs, cases):
        g = torch.Generator().manual_seed(18)
        for n in ("q", "k_new", "v_new"):
            x[n] = normal(g, *x[n].shape, dtype=dtype)
            r[0][n].copy_(x[n])
        r[3].zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for r in runs:
            with torch.cuda.stream(r[4]):
                r[5].replay()
    torch.cuda.synchronize()
    for r, (c, x, lens) in zip(runs, cases):
        c.append(x["k_new"], x["v_new"], lens)
        assert c.same(*r[1][:3])
        check(c, x, lens, r[3], dtype)


@pytest.mark.gpu
def test_binding_refusals():
    c, x, lens = make(2, 2, 4, [5, 9], 8, "bf16", 19)
    k, v, s, table = c.cuda()
    d = {n: t.cuda() for n, t in x.items()}
    ln = lens.cuda()

    def go(**kw):
        a = dict(q=d["q"], k_new=d["k_new"], v_new=d["v_new"], k_pool=k, v_pool=v, kv_scale=s, block_table=table,
                 cache_seqlens=ln, pos_bias_u=d["u"], pos_bias_v=d["vb"], rel=d["rel"])
        a.update(kw)
        return capi.oasr_chunk_step_paged_e4m3(**a)

    go()
    for kw in (dict(q=d["q"].transpose(0, 1)), dict(k_pool=k.view(torch.uint8)), dict(kv_scale=s.to(torch.int32)),
               dict(kv_scale=s[:1]), dict(v_pool=v[:1]), dict(k_new=d["k_new"].float()), dict(k_new=d["k_new"][:1]),
               dict(cache_seqlens=ln.long()), dict(block_table=table[:1]), dict(rel=d["rel"][:, :1]),
               dict(pos_bias_u=d["u"][:1]), dict(out=d["q"].float()), dict(q=x["q"]), dict(k_pool=c.k),
               dict(q=torch.empty_strided((2, 4, 2, 64), (1024, 256, 128, 2), dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            go(**kw)
    with pytest.raises(ValueError):
        capi.oasr_paged_read_e4m3(k, v, s, table, ln, 4, start=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        capi.oasr_paged_read_e4m3(k, v, s, table, ln, 4, dtype=torch.float16)
