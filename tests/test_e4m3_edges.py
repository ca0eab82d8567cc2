"""The 8-bit attention where its pieces meet: ring slots used over and over, values at the ends of the formats."""
import threading

import pytest
import torch

from paged_kv_chunk_gb300 import build, capi

import e4m3_ref as ref
from test_e4m3_cache import check, make, step

# ------------------------------------------------------------------- CPU

@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


FAKE = 1 << 20


@pytest.mark.parametrize("dt,H", [(capi.OASR_BF16, 33), (capi.OASR_F32, 43)])
def test_too_many_items_are_refused_before_the_append(lib, dt, H):
    """2^24 streams of 33 frames are rows that the append takes, but more query tiles than the attention can count:
    the step says so before it looks for a device, and so before it enqueues the append."""
    a = dict(q=FAKE, k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, sc=FAKE, nb=16, bs=16, bt=FAKE, mbps=8, cs=FAKE, u=FAKE,
             vb=FAKE, rel=FAKE, R=95, out=FAKE, B=1 << 24, T=33, H=H, D=64, scale=0.125, dt=dt)
    assert lib.oasr_chunk_step_paged_e4m3(*a.values(), None) == capi.OASR_ERR_UNSUPPORTED
    del a["k"], a["v"]
    assert lib.oasr_chunk_relattn_paged_e4m3(*a.values(), None) == capi.OASR_ERR_UNSUPPORTED


# ------------------------------------------------------------------- GPU

@pytest.mark.gpu
@pytest.mark.parametrize("B,T,C", [(40, 16, 700), (12, 40, 900), (3, 1, 4000)])
def test_slots_are_refilled_only_once_read(B, T, C):
    """Long histories, every ring slot refilled many times beside other CTAs: the same bits each time, and
    those of the definition (a copy that lands under a slot's readers changes some of them)."""
    c, x, lens = make(B, 4, T, [C - 5 * (b % 7) for b in range(B)], 16, "bf16", 70 + T)
    pools = c.cuda()
    outs = []
    for fused in (True, False):
        outs.append(step(c, x, lens, pools=pools, fused=fused)[0])
        assert all(torch.equal(step(c, x, lens, pools=pools, fused=fused)[0], outs[-1]) for _ in range(15))
    c.append(x["k_new"], x["v_new"], lens)
    assert c.same(*pools[:3])
    for out in outs:
        check(c, x, lens, out, "bf16", streams=[0, B - 1])
    assert capi.oasr_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 20])
def test_bad_blocks_beside_nan_rows(T):
    """Streams whose pages name no block take their turns in ring slots that held NaN scales: zero rows."""
    B, C = 300, 90
    c, x, lens = make(B, 2, T, [C] * B, 16, "bf16", 80 + T)
    for b in range(0, B, 2):
        c.scale[c.table[b].long()] = 255
        c.table[b + 1, torch.arange(0, c.mbps - 2, 2)] = -1 - b
    for fused in (True, False):
        for _ in range(3):
            out, _ = step(c, x, lens, fused=fused)
            assert out[1::2].isfinite().all()
    assert capi.oasr_device_status() == capi.STATUS_BOUNDS_BIT
    c.append(x["k_new"], x["v_new"], lens)
    check(c, x, lens, out, "bf16", streams=range(1, B, 30))


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("T", [5, 20])
@pytest.mark.parametrize("kind", ["q = u = 0", "q = -u", "tiny"])
def test_rows_without_a_content_term(kind, T, sign):
    """Query rows whose q + u is zero (a padded frame where u is zero) or next to it, with a position term far
    above: 64 products of +-1 and 4, some of them turned, a logit of up to 32."""
    c, x, lens = make(2, 2, T, [70, 0], 16, "bf16", 90 + T)
    x["vb"] = torch.full((2, 64), float(sign), dtype=torch.bfloat16)
    x["rel"] = torch.full_like(x["rel"], 4.0)
    turned = torch.arange(x["rel"].shape[0]) % 5
    for i in range(x["rel"].shape[0]):
        x["rel"][i, :, :6 * int(turned[i])] *= -1
    if kind == "q = u = 0":
        x["q"][:, ::2], x["u"] = 0, torch.zeros_like(x["u"])
    elif kind == "q = -u":
        x["q"][:, ::2] = -x["u"]
        x["vb"] = x["vb"] * 2.0 ** 4
        x["rel"] = x["rel"] * 0.25
    else:
        x["q"][:, ::2], x["u"] = x["q"][:, ::2] * 2.0 ** -120, x["u"] * 2.0 ** -120
    out, _ = step(c, x, lens)
    c.append(x["k_new"], x["v_new"], lens)
    check(c, x, lens, out, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("bs", [8, 32])
@pytest.mark.parametrize("T,dtype", [(1, "bf16"), (6, "bf16"), (16, "bf16"), (20, "bf16"), (6, "f32")])
def test_negative_lengths(T, dtype, bs):
    """Rows at negative positions are dropped on every path: the fused step writes what the append does, the
    other streams are attended to as ever."""
    c, x, lens = make(4, 2, T, [20, 21, 22, 23], bs, dtype, 100 + T)
    lens = torch.tensor([-2, 21, -1000, -2 ** 31], dtype=torch.int32)
    for fused in (True, False):
        capi.oasr_device_status()
        out, pools = step(c, x, lens, fused=fused)
        assert capi.oasr_device_status() == capi.STATUS_BOUNDS_BIT
        d, _, _ = make(4, 2, T, [20, 21, 22, 23], bs, dtype, 100 + T)
        d.append(x["k_new"], x["v_new"], lens)
        assert d.same(*pools[:3])
        check(d, x, lens, out, dtype, streams=[1])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 24])
def test_threads_with_tables_of_many_widths(T):
    """The shared memory of a launch grows with the block table: threads that want different amounts at once."""
    jobs = []
    for i, mbps in enumerate((512, 30, 400, 35)):
        c, x, lens = make(2, 1, T, [150 + i, 7], 8, "bf16", 110 + i, mbps=mbps)
        jobs.append((c, x, lens, c.cuda()))
    torch.cuda.synchronize()
    outs, wrong = [None] * len(jobs), []

    def work(i):
        c, x, lens, pools = jobs[i]
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    outs[i], _ = step(c, x, lens, pools=pools)
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    for (c, x, lens, pools), out in zip(jobs, outs):
        c.append(x["k_new"], x["v_new"], lens)
        assert c.same(*pools[:3])
        check(c, x, lens, out, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 20])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("loud", [2.0 ** 40, 2.0 ** 100])
@pytest.mark.parametrize("gap", [100, 140, 200])
@pytest.mark.parametrize("order", ["early", "late", "apart", "rising"])
def test_zero_value_rows_with_all_the_weight(order, gap, loud, dtype, T):
    """Keys whose value rows are zero take the whole weight, `gap` octaves above keys of large values: in the same
    slices of keys, in stages before them, before stages of rising values.  The row sum spans the scales' range and
    the output is that of the definition, next to nothing.

    The bound takes in what fp32 weights cannot hold: one below 2^-126 may count as zero, at most C + T of them
    with values up to max|v|."""
    C = 220
    c, x, lens = make(1, 2, T, [C], 16, dtype, 120, fill=False)
    k, v = torch.zeros(1, C, 2, 64), torch.randn(1, C, 2, 64, generator=torch.Generator().manual_seed(gap)) * loud
    at = dict(early=[1, 70], late=[14, 218], apart=list(range(64)), rising=list(range(64)))[order]
    k[:, at], v[:, at] = 1.0, 0.0
    if order == "rising":
        v[:, 64:128] *= 2.0 ** -20 / loud
        v[:, 128:192] *= loud ** -0.5
    c.append(k.to(x["q"].dtype), v.to(x["q"].dtype), [0])
    x["q"], x["u"] = torch.full_like(x["q"], gap * 0.6931 / 8), torch.zeros_like(x["u"])     # 64 products times 1/8
    x["rel"], x["k_new"], x["v_new"] = (torch.zeros_like(x[n]) for n in ("rel", "k_new", "v_new"))
    out, pools = step(c, x, lens)
    c.append(x["k_new"], x["v_new"], lens)
    assert c.same(*pools[:3])
    history = c.history(0, C + T)
    want, tol = ref.attention(x["q"][0], x["u"], x["vb"], x["rel"], history, C, 0.125, x["q"].dtype)
    tol = tol + (C + T) * 2.0 ** -126 * float(history[1].abs().max())
    err = (out[0].double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 16, 20, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_query_rows_that_are_not_finite(T, dtype):
    """A query row with a NaN or an infinity is NaN itself; its neighbours in the tile and the next stream are not."""
    c, x, lens = make(3, 2, T, [90, 0, 33], 16, dtype, 130 + T)
    x["q"][0, 1, 0, 3], x["q"][1, T - 1, 1, 63], x["q"][2, 0, 0, 0] = float("nan"), float("inf"), float("-inf")
    for fused in (True, False):
        out, pools = step(c, x, lens, fused=fused)
        for b, t, h in ((0, 1, 0), (1, T - 1, 1), (2, 0, 0)):
            assert out[b, t, h].isnan().all()
        d, y, _ = make(3, 2, T, [90, 0, 33], 16, dtype, 130 + T)
        d.append(y["k_new"], y["v_new"], lens)
        assert d.same(*pools[:3])
        for b, t, h in ((0, 1, 0), (1, T - 1, 1), (2, 0, 0)):
            y["q"][b, t, h] = 0
            out[b, t, h] = step(c, y, lens, fused=fused)[0][b, t, h]
        check(d, y, lens, out, dtype)


@pytest.mark.gpu
def test_calls_on_a_stream_that_is_named():
    """Every call of a step enqueued on a stream given by name, none of it on the current one."""
    c, x, lens = make(2, 2, 9, [70, 12], 16, "bf16", 140)
    pools, d, ln = c.cuda(), {n: t.cuda() for n, t in x.items()}, lens.cuda()
    out = torch.empty_like(d["q"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        capi.oasr_paged_append_e4m3(d["k_new"], d["v_new"], *pools, ln, stream=handle)
        capi.oasr_chunk_relattn_paged_e4m3(d["q"], *pools, ln, d["u"], d["vb"], d["rel"], out=out, stream=handle)
        side.synchronize()
        c.append(x["k_new"], x["v_new"], lens)
        assert c.same(*pools[:3])
        check(c, x, lens, out, "bf16")
