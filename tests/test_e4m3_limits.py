"""The 8-bit cache at the ends of its ranges: the longest block tables, pools past 4 GB, calls side by side."""
import threading

import pytest
import torch

from paged_kv_chunk_gb300 import capi

import e4m3_ref as ref
from test_e4m3_cache import DT, make, normal, step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,bs", [(1, 256), (2, 64), (17, 16)])
def test_longest_tables(T, bs, dtype):
    """512 pages, filled to the last row, with random bytes and scales an octave apart."""
    mbps = 512
    K = mbps * bs
    C = K - T
    g = torch.Generator().manual_seed(bs + T)
    c = ref.Cache(1, 1, bs, mbps, 5)
    for pool in (c.k, c.v):
        pool.copy_(torch.randint(0, 0x78, pool.shape, generator=g) | torch.randint(0, 2, pool.shape, generator=g) << 7)
    c.scale.copy_(torch.randint(118, 120, c.scale.shape, generator=g))
    x = dict(q=normal(g, 1, T, 1, 64, dtype=dtype, std=0.5), k_new=normal(g, 1, T, 1, 64, dtype=dtype),
             v_new=normal(g, 1, T, 1, 64, dtype=dtype), u=normal(g, 1, 64, dtype=dtype, std=0.25),
             vb=normal(g, 1, 64, dtype=dtype, std=0.25), rel=normal(g, C + 2 * T - 1, 1, 64, dtype=dtype, std=0.5))
    lens = torch.tensor([C], dtype=torch.int32)
    capi.oasr_device_status()
    outs = [step(c, x, lens, fused=fused) for fused in (True, False)]
    assert capi.oasr_device_status() == 0
    c.append(x["k_new"], x["v_new"], lens)
    page = c.table[0].long()
    history = [ref.values(pool[page].view(torch.float8_e4m3fn).double(), c.scale[page, :, i])
               .permute(0, 2, 1, 3).reshape(K, 1, 64) for i, pool in enumerate((c.k, c.v))]
    want, tol = ref.attention(x["q"][0], x["u"], x["vb"], x["rel"], history, C, 0.125, DT[dtype])
    for out, pools in outs:
        assert c.same(*pools[:3])
        err = (out[0].double().cpu() - want).abs()
        assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("T", [1, 16, 40])
def test_pages_past_four_gigabytes(T):
    """The same pages at the end of pools of 4.5 GB: the same bits."""
    B, H, bs, nb = 2, 4, 16, 1_100_000
    c, x, lens = make(B, H, T, [70, 9], bs, "bf16", 50)
    small, pools = step(c, x, lens)
    read = capi.oasr_paged_read_e4m3(*pools, (lens + T).cuda(), 70 + T)
    k, v = (torch.empty(nb, H, bs, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    s = torch.empty(nb, H, 2, bs, dtype=torch.uint8, device="cuda")
    shift = nb - c.nb
    for big, part in ((k, c.k), (v, c.v), (s, c.scale)):
        big[shift:] = part.cuda()
    far = (k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), s, (c.table + shift).cuda())
    for fused in (True, False):
        out, _ = step(c, x, lens, pools=far, fused=fused)
        if fused:
            assert torch.equal(out, small)
        assert all(torch.equal(p[shift:], q.view(torch.uint8)) for p, q in zip((k, v, s), pools[:3]))
    again = capi.oasr_paged_read_e4m3(*far, (lens + T).cuda(), 70 + T)
    assert all(torch.equal(p, q) for p, q in zip(read, again))
    assert capi.oasr_device_status() == 0


def test_calls_side_by_side():
    """Threads with streams of their own, each through every call: the bits of one at a time."""
    jobs = []
    for i, (T, dtype) in enumerate(((1, "bf16"), (16, "bf16"), (40, "bf16"), (7, "f32"))):
        c, x, lens = make(3, 2, T, [300, 0, 77], 16, dtype, 60 + i)
        want, pools = step(c, x, lens)
        x8 = torch.randint(-128, 128, (300, 256), dtype=torch.int8, device="cuda")
        w8 = torch.randint(-128, 128, (700, 256), dtype=torch.int8, device="cuda")
        xs, ws = torch.rand(300, device="cuda"), torch.rand(700, device="cuda")
        jobs.append((c, x, lens, want, pools, (x8, xs, w8, ws), capi.oasr_linear_w8a8(x8, xs, w8, ws, out_dtype=DT[dtype])))
    torch.cuda.synchronize()
    wrong = []

    def work(job):
        c, x, lens, want, pools, lin, y = job
        with torch.cuda.stream(torch.cuda.Stream()):
            for n in range(30):
                out, after = step(c, x, lens, fused=True)
                z = capi.oasr_linear_w8a8(*lin, out_dtype=y.dtype)
                if not (torch.equal(out, want) and all(torch.equal(p.view(torch.uint8), q.view(torch.uint8))
                                                       for p, q in zip(after[:3], pools[:3])) and torch.equal(z, y)):
                    wrong.append(n)
                    return

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and capi.oasr_device_status() == 0
