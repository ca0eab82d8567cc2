"""The 8-bit serving operators of the streaming encoder layer, in their plain form and through the library.

  append    oasr_paged_append_e4m3: a chunk's K/V rows quantised to e4m3 with one power-of-two scale per
            (frame, head) as they are written into the paged pools
  read      oasr_paged_read_e4m3: cached rows read back into dense [B, L, H, 64] tensors
  step      oasr_chunk_step_paged_e4m3: append, then relative-position attention over the 8-bit cache
  linear    oasr_quantize_rows + oasr_linear_w8a8: activations quantised per token, an 8-bit integer
            product with a scale per token and per output channel
  project   oasr_quantize_rows + oasr_project_qkv_pos_w8a8: the same product for a step's q, k, v and
            its relative-position table, in one launch

`run` is one pass: with `own` false in elementary fp32 torch operations, with `own` true the
library's calls.  Pools are [num_blocks, H, block_size, 64] float8_e4m3fn, scales uint8
[num_blocks, H, 2 (K, V), block_size], the byte e standing for 2^(e - 127).
"""
import math

import torch

own = False

D = 64
LEAST = -100          # smallest scale exponent of a cached row
TINY = 2.0 ** -100    # smallest row maximum of quantize_rows


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one stream's single new frame into a small cache: the smallest write of a session
        dict(name="append_one_frame", op="append", B=1, H=4, T=1, C=63, bs=16, dtype="f32", ragged=False),
        # a cohort of 256 streams writing chunks of 64 frames, eight heads: the widest write
        dict(name="append_wide", op="append", B=256, H=8, T=64, C=512, bs=32, dtype="bf16", ragged=True),
        # two streams of uneven length read back to fp32 (inspection, a session moved to another pool)
        dict(name="read_ragged", op="read", B=2, H=4, L=77, C=150, bs=8, dtype="f32", ragged=True),
        # a cohort's whole history read back to bf16
        dict(name="read_cohort", op="read", B=64, H=8, L=1024, C=1024, bs=16, dtype="bf16", ragged=False),
        # one stream with a long history and a single new frame: latency, the split over keys
        dict(name="step_single", op="step", B=1, H=4, T=1, C=8000, bs=16, dtype="bf16", ragged=False),
        # Conformer-small streaming step (64 streams, chunk 16, window 256)
        dict(name="step_small", op="step", B=64, H=4, T=16, C=256, bs=16, dtype="bf16", ragged=False),
        # Conformer-large streaming step (256 streams, chunk 16, window 512)
        dict(name="step_large", op="step", B=256, H=8, T=16, C=512, bs=32, dtype="bf16", ragged=False),
        # chunks of 64 frames, window 1024: the most arithmetic per cached byte, uneven histories
        dict(name="step_wide", op="step", B=128, H=8, T=64, C=1024, bs=16, dtype="bf16", ragged=True),
        # one token through a feed-forward matrix: weight bytes alone
        dict(name="linear_token", op="linear", M=1, N=2048, K=512, dtype="bf16", bias=True),
        # a packed offline batch through a wide layer, fp32 results, odd row count
        dict(name="linear_packed", op="linear", M=8191, N=4096, K=1024, dtype="f32", bias=False),
        # projections of the Conformer-small step
        dict(name="project_small", op="project", M=1024, R=287, H=4, dtype="bf16"),
        # projections of the Conformer-large step
        dict(name="project_large", op="project", M=4096, R=543, H=8, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "step", "step", "step", "linear", "linear", "project"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "linear":
        while True:
            M, N, K = _log(rng, 1, 8191), _log(rng, 40, 4096), 16 * _log(rng, 4, 128)
            if M * N * K <= 8191 * 4096 * 1024:
                return dict(op=op, M=M, N=N, K=K, dtype=dtype, bias=rng.random() < 0.5)
    if op == "project":
        return dict(op=op, M=_log(rng, 1, 4096), R=_log(rng, 31, 1200), H=rng.choice([2, 4, 6, 8]), dtype="bf16")
    bs = rng.choice([8, 16, 32, 64, 128])
    H = rng.choice([1, 2, 3, 4, 8])
    ragged = rng.random() < 0.6
    while True:
        B, T, C = _log(rng, 1, 256), _log(rng, 1, 64), _log(rng, 1, 4000)
        if op == "read":
            L = _log(rng, 1, 1100)
            if B * L * H <= 64 * 1024 * 8 and B * (C + L) * H <= 2_000_000:
                return dict(op=op, B=B, H=H, L=L, C=C, bs=bs, dtype=dtype, ragged=ragged)
        elif op == "append":
            if B * T * H <= 256 * 64 * 8 and B * (C + T) * H <= 2_000_000:
                return dict(op=op, B=B, H=H, T=T, C=C, bs=bs, dtype=dtype, ragged=ragged)
        # the table of a stream may have 512 pages
        elif B * H * T * (C + T) <= 128 * 8 * 64 * (1024 if dtype == "bf16" else 128) and \
                B * H * (C + T) <= 1_100_000 and C + T <= 512 * bs:
            return dict(op=op, B=B, H=H, T=T, C=C, bs=bs, dtype=dtype, ragged=ragged)


def work(case):
    c = case
    if c["op"] in ("linear", "project"):
        e = 2 if c["dtype"] == "bf16" else 4
        if c["op"] == "linear":
            M, N, K = c["M"], c["N"], c["K"]
            # activations in, their 8-bit form and scales out, weights in, results out
            return {"bytes": M * K * (e + 1) + 4 * M + N * K + 4 * N + (e * N if c["bias"] else 0) + e * M * N,
                    "flops": 2 * M * N * K}
        M, R, d = c["M"], c["R"], 64 * c["H"]
        return {"bytes": (M + R) * (d * (e + 1) + 4) + 4 * d * (d + 4) + 3 * d * e + e * d * (3 * M + R),
                "flops": 2 * d * d * (3 * M + R)}
    e = 2 if c["dtype"] == "bf16" else 4
    B, H = c["B"], c["H"]
    mean = c["C"] / 2 if c["ragged"] else c["C"]
    row = D + 1
    if c["op"] == "append":
        n = B * c["T"] * H
        return {"bytes": 2 * n * (D * e + row), "flops": 4 * n * D}
    if c["op"] == "read":
        L = c["L"]
        # frames a stream has in the window it is asked for: reading starts at max(0, len - L)
        kept = _mean_kept(c)
        return {"bytes": int(2 * B * H * (kept * row + L * D * e)), "flops": int(2 * B * H * kept * D)}
    T, R = c["T"], _rows(c)
    n = B * T * H
    return {"bytes": int(2 * B * mean * H * row + 2 * n * row + 4 * n * D * e + R * H * D * e),
            "flops": int(6 * D * B * H * T * (mean + T))}


def _mean_kept(c):
    if not c["ragged"]:
        return min(c["C"], c["L"])
    C, L = c["C"], min(c["L"], c["C"])
    # lengths uniform on 0 .. C
    return (L * (L + 1) / 2 + (C - L) * L) / (C + 1)


def _rows(c):
    return c["C"] + 2 * c["T"] - 1


# ----------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def prepare(case, seed):
    c, g = case, _generator(seed)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    s = {"op": c["op"], "dt": dt}
    if c["op"] == "linear":
        # activations after a norm: unit scale, a few louder channels
        loud = 1 + 7 * (torch.rand(c["K"], generator=g, device="cuda") < 0.02)
        s["x"] = (_normal(g, (c["M"], c["K"]), torch.float32) * loud).to(dt)
        s["w"], s["w_scale"] = _quantised_weight(g, c["N"], c["K"])
        s["bias"] = _normal(g, (c["N"],), dt, 0.1) if c["bias"] else None
        return s
    if c["op"] == "project":
        d = 64 * c["H"]
        s["H"] = c["H"]
        s["x"] = _normal(g, (c["M"], d), dt)
        s["w"], s["w_scale"] = _quantised_weight(g, 3 * d, d)
        s["bias"] = _normal(g, (3 * d,), dt, 0.1)
        s["pos"] = _normal(g, (c["R"], d), dt)
        s["w_pos"], s["w_pos_scale"] = _quantised_weight(g, d, d)
        return s
    B, H, bs = c["B"], c["H"], c["bs"]
    new = c["T"] if c["op"] != "read" else 0
    lens = torch.full((B,), c["C"], dtype=torch.int32, device="cuda")
    if c["ragged"]:
        lens = torch.randint(0, c["C"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    pages = max(1, -(-(c["C"] + new) // bs))
    num = 2 * B * pages     # twice what the streams need, blocks shuffled
    order = torch.randperm(num, generator=g, device="cuda", dtype=torch.int64)
    s["table"] = order[:B * pages].reshape(B, pages).to(torch.int32)
    s["lens"] = lens
    # what earlier steps left in the pools: rows whose largest value fills e4m3's top octave,
    # scales a few octaves apart between frames and heads
    rows = torch.randn((num, H, bs, D), generator=g, device="cuda")
    s["k_pool"] = (rows * (448 / rows.abs().amax(-1, keepdim=True))).to(torch.float8_e4m3fn)
    rows = torch.randn((num, H, bs, D), generator=g, device="cuda")
    s["v_pool"] = (rows * (448 / rows.abs().amax(-1, keepdim=True))).to(torch.float8_e4m3fn)
    s["scale"] = torch.randint(118, 121, (num, H, 2, bs), generator=g, device="cuda", dtype=torch.uint8)
    if c["op"] == "read":
        s["start"] = (lens - c["L"]).clamp_(min=0)      # the latest L frames of each stream
        s["L"] = c["L"]
        return s
    T = c["T"]
    s["k_new"] = _normal(g, (B, T, H, D), dt)
    s["v_new"] = _normal(g, (B, T, H, D), dt)
    if c["op"] == "step":
        s["q"] = _normal(g, (B, T, H, D), dt)
        s["u"] = _normal(g, (H, D), dt, 0.25)
        s["vb"] = _normal(g, (H, D), dt, 0.25)
        s["rel"] = _normal(g, (_rows(c), H, D), dt, 0.5)
        s["most"] = c["C"] + T      # keys of the longest stream a program plans for
    return s


def _quantised_weight(g, N, K):
    """A weight laid out once in 8 bits, a scale for each output channel."""
    w = torch.randn((N, K), generator=g, device="cuda") * (K ** -0.5)
    scale = w.abs().amax(1) / 127
    return torch.round(w / scale[:, None]).clamp_(-127, 127).to(torch.int8), scale


# ------------------------------------------------------------------ run

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import paged_kv_chunk_gb300 as lib
    op = s["op"]
    if op == "linear":
        x8, x_scale = lib.oasr_quantize_rows(s["x"])
        return x8, x_scale, lib.oasr_linear_w8a8(x8, x_scale, s["w"], s["w_scale"], s["bias"], out_dtype=s["dt"])
    if op == "project":
        x8, x_scale = lib.oasr_quantize_rows(s["x"])
        p8, p_scale = lib.oasr_quantize_rows(s["pos"])
        return (x8, x_scale, p8, p_scale) + tuple(lib.oasr_project_qkv_pos_w8a8(
            x8, x_scale, s["w"], s["w_scale"], s["bias"], p8, p_scale, s["w_pos"], s["w_pos_scale"], s["H"]))
    if op == "read":
        return lib.oasr_paged_read_e4m3(s["k_pool"], s["v_pool"], s["scale"], s["table"], s["lens"], s["L"],
                                        start=s["start"], dtype=s["dt"])
    if op == "append":
        lib.oasr_paged_append_e4m3(s["k_new"], s["v_new"], s["k_pool"], s["v_pool"], s["scale"], s["table"],
                                   s["lens"])
        return s["k_pool"], s["v_pool"], s["scale"]
    out = lib.oasr_chunk_step_paged_e4m3(s["q"], s["k_new"], s["v_new"], s["k_pool"], s["v_pool"], s["scale"],
                                         s["table"], s["lens"], s["u"], s["vb"], s["rel"])
    return out, s["k_pool"], s["v_pool"], s["scale"]


def _plain(s):
    op = s["op"]
    if op == "linear":
        x8, x_scale = _plain_rows(s["x"])
        return x8, x_scale, _plain_product(x8, x_scale, s["w"], s["w_scale"], s["bias"], s["dt"])
    if op == "project":
        x8, x_scale = _plain_rows(s["x"])
        p8, p_scale = _plain_rows(s["pos"])
        y = _plain_product(x8, x_scale, s["w"], s["w_scale"], s["bias"], s["dt"])
        q, k, v = y.reshape(y.shape[0], 3, s["H"], D).unbind(1)
        rel = _plain_product(p8, p_scale, s["w_pos"], s["w_pos_scale"], None, s["dt"])
        return x8, x_scale, p8, p_scale, q.contiguous(), k.contiguous(), v.contiguous(), rel.reshape(-1, s["H"], D)
    if op == "read":
        k, v, kept = _plain_gather(s, s["start"], s["L"], s["lens"])
        k = torch.where(kept[:, :, None, None], k, 0.0)
        v = torch.where(kept[:, :, None, None], v, 0.0)
        return k.to(s["dt"]), v.to(s["dt"])
    _plain_append(s)
    if op == "append":
        return s["k_pool"], s["v_pool"], s["scale"]
    return _plain_attention(s), s["k_pool"], s["v_pool"], s["scale"]


def _plain_rows(x):
    x = x.float()
    most = x.abs().amax(1, keepdim=True).clamp(min=TINY)
    return torch.round(x * (127.0 / most)).to(torch.int8), (most / 127.0)[:, 0]


def _plain_product(x8, x_scale, w8, w_scale, bias, dt):
    y = torch.matmul(x8.float(), w8.float().t()) * x_scale[:, None] * w_scale
    return (y if bias is None else y + bias.float()).to(dt)


def _power(byte):
    """2^(byte - 127), exactly: the byte is the exponent field of an fp32 number."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _plain_e4m3(x):
    """e4m3 bytes of rows [..., 64] and the byte of their power-of-two scale."""
    x = x.float()
    most = x.abs().amax(-1)
    part, power = torch.frexp(most)
    e = power - torch.where(part > 0.875, 8, 9)      # 448 = 0.875 * 2^9
    e = torch.where(most > 0, e, LEAST).clamp(min=LEAST)
    q = (x * _power(127 - e)[..., None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), (e + 127).to(torch.uint8)


def _plain_append(s):
    B, T = s["k_new"].shape[:2]
    bs = s["scale"].shape[3]
    at = s["lens"].long()[:, None] + torch.arange(T, device="cuda")
    block = s["table"].long().gather(1, at // bs)
    slot = at % bs
    for i, (new, pool) in enumerate(((s["k_new"], s["k_pool"]), (s["v_new"], s["v_pool"]))):
        q, e = _plain_e4m3(new)
        pool.view(torch.uint8)[block, :, slot] = q
        s["scale"][block, :, i, slot] = e


def _plain_gather(s, start, L, lens):
    """fp32 K and V rows [B, L, H, 64] from each stream's position `start` on, and which of them it has."""
    bs = s["scale"].shape[3]
    at = start.long()[:, None] + torch.arange(L, device="cuda")
    kept = at < lens[:, None]
    block = s["table"].long().gather(1, torch.where(kept, at, 0) // bs)
    slot = torch.where(kept, at, 0) % bs
    both = []
    for i, pool in enumerate((s["k_pool"], s["v_pool"])):
        q = pool.view(torch.uint8)[block, :, slot].view(torch.float8_e4m3fn).float()
        both.append(q * _power(s["scale"][block, :, i, slot])[..., None])
    return both[0], both[1], kept


def _plain_attention(s):
    B, T, H, _ = s["q"].shape
    L, R = s["most"], s["rel"].shape[0]
    lens = s["lens"].long()
    k, v, kept = _plain_gather(s, torch.zeros_like(lens), L, lens + T)
    q = s["q"].float()
    score = torch.einsum("bihd,bjhd->bhij", q + s["u"].float(), k)
    # position term against every table row, then row R - T - C + j - i of it for query i and key j
    term = torch.einsum("bihd,rhd->bhir", q + s["vb"].float(), s["rel"].float())
    i = torch.arange(T, device="cuda")[:, None]
    j = torch.arange(L, device="cuda")
    rho = (R - T - lens)[:, None, None] + j - i
    score += term.gather(3, rho.clamp(0, R - 1)[:, None].expand(B, H, T, L))
    score = (score * D ** -0.5).masked_fill(~kept[:, None, None, :], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p /= p.sum(-1, keepdim=True)
    return torch.einsum("bhij,bjhd->bihd", p, v).to(s["dt"])


# ---------------------------------------------------------------- exact

def exact(case, seed):
    """The operators' definitions in 64 bits (whole numbers have no such value: None)."""
    s = prepare(case, seed)
    op = s["op"]
    if op in ("linear", "project"):
        x, xs = _exact_rows(s["x"])
        y = _exact_product(x, xs, s["w"], s["w_scale"], s["bias"])
        if op == "linear":
            return None, xs, y
        p, ps = _exact_rows(s["pos"])
        d, H = 64 * s["H"], s["H"]
        rel = _exact_product(p, ps, s["w_pos"], s["w_pos_scale"], None)
        return (None, xs, None, ps, y[:, :d].reshape(-1, H, D), y[:, d:2 * d].reshape(-1, H, D),
                y[:, 2 * d:].reshape(-1, H, D), rel.reshape(-1, H, D))
    B, bs = s["table"].shape[0], s["scale"].shape[3]
    lens = s["lens"].tolist()
    # per stream, because each has a length of its own
    if op == "read":
        ks, vs = [], []
        for b, n in enumerate(lens):
            first = max(0, n - s["L"])
            k, v = _exact_history(s, b, first, min(n, first + s["L"]), bs)
            short = s["L"] - k.shape[0]
            ks.append(torch.cat([k, k.new_zeros((short,) + tuple(k.shape[1:]))]))
            vs.append(torch.cat([v, v.new_zeros((short,) + tuple(v.shape[1:]))]))
        return torch.stack(ks), torch.stack(vs)
    k8, ke = _exact_e4m3(s["k_new"])
    v8, ve = _exact_e4m3(s["v_new"])
    T = s["k_new"].shape[1]
    k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
    for b, n in enumerate(lens):
        at = torch.arange(n, n + T, device="cuda")
        block = s["table"][b].long()[at // bs]
        k_pool[block, :, at % bs] = k8[b]
        v_pool[block, :, at % bs] = v8[b]
    if op == "append":
        return k_pool, v_pool, None
    outs = []
    R = s["rel"].shape[0]
    rel, u, vb = s["rel"].double(), s["u"].double(), s["vb"].double()
    for b, n in enumerate(lens):
        k, v = _exact_history(s, b, 0, n, bs)
        k = torch.cat([k, k8[b] * _exact_power(ke[b])[..., None]]).transpose(0, 1)
        v = torch.cat([v, v8[b] * _exact_power(ve[b])[..., None]]).transpose(0, 1)
        q = s["q"][b].double()
        a = (q + u).transpose(0, 1) @ k.transpose(1, 2)
        # query i sees the table rows R - T - n - i .. of its own, one for each key
        g = torch.stack([((q[i] + vb)[None] * rel[R - T - n - i:R - i]).sum(-1).t() for i in range(T)], 1)
        p = torch.softmax((a + g) / 8.0, -1)
        outs.append((p @ v).transpose(0, 1))
    return torch.stack(outs), k_pool, v_pool, None


def _exact_rows(x):
    x = x.double()
    # the definition's steps are fp32: the factor 127 / max and its product with x, each rounded once
    most = x.abs().amax(1).clamp(min=TINY)
    factor = (127.0 / most).float().double()
    return torch.round((x * factor[:, None]).float().double()), most / 127.0


def _exact_product(x, xs, w8, w_scale, bias):
    y = (x @ w8.double().t()) * xs[:, None] * w_scale.double()
    return y if bias is None else y + bias.double()


def _exact_e4m3(x):
    """Values of the e4m3 rows and the exponents of their scales."""
    x = x.double()
    most = x.abs().amax(-1)
    e = torch.where(most > 0, torch.ceil(torch.log2(most / 448.0)), LEAST).clamp(min=LEAST)
    y = x * _exact_power(-e)[..., None]
    octave = (torch.frexp(y)[1] - 1).clamp(min=-6)
    step = _exact_power(octave - 3)
    return torch.round(y / step) * step, e


def _exact_power(e):
    """2^e in 64 bits, without the rounding of a power function."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_history(s, b, first, end, bs):
    at = torch.arange(first, end, device="cuda")
    block = s["table"][b].long()[at // bs]
    k = s["k_pool"].view(torch.uint8)[block, :, at % bs].view(torch.float8_e4m3fn).double()
    v = s["v_pool"].view(torch.uint8)[block, :, at % bs].view(torch.float8_e4m3fn).double()
    power = _exact_power(s["scale"][block, :, :, at % bs].long() - 127)
    return k * power[:, :, 0, None], v * power[:, :, 1, None]
