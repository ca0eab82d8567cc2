"""The operators between a batch of requests and a decoder that attends to the encoder's states, in
their plain form and through the library.

  table    oasr_block_table_update: pages taken from and given back to a ring of free blocks as requests
           grow, shrink and end, and the slot of every new row
  append   oasr_paged_append_slots: rows of requests of different lengths into the paged pools by that map
  cross    oasr_cross_attn_packed, oasr_cross_attn_paged: a decoder's tokens (hypotheses side by side) over
           the encoder's states of their utterance, packed or in pages
  linear   oasr_quantize_blocks + oasr_linear_e4m3: activations quantised to e4m3 with one power-of-two
           scale for each 128 values of a row, and their product with weights held the same way

`run` is one pass: with `own` false in elementary fp32 torch operations, with `own` true the library's
calls.
"""
import math

import torch

own = False

D = 64
LEAST = -100     # smallest scale exponent of a block
BLOCK = 128      # values that share a scale


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one session's next chunk of 16 frames: its length crosses into a new page
        dict(name="table_session", op="table", B=1, C=300, grow=16, bs=16, gone=False),
        # a batch of 256 utterances of up to 1500 frames turning over: some end, the others grow
        dict(name="table_batch", op="table", B=256, C=1500, grow=1500, bs=32, gone=True),
        # one session's chunk of encoder states written through its slots, fp32
        dict(name="append_session", op="append", B=1, H=4, grow=16, bs=16, dtype="f32"),
        # the states of an offline batch of 256 utterances (50 to 1500 frames) written into pages
        dict(name="append_batch", op="append", B=256, H=8, grow=1500, bs=32, dtype="bf16"),
        # greedy decoding of one utterance: a single token over its 1500 states, latency
        dict(name="cross_token", op="cross", layout="packed", N=1, H=4, Hkv=4, hyps=1, tlo=1, thi=1, klo=1500,
             khi=1500, bs=16, dtype="bf16", empty=False),
        # a beam of 8 over 256 utterances in pages: the next token of every hypothesis
        dict(name="cross_beam", op="cross", layout="paged", N=256, H=8, Hkv=8, hyps=8, tlo=1, thi=1, klo=50,
             khi=1500, bs=32, dtype="bf16", empty=False),
        # ten hypotheses of each of 64 utterances rescored at once
        dict(name="cross_rescore", op="cross", layout="packed", N=64, H=8, Hkv=8, hyps=10, tlo=2, thi=40, klo=50,
             khi=1500, bs=16, dtype="bf16", empty=False),
        # whole transcripts against their utterances, an offline batch: the most arithmetic
        dict(name="cross_transcripts", op="cross", layout="paged", N=256, H=8, Hkv=8, hyps=1, tlo=20, thi=448,
             klo=50, khi=1500, bs=32, dtype="bf16", empty=True),
        # shared key heads, odd lengths, fp32: a check of a new model against its training code
        dict(name="cross_shared_f32", op="cross", layout="packed", N=5, H=8, Hkv=2, hyps=1, tlo=1, thi=37, klo=3,
             khi=333, bs=16, dtype="f32", empty=True),
        # one token through a projection: weight bytes and launches
        dict(name="linear_token", op="linear", M=1, N=2048, K=512, dtype="bf16", bias=True),
        # keys and values of an offline batch's states (d_model 512, both in one product), odd row count
        dict(name="linear_states", op="linear", M=65537, N=1024, K=512, dtype="bf16", bias=True),
        # a feed-forward matrix back to d_model over a streaming cohort's frames, fp32 results
        dict(name="linear_down", op="linear", M=4096, N=512, K=2048, dtype="f32", bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "append", "cross", "cross", "cross", "cross", "linear", "linear", "linear"])
    if op == "linear":
        while True:
            M, N, K = _log(rng, 1, 65537), _log(rng, 40, 4096), 16 * _log(rng, 4, 128)
            if M * N * K <= 65537 * 1024 * 512 and M * (N + K) <= 65537 * 1536:
                return dict(op=op, M=M, N=N, K=K, dtype=rng.choice(["bf16", "bf16", "f32"]), bias=rng.random() < 0.5)
    bs = rng.choice([8, 16, 32, 64, 128])
    if op == "table":
        B, C, grow = _log(rng, 1, 256), _log(rng, 1, 1500), _log(rng, 1, 1500)
        return dict(op=op, B=B, C=C, grow=grow, bs=bs, gone=rng.random() < 0.5)
    if op == "append":
        while True:
            B, H, grow = _log(rng, 1, 256), rng.choice([1, 2, 3, 4, 8]), _log(rng, 1, 1500)
            dtype = rng.choice(["bf16", "bf16", "f32"])
            if B * H * grow * (1 if dtype == "bf16" else 2) <= 256 * 8 * 1500:
                return dict(op=op, B=B, H=H, grow=grow, bs=bs, dtype=dtype)
    while True:
        N, Hkv, G = _log(rng, 1, 256), rng.choice([1, 2, 4, 8]), rng.choice([1, 1, 1, 2, 3, 4])
        hyps, tlo = _log(rng, 1, 16), _log(rng, 1, 40)
        thi, klo = tlo + _log(rng, 1, 100) - 1, _log(rng, 1, 400)
        khi = klo + _log(rng, 1, 1200) - 1
        f32 = rng.random() < 0.25
        rows = hyps * (tlo + thi) / 2
        cost = N * Hkv * G * rows * (klo + khi) / 2
        if hyps * thi <= 448 and khi <= 512 * bs and \
                cost <= 256 * 8 * 234 * 775 / (16 if f32 else 1) and N * Hkv * khi <= 256 * 8 * 1500 and \
                N * Hkv * G * hyps * thi * khi <= 256 * 8 * 448 * 1500:
            return dict(op=op, layout=rng.choice(["packed", "paged"]), N=N, H=Hkv * G, Hkv=Hkv, hyps=hyps, tlo=tlo, thi=thi,
                        klo=klo, khi=khi, bs=bs, dtype="f32" if f32 else "bf16", empty=rng.random() < 0.3)


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def _grown(c):
    """Rows a stream of a "table" case gets on average: a third of them end where `gone`."""
    return (2 / 3 if c["gone"] else 1) * (1 + c["grow"]) / 2


def work(case):
    c = case
    if c["op"] == "table":
        rows, B = _grown(c) * c["B"], c["B"]
        pages = rows / c["bs"] + (B * c["C"] / 3 / c["bs"] if c["gone"] else 0)
        # both lengths in, offsets out, a page's id from one place to the other, a slot for each row
        return {"bytes": int(8 * B + 4 * (B + 1) + 8 * pages + 4 * B * c["grow"]), "flops": int(rows) + B}
    if c["op"] == "append":
        rows = c["B"] * _mean(c)
        return {"bytes": int(rows * (4 * c["H"] * D * _size(c["dtype"]) + 4)), "flops": int(rows)}
    if c["op"] == "linear":
        M, N, K, e = c["M"], c["N"], c["K"], _size(c["dtype"])
        kb = -(-K // BLOCK)
        # activations in, their 8-bit form and scales out, weights in, results out
        return {"bytes": M * K * (e + 1) + M * kb + N * (K + kb) + (e * N if c["bias"] else 0) + e * M * N,
                "flops": 2 * M * N * K}
    e = _size(c["dtype"])
    full = 1 - (c["N"] + 2) // 4 / c["N"] if c["empty"] else 1      # a quarter of the utterances have no states
    rows, keys = c["N"] * c["hyps"] * (c["tlo"] + c["thi"]) / 2, c["N"] * full * (c["klo"] + c["khi"]) / 2
    return {"bytes": int(2 * rows * c["H"] * D * e + 2 * keys * c["Hkv"] * D * e),
            "flops": int(4 * D * c["H"] * rows * keys / c["N"])}


def _mean(c):
    lo = min(50, c["grow"])
    return (lo + c["grow"]) / 2


# ----------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _uniform(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _spread(g, lo, hi, n):
    """n lengths spread evenly over lo .. hi in random order: their sum goes by the case alone."""
    i = torch.randperm(n, generator=g, device="cuda")
    return (hi - (hi - lo) * i // max(1, n - 1)).to(torch.int32)


def _offsets(n):
    """[0, n0, n0 + n1, ...]"""
    return torch.nn.functional.pad(n.cumsum(0), (1, 0)).to(torch.int32)


def prepare(case, seed):
    c, g = case, _generator(seed)
    s = {"op": c["op"]}
    if c["op"] == "table":
        B, bs = c["B"], c["bs"]
        lens = _uniform(g, 0, c["C"], B) if c["gone"] else torch.full((B,), c["C"], dtype=torch.int32, device="cuda")
        new = lens + _uniform(g, 1, c["grow"], B)
        if c["gone"]:       # a third of the requests end
            new = torch.where(_uniform(g, 0, 2, B) == 0, 0, new)
        width = -(-(c["C"] + c["grow"]) // bs)
        num = 2 * B * width
        order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
        held = (lens + bs - 1) // bs
        first = _offsets(held)
        page = torch.arange(width, device="cuda", dtype=torch.int32)
        table = torch.where(page < held[:, None], order[(first[:B, None] + page).clamp(max=num - 1).long()], -1)
        used, head = int(first[B]), int(torch.randint(num, (1,), generator=g, device="cuda"))
        free = torch.full((num,), -1, dtype=torch.int32, device="cuda")
        free[(head + torch.arange(num - used, device="cuda")) % num] = order[used:]
        state = torch.tensor([head, num - used, 0, 0], dtype=torch.int32, device="cuda")
        s.update(lens=lens, new=new.to(torch.int32), bs=bs, total=B * c["grow"], shape=(B, width), num=num)
        # a session's state as it stands before the call; the call works on `now`, refilled from it in each pass
        s["before"] = torch.cat([table.reshape(-1), free, state])
        s["now"] = s["before"].clone()
        return s
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    s["dt"] = dt
    if c["op"] == "linear":
        # activations after a norm: unit scale, a few louder channels
        loud = 1 + 7 * (torch.rand(c["K"], generator=g, device="cuda") < 0.02)
        s["x"] = (_normal(g, (c["M"], c["K"]), torch.float32) * loud).to(dt)
        s["w"], s["w_scale"] = _plain_blocks(torch.randn((c["N"], c["K"]), generator=g, device="cuda") * c["K"] ** -0.5)
        s["bias"] = _normal(g, (c["N"],), dt, 0.1) if c["bias"] else None
        return s
    if c["op"] == "append":
        B, H, bs = c["B"], c["H"], c["bs"]
        n = _spread(g, min(50, c["grow"]), c["grow"], B)
        cu = _offsets(n)
        rows, width = int(cu[B]), -(-c["grow"] // bs)
        num = B * width
        order = torch.randperm(num, generator=g, device="cuda").reshape(B, width)
        at = torch.arange(rows, device="cuda")
        b = torch.searchsorted(cu[1:].long(), at, right=True)
        t = at - cu.long()[b]
        s["slot_map"] = (order[b, t // bs] * bs + t % bs).to(torch.int32)
        # keys and values side by side, as one product for both leaves them
        s["kv"] = _normal(g, (rows, 2, H, D), dt)
        s["k_pool"], s["v_pool"] = (torch.zeros((num, bs, H, D), dtype=dt, device="cuda") for _ in range(2))
        return s
    N, H, Hkv, bs = c["N"], c["H"], c["Hkv"], c["bs"]
    tokens, keys = _spread(g, c["tlo"], c["thi"], N), _spread(g, c["klo"], c["khi"], N)
    if c["empty"]:
        keys = torch.where(keys.argsort().argsort() % 4 == 1, 0, keys)
    s["cu_q"] = _offsets(tokens * c["hyps"])
    s["keys"] = keys
    s["max_q"], s["max_k"], s["Hkv"] = c["hyps"] * c["thi"], c["khi"], Hkv
    s["q"] = _normal(g, (int(s["cu_q"][N]), H, D), dt)
    s["layout"] = c["layout"]
    if c["layout"] == "packed":
        s["cu_k"] = _offsets(keys)
        kv = _normal(g, (max(1, int(s["cu_k"][N])), 2, Hkv, D), dt)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
    else:
        width = -(-c["khi"] // bs)
        num = N * width + 1
        s["table"] = torch.randperm(num, generator=g, device="cuda")[:N * width].reshape(N, width).to(torch.int32)
        s["k"] = _normal(g, (num, bs, Hkv, D), dt)
        s["v"] = _normal(g, (num, bs, Hkv, D), dt)
    return s


# ------------------------------------------------------------------ run

def run(s):
    return _own(s) if own else _plain(s)


def _views(s):
    """The table, the ring of free blocks and its state within one buffer."""
    (B, width), num = s["shape"], s["num"]
    now = s["now"]
    return now[:B * width].view(B, width), now[B * width:B * width + num], now[B * width + num:]


def _own(s):
    import paged_kv_chunk_gb300 as lib
    op = s["op"]
    if op == "table":
        s["now"].copy_(s["before"])
        table, free, state = _views(s)
        slots, cu = lib.oasr_block_table_update(table, s["lens"], s["new"], free, state, s["bs"], s["total"])
        return table, free, state, slots, cu
    if op == "append":
        lib.oasr_paged_append_slots(s["kv"][:, 0], s["kv"][:, 1], s["k_pool"], s["v_pool"], s["slot_map"])
        return s["k_pool"], s["v_pool"]
    if op == "linear":
        x8, x_scale = lib.oasr_quantize_blocks(s["x"])
        return lib.oasr_linear_e4m3(x8, x_scale, s["w"], s["w_scale"], s["bias"], out_dtype=s["dt"])
    if s["layout"] == "packed":
        return lib.oasr_cross_attn_packed(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["max_q"], s["max_k"])
    return lib.oasr_cross_attn_paged(s["q"], s["k"], s["v"], s["table"], s["keys"], s["cu_q"], s["max_q"])


def _plain(s):
    op = s["op"]
    if op == "table":
        return _plain_table(s)
    if op == "append":
        H = s["kv"].shape[2]
        for i, pool in enumerate((s["k_pool"], s["v_pool"])):
            pool.view(-1, H, D)[s["slot_map"].long()] = s["kv"][:, i]
        return s["k_pool"], s["v_pool"]
    if op == "linear":
        x8, x_scale = _plain_blocks(s["x"])
        y = torch.matmul(_plain_values(x8, x_scale), _plain_values(s["w"], s["w_scale"]).t())
        return (y if s["bias"] is None else y + s["bias"].float()).to(s["dt"])
    return _plain_cross(s)


def _plain_table(s):
    s["now"].copy_(s["before"])
    table, free, state = _views(s)
    (B, width), num, bs = s["shape"], s["num"], s["bs"]
    lens, new = s["lens"].long(), s["new"].long()
    head, count = state[0].long(), state[1].long()
    P0, P1 = (lens + bs - 1) // bs, (new + bs - 1) // bs
    need, give = (P1 - P0).clamp(min=0), (P0 - P1).clamp(min=0)
    a, f = need.sum(), give.sum()
    granted = a <= count
    page = torch.arange(width, device="cuda")
    # pages given back: to the tail of the ring, in the streams' order
    leave = (page >= P1[:, None]) & (page < P0[:, None])
    to = (head + count + (give.cumsum(0) - give)[:, None] + page - P1[:, None]) % num
    take = (page >= P0[:, None]) & (page < P1[:, None]) & granted
    at = (head + (need.cumsum(0) - need)[:, None] + page - P0[:, None]) % num
    got = free[at]
    spare = torch.cat([free, free[:1]])     # a place for what is not written
    spare[torch.where(leave, to, num)] = table
    free.copy_(spare[:num])
    table.copy_(torch.where(take, got, torch.where(leave, -1, table)))
    taken = torch.where(granted, a, 0)
    state.copy_(torch.stack([(head + taken) % num, count - taken + f, torch.where(granted, 0, a - count),
                             state[3].long()]))
    rows = (new - lens).clamp(min=0)
    cu = torch.nn.functional.pad(rows.cumsum(0), (1, 0))
    i = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(cu[1:], i, right=True)
    inside = (b < B) & granted
    b = b.clamp(max=B - 1)
    p = torch.where(inside, lens[b] + i - cu[b], 0)
    slots = torch.where(inside, table[b, p // bs] * bs + p % bs, -1)
    return table, free, state, slots.to(torch.int32), cu.to(torch.int32)


def _power(byte):
    """2^(byte - 127), exactly: the byte is the exponent field of an fp32 number."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _by_block(x):
    """[M, K] as [M, blocks, 128], zeros behind K."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % BLOCK)).view(x.shape[0], -1, BLOCK)


def _plain_blocks(x):
    """e4m3 values of x [M, K] and the bytes of their blocks' power-of-two scales."""
    M, K = x.shape
    x = _by_block(x.float())
    part, power = torch.frexp(x.abs().amax(-1))
    e = power - torch.where(part > 0.875, 8, 9)      # 448 = 0.875 * 2^9
    e = torch.where(part > 0, e, LEAST).clamp(min=LEAST)
    q = (x * _power(127 - e)[..., None]).view(M, -1)[:, :K]
    return q.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _plain_values(q, scale):
    return (_by_block(q.float()) * _power(scale)[..., None]).view(q.shape[0], -1)[:, :q.shape[1]]


def _plain_cross(s):
    N, H, G = s["keys"].shape[0], s["q"].shape[1], s["q"].shape[1] // s["Hkv"]
    cu, keys = s["cu_q"].long(), s["keys"].long()
    i, j = torch.arange(s["max_q"], device="cuda"), torch.arange(s["max_k"], device="cuda")
    kept = j < keys[:, None]
    if s["layout"] == "packed":
        at = torch.where(kept, s["cu_k"].long()[:N, None] + j, 0)
        k, v = s["k"][at].float(), s["v"][at].float()
    else:
        bs = s["k"].shape[1]
        block, slot = s["table"].long()[:, j // bs], j % bs
        k, v = s["k"][block, slot].float(), s["v"][block, slot].float()
    row = i < (cu[1:] - cu[:-1])[:, None]
    q = s["q"][torch.where(row, cu[:N, None] + i, 0)].float().view(N, -1, s["Hkv"], G, D)
    score = torch.einsum("nihgd,njhd->nhgij", q, k) * D ** -0.5
    score.masked_fill_(~kept[:, None, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0))
    del score
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total > 0, total, 1)        # an utterance without states: zeros
    out = torch.einsum("nhgij,njhd->nihgd", p, v).reshape(N, -1, H, D)
    return out[row].to(s["dt"])


# ---------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "table":
        return _exact_table(s)
    if case["op"] == "append":
        slot = s["slot_map"].tolist()
        flat = torch.full((s["k_pool"].shape[0] * s["k_pool"].shape[1],), -1, dtype=torch.int64)
        flat[torch.tensor(slot)] = torch.arange(len(slot))      # which row a slot has
        flat = flat.cuda()
        both = []
        for i in range(2):
            rows = torch.cat([s["kv"][:, i].double(), torch.zeros_like(s["kv"][:1, i]).double()])
            both.append(rows[flat].view(s["k_pool"].shape))
        return tuple(both)
    if case["op"] == "linear":
        y = _exact_blocks(s["x"]) @ _exact_weight(s["w"], s["w_scale"]).t()
        return y if s["bias"] is None else y + s["bias"].double()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    q0, keys = s["cu_q"].tolist(), s["keys"].tolist()
    k0 = s["cu_k"].tolist() if s["layout"] == "packed" else None
    G = s["q"].shape[1] // s["Hkv"]
    for n, L in enumerate(keys):
        if not L:
            continue
        if k0:
            k, v = s["k"][k0[n]:k0[n] + L], s["v"][k0[n]:k0[n] + L]
        else:
            k, v = (t[s["table"][n].long()].reshape(-1, s["Hkv"], D)[:L] for t in (s["k"], s["v"]))
        k, v = (t.double().transpose(0, 1).repeat_interleave(G, 0) for t in (k, v))
        q = s["q"][q0[n]:q0[n + 1]].double().transpose(0, 1)
        p = torch.softmax(q @ k.transpose(1, 2) / math.sqrt(D), -1)
        out[q0[n]:q0[n + 1]] = (p @ v).transpose(0, 1)
    return out


def _exact_table(s):
    (B, width), num, bs = s["shape"], s["num"], s["bs"]
    table, free, state = (t.tolist() for t in _views(s))
    lens, new = s["lens"].tolist(), s["new"].tolist()
    pages = [(-(-c // bs), -(-n // bs)) for c, n in zip(lens, new)]
    wanted = sum(max(0, p1 - p0) for p0, p1 in pages)
    granted = wanted <= state[1]
    state[2] = 0 if granted else wanted - state[1]
    tail = state[0] + state[1]
    slots, cu = [], [0]
    for b, (p0, p1) in enumerate(pages):
        if granted:
            for p in range(p0, p1):
                table[b][p] = free[state[0]]
                state[0] = (state[0] + 1) % num
                state[1] -= 1
        for i in range(lens[b], new[b]):
            slots.append(table[b][i // bs] * bs + i % bs if granted else -1)
        cu.append(len(slots))
    for b, (p0, p1) in enumerate(pages):
        for p in range(p1, p0):
            free[tail % num] = table[b][p]
            table[b][p] = -1
            tail += 1
            state[1] += 1
    slots += [-1] * (s["total"] - len(slots))
    return tuple(torch.tensor(t, dtype=torch.int32, device="cuda") for t in (table, free, state, slots, cu))


def _exact_power(e):
    """2^e in 64 bits, without the rounding of a power function."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_blocks(x):
    """The values that the rows' blocks stand for."""
    M, K = x.shape
    out = torch.empty((M, K), dtype=torch.float64, device=x.device)
    for k in range(0, K, BLOCK):
        v = x[:, k:k + BLOCK].double()
        most = v.abs().amax(1)
        e = torch.where(most > 0, torch.ceil(torch.log2(most / 448.0)), LEAST).clamp(min=LEAST)
        y = v * _exact_power(-e)[:, None]
        step = _exact_power((torch.frexp(y)[1] - 1).clamp(min=-6) - 3)
        out[:, k:k + BLOCK] = torch.round(y / step) * step * _exact_power(e)[:, None]
    return out


def _exact_weight(q, scale):
    return q.double() * _exact_power(scale.long() - 127).repeat_interleave(BLOCK, 1)[:, :q.shape[1]]
