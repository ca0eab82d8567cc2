"""Pages for requests of any lengths and the rows written by their slots, against the definition walked through
one page at a time; every value is a whole number or a copy and has to be equal."""
import random

import pytest
import torch

from paged_kv_chunk_gb300 import build, capi

FAKE = 1 << 20


def walk(table, lens, new, ring, state, bs, total):
    """The call on lists: (table, ring, state, slots, cu) afterwards."""
    table, ring, state = [list(r) for r in table], list(ring), list(state)
    nb, mbps = len(ring), len(table[0])
    lens, new = ([min(max(n, 0), mbps * bs) for n in x] for x in (lens, new))
    pages = [(-(-c // bs), -(-n // bs)) for c, n in zip(lens, new)]
    need = sum(max(0, p1 - p0) for p0, p1 in pages)
    head, count = state[0], state[1]
    ok = need <= count
    tail = head + count
    slots, cu = [], [0]
    for b, (p0, p1) in enumerate(pages):
        for p in range(p0, p1) if ok else ():
            table[b][p] = ring[head % nb]
            head, count = (head + 1) % nb, count - 1
        for i in range(lens[b], new[b]):
            slots.append(table[b][i // bs] * bs + i % bs if ok else -1)
        cu.append(len(slots))
    for b, (p0, p1) in enumerate(pages):
        for p in range(p1, p0):
            ring[tail % nb] = table[b][p]
            table[b][p] = -1
            tail, count = tail + 1, count + 1
    return table, ring, [head, count, 0 if ok else need - state[1], 0], slots[:total] + [-1] * (total - len(slots)), cu


def batch(seed, lens, bs, mbps, nb, head=None, spare=None):
    """A consistent state: streams of the given lengths with pages of a shuffled pool, the rest (or `spare` of it)
    in the ring."""
    rng = random.Random(seed)
    ids = list(range(nb))
    rng.shuffle(ids)
    table = []
    for n in lens:
        held = -(-n // bs)
        table.append([ids.pop() for _ in range(held)] + [-1] * (mbps - held))
    if spare is not None:
        ids = ids[:spare]
    head = rng.randrange(nb) if head is None else head
    ring = [-7] * nb
    for i, x in enumerate(ids):
        ring[(head + i) % nb] = x
    return table, ring, [head, len(ids), 0, 0]


def cuda(*lists):
    return [torch.tensor(x, dtype=torch.int32, device="cuda") for x in lists]


# ------------------------------------------------------------------- CPU

@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


@pytest.mark.parametrize("kw,expect", [
    (dict(bt=None), capi.OASR_ERR_INVALID_ARG), (dict(new=None), capi.OASR_ERR_INVALID_ARG),
    (dict(state=None), capi.OASR_ERR_INVALID_ARG), (dict(slots=None), capi.OASR_ERR_INVALID_ARG),
    (dict(cu=None), capi.OASR_ERR_INVALID_ARG), (dict(B=0), capi.OASR_ERR_INVALID_ARG),
    (dict(bs=0), capi.OASR_ERR_INVALID_ARG), (dict(nb=-1), capi.OASR_ERR_INVALID_ARG),
    (dict(total=-1), capi.OASR_ERR_INVALID_ARG), (dict(B=4097), capi.OASR_ERR_UNSUPPORTED),
    (dict(nb=1 << 27), capi.OASR_ERR_UNSUPPORTED), (dict(mbps=1 << 27), capi.OASR_ERR_UNSUPPORTED),
    (dict(B=4096, mbps=1 << 19), capi.OASR_ERR_UNSUPPORTED),
])
def test_update_refusals(lib, kw, expect):
    a = dict(bt=FAKE, cs=FAKE, new=FAKE, B=4, mbps=8, bs=16, free=FAKE, nb=64, state=FAKE, slots=FAKE, total=64, cu=FAKE)
    a.update(kw)
    assert lib.oasr_block_table_update(*a.values(), None) == expect


@pytest.mark.parametrize("mbps,bs", [(2 ** 31 - 2, 1), (2 ** 31 - 257, 1), (2 ** 30 - 129, 2), (1, 2 ** 30 - 128)])
def test_update_refuses_lengths_within_a_step_of_2_31(lib, mbps, bs):
    """A stream's rows and pages are walked 256 at a time in 32 bits."""
    a = dict(bt=FAKE, cs=FAKE, new=FAKE, B=1, mbps=mbps, bs=bs, free=FAKE, nb=1, state=FAKE, slots=FAKE, total=64, cu=FAKE)
    assert lib.oasr_block_table_update(*a.values(), None) == capi.OASR_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,expect", [
    (dict(k=None), capi.OASR_ERR_INVALID_ARG), (dict(slots=None), capi.OASR_ERR_INVALID_ARG),
    (dict(total=0), capi.OASR_ERR_INVALID_ARG), (dict(ks=255), capi.OASR_ERR_INVALID_ARG),
    (dict(vs=260), capi.OASR_ERR_INVALID_ARG), (dict(kp=FAKE + 8), capi.OASR_ERR_INVALID_ARG),
    (dict(D=60), capi.OASR_ERR_UNSUPPORTED), (dict(dt=2), capi.OASR_ERR_UNSUPPORTED),
    (dict(nb=1 << 27), capi.OASR_ERR_UNSUPPORTED),
])
def test_append_refusals(lib, kw, expect):
    a = dict(k=FAKE, v=FAKE, ks=256, vs=256, kp=FAKE, vp=FAKE, nb=16, bs=16, slots=FAKE, total=8, H=4, D=64, dt=capi.OASR_BF16)
    a.update(kw)
    assert lib.oasr_paged_append_slots(*a.values(), None) == expect


def test_binding_refusals():
    i32 = torch.int32
    table, lens, ring, state = (torch.zeros(s, dtype=i32) for s in ((2, 4), (2,), (8,), (4,)))
    with pytest.raises(ValueError, match="CUDA"):
        capi.oasr_block_table_update(table, lens, lens, ring, state, 16, 32)
    with pytest.raises(ValueError, match=r"\[4\]"):
        capi.oasr_block_table_update(table, lens, lens, ring, state[:3], 16, 32)
    with pytest.raises(ValueError, match="new_seqlens"):
        capi.oasr_block_table_update(table, lens, lens[:1], ring, state, 16, 32)
    with pytest.raises(ValueError, match="slot_map"):
        capi.oasr_block_table_update(table, lens, lens, ring, state, 16, 32, slot_map=torch.zeros(31, dtype=i32))
    x, pool = torch.zeros(6, 2, 64), torch.zeros(3, 4, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        capi.oasr_paged_append_slots(x, x, pool, pool, torch.zeros(6, dtype=i32))
    with pytest.raises(ValueError, match="share"):
        capi.oasr_paged_append_slots(x, x[:5], pool, pool, torch.zeros(6, dtype=i32))
    with pytest.raises(ValueError, match="k_pool"):
        capi.oasr_paged_append_slots(x, x, pool, pool[:2], torch.zeros(6, dtype=i32))
    with pytest.raises(TypeError):
        capi.oasr_paged_append_slots(x.half(), x.half(), pool.half(), pool.half(), torch.zeros(6, dtype=i32))


# ------------------------------------------------------------------- GPU

CASES = [  # lens, new, bs, mbps, spare pages
    ([300], [316], 16, 32, 8),                       # one session's chunk, into a new page
    ([0], [1], 1, 4, 4),
    ([5], [5], 16, 4, 4),                            # no change
    ([16, 17, 0, 31], [17, 0, 33, 32], 16, 4, 9),    # growing, ending, starting, within its page
    ([7, 7, 7], [0, 0, 0], 3, 5, 0),                 # all end, the ring is empty before
    ([0] * 9, [12] * 9, 5, 3, 27),                   # the ring is empty behind
    ([0] * 9, [12] * 9, 5, 3, 26),                   # a page short
    ([40, 3], [0, 50], 8, 7, 2),                     # short, while another stream ends
]


@pytest.mark.gpu
@pytest.mark.parametrize("extra", [0, 37])
@pytest.mark.parametrize("lens,new,bs,mbps,spare", CASES)
def test_update(lens, new, bs, mbps, spare, extra):
    nb = sum(-(-n // bs) for n in lens) + spare + 3
    for head in (0, nb - 1, nb // 2):
        state = batch(len(lens) + head, lens, bs, mbps, nb, head, spare)
        total = sum(max(0, n - c) for c, n in zip(lens, new)) + extra
        want = walk(state[0], lens, new, *state[1:], bs, total)
        table, ring, st, c, n = cuda(*state, lens, new)
        slots, cu = capi.oasr_block_table_update(table, c, n, ring, st, bs, total)
        got = (table, ring, st, slots, cu)
        assert [x.tolist() for x in got] == list(want)
        assert c.tolist() == lens and capi.oasr_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B,bs,longest", [(256, 32, 1500), (1000, 16, 90), (4096, 1, 5)])
def test_update_batches(B, bs, longest):
    """Batches turning over for several rounds: every round's result is the next one's start."""
    rng = random.Random(B)
    lens = [rng.randint(0, longest) for _ in range(B)]
    mbps, nb = -(-2 * longest // bs), B * -(-2 * longest // bs)
    table, ring, state = batch(B, lens, bs, mbps, nb)
    t_d, r_d, s_d = cuda(table, ring, state)
    for _ in range(3):
        new = [rng.choice([0, n, min(2 * longest, n + rng.randint(1, longest)), n // 2]) for n in lens]
        total = sum(max(0, n - c) for c, n in zip(lens, new))
        table, ring, state, slots, cu = walk(table, lens, new, ring, state, bs, total)
        got = capi.oasr_block_table_update(t_d, *cuda(lens, new), r_d, s_d, bs, total)
        assert got[0].tolist() == slots and got[1].tolist() == cu
        assert t_d.tolist() == table and r_d.tolist() == ring and s_d.tolist() == state
        named = [x for c, row in zip(new, table) for x in row[:-(-c // bs)]]
        assert len(set(named)) == len(named)      # no block in two places
        lens = new
    assert capi.oasr_device_status() == 0


@pytest.mark.gpu
def test_update_clamps_what_is_out_of_range():
    """Lengths below zero and past the table, a page that names no block, fewer slots than rows, a ring state that
    no call left behind: flagged, and nothing outside the tensors is touched."""
    bs, mbps, nb = 4, 3, 12
    lens, new = [-3, 5, 2], [6, 99, 4]
    table, ring, state = batch(1, [0, 5, 2], bs, mbps, nb, 10)
    want = walk(table, lens, new, ring, state, bs, 12)
    t, r, s, c, n = cuda(table, ring, state, lens, new)
    slots = torch.full((14,), 77, dtype=torch.int32, device="cuda")
    _, cu = capi.oasr_block_table_update(t, c, n, r, s, bs, 12, slot_map=slots[1:13])
    assert [x.tolist() for x in (t, r, s, slots[1:13], cu)] == list(want)
    assert slots[0] == 77 and slots[13] == 77
    assert capi.oasr_device_status() == capi.STATUS_BOUNDS_BIT
    t, r, s, c, n = cuda(table, ring, state, [0, 5, 2], [1, 6, 3])
    t[1, 1] = nb + 4
    slots, cu = capi.oasr_block_table_update(t, c, n, r, s, bs, 2, slot_map=slots[:2])
    assert cu.tolist() == [0, 1, 2, 3] and slots.tolist()[1] == -1
    assert capi.oasr_device_status() == capi.STATUS_BOUNDS_BIT
    t, r, s, c, n = cuda(table, ring, [nb, 3, 0, 0], [0, 5, 2], [5, 0, 9])
    slots, cu = capi.oasr_block_table_update(t, c, n, r, s, bs, 12)
    assert r.tolist() == ring and set(slots.tolist()) == {-1}
    assert capi.oasr_device_status() == capi.STATUS_BOUNDS_BIT


@pytest.mark.gpu
@pytest.mark.parametrize("head,count", [(12, 3), (-1, 3), (2, 13), (2, -1), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_update_with_a_state_out_of_range(head, count):
    """Nothing is handed out, no page is lost: table, ring and the state's first two stay; rows within a page that a
    stream has get their slots where no stream needs a new page."""
    bs, mbps, nb = 4, 3, 12
    for lens, new in (([0, 9, 2], [5, 0, 9]), ([0, 9, 2], [0, 1, 4])):
        table, ring, _ = batch(4, lens, bs, mbps, nb)
        t, r, s, c, n = cuda(table, ring, [head, count, 0, 0], lens, new)
        slots, cu = capi.oasr_block_table_update(t, c, n, r, s, bs, 16)
        assert t.tolist() == table and r.tolist() == ring and s.tolist()[:2] == [head, count] and s.tolist()[3] == 0
        if new[2] == 4:
            assert slots.tolist() == [table[2][0] * bs + 2, table[2][0] * bs + 3] + [-1] * 14 and cu.tolist() == [0, 0, 0, 2]
        else:
            assert set(slots.tolist()) == {-1} and cu.tolist() == [0, 5, 5, 12] and s.tolist()[2] > 0
        assert capi.oasr_device_status() == capi.STATUS_BOUNDS_BIT


def walk_any(table, lens, new, ring, state, bs, total):
    """`walk` where entries given back may name no block: (table, the ring's ids in their order, count, short, slots,
    cu)."""
    nb, (head, count) = len(ring), state[:2]
    free = [ring[(head + i) % nb] for i in range(count)]
    back = []
    for b, (c, n) in enumerate(zip(lens, new)):
        back += [x for x in table[b][-(-n // bs):-(-c // bs)] if 0 <= x < nb]
    table, _, (_, _, short, _), slots, cu = walk(table, lens, new, ring, state, bs, total)
    got = sum(max(0, -(-n // bs) - -(-c // bs)) for c, n in zip(lens, new))
    free = (free if short else free[got:]) + back
    return table, free[:nb], len(free[:nb]), short, slots, cu


def live(ring, state):
    ring, (head, count, _, zero) = ring.tolist(), state.tolist()
    assert zero == 0
    return [ring[(head + i) % len(ring)] for i in range(count)], count


@pytest.mark.gpu
def test_update_short_and_repeated():
    """A short call, then the same call again: what the shrinking streams gave back counts once."""
    lens, new, bs, mbps, nb = [40, 3], [0, 50], 8, 7, 16
    table, ring, state = batch(1, lens, bs, mbps, nb, 3, 2)
    t, r, s, c, n = cuda(table, ring, state, lens, new)
    slots, _ = capi.oasr_block_table_update(t, c, n, r, s, bs, 50)
    assert s.tolist()[1:3] == [7, 4] and set(slots.tolist()) == {-1}
    assert live(r, s)[0] == [ring[3], ring[4]] + table[0][:5]
    slots, cu = capi.oasr_block_table_update(t, c, n, r, s, bs, 50)
    assert t.tolist()[0] == [-1] * 7 and t.tolist()[1] == [table[1][0], ring[3], ring[4]] + table[0][:4]
    assert live(r, s) == ([table[0][4]], 1) and s.tolist()[2] == 0
    row = t.tolist()[1]
    assert slots.tolist() == [row[i // bs] * bs + i % bs for i in range(3, 50)] + [-1] * 3 and cu.tolist() == [0, 0, 47]
    assert capi.oasr_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("commit", ["the shorter", "all"])
@pytest.mark.parametrize("B,bs,longest", [(3, 4, 60), (40, 8, 300), (700, 2, 40), (30, 1, 3000)])
def test_update_of_a_pool_that_is_too_small(B, bs, longest, commit):
    """A pool of half of what the streams want, through thirty batches: free and held ids stay apart and whole, where
    the lengths committed after a short call are the shorter ones and also where they are all committed."""
    rng = random.Random(B)
    mbps = -(-longest // bs)
    nb = B * mbps // 4 + 2
    lens = [0] * B
    table, ring, state = batch(B, lens, bs, mbps, nb)
    t, r, s = cuda(table, ring, state)
    cut = lambda: [row[:] for row in t.tolist()]
    shorts = 0
    for step in range(30):
        new = [rng.choice([0, n, n // 2, min(longest, n + rng.randint(1, longest))]) for n in lens]
        if step % 10 == 9:
            new = [0] * B
        total = sum(max(0, n - c) for c, n in zip(lens, new))
        want = walk_any(cut(), lens, new, r.tolist(), s.tolist(), bs, total)
        slots, cu = capi.oasr_block_table_update(t, *cuda(lens, new), r, s, bs, total)
        short = s.tolist()[2]
        shorts += short > 0
        ids, count = live(r, s)
        assert (t.tolist(), ids, count, short, cu.tolist()) == want[:4] + want[5:]
        if commit != "all":
            assert slots.tolist() == want[4]
        held = [x for row in t.tolist() for x in row if x != -1]
        assert sorted(held + ids) == list(range(nb))       # no block lost, none in two places
        lens = new if commit == "all" or not short else [min(c, n) for c, n in zip(lens, new)]
        # a stream that was refused and committed all the same has pages missing: its next slots are flagged
        assert capi.oasr_device_status() == 0 or commit == "all"
    assert shorts > 1


@pytest.mark.gpu
@pytest.mark.parametrize("room", ["enough", "too little"])
@pytest.mark.parametrize("B", [2, 9, 600])
def test_update_entries_that_name_no_block(B, room):
    """Entries of -1, of other negative values and of large ones among those given back, more of them than a step of the
    sorting takes; and more entries than the ring has places."""
    rng = random.Random(B)
    bs, mbps = 1, 5000 if B < 10 else 40
    nb = 4 * B * mbps if room == "enough" else B * mbps // 20
    ids = rng.sample(range(nb), nb * 9 // 10)
    held, spare = (ids[:B * mbps // 2], ids[-nb // 2:]) if room == "enough" else (ids[:nb // 2], ids[nb // 2:])
    places = set(rng.sample(range(B * mbps), len(held)))
    fill = iter(held)
    table = [[next(fill) if b * mbps + p in places else -1 for p in range(mbps)] for b in range(B)]
    for flagged in (False, True):
        ring = [-7] * nb
        head = nb - 5
        for i, x in enumerate(spare):
            ring[(head + i) % nb] = x
        if flagged:
            b, p = next((b, p) for b in range(B) for p in range(mbps) if table[b][p] == -1)
            table[b][p] = nb
            b, p = next((b, p) for b in reversed(range(B)) for p in reversed(range(mbps)) if table[b][p] == -1)
            table[b][p] = -2 ** 31
        lens, new = [mbps] * B, [0] * B
        new[B // 2] = 3
        state = [head, len(spare), 0, 0]
        want = walk_any(table, lens, new, ring, state, bs, 5)
        t, r, s, c, n = cuda(table, ring, state, lens, new)
        slots, cu = capi.oasr_block_table_update(t, c, n, r, s, bs, 5)
        got, count = live(r, s)
        assert (t.tolist(), got, count) == want[:3] and slots.tolist() == [-1] * 5 and not any(cu.tolist())
        assert capi.oasr_device_status() == (capi.STATUS_BOUNDS_BIT if flagged else 0)


@pytest.mark.gpu
def test_update_more_pages_than_were_ever_out():
    """A block in two streams' tables: the ring is full before all are back, the rest is dropped and flagged."""
    bs, mbps, nb = 2, 4, 6
    t, r, s, c, n = cuda([[0, 1, 2, 3], [3, 2, 1, 0]], [4, 5, -7, -7, -7, -7], [0, 2, 0, 0], [8, 8], [0, 0])
    capi.oasr_block_table_update(t, c, n, r, s, bs, 0)
    assert live(r, s) == ([4, 5, 0, 1, 2, 3], 6) and set(t.flatten().tolist()) == {-1}
    assert capi.oasr_device_status() == capi.STATUS_BOUNDS_BIT


@pytest.mark.gpu
def test_update_captured():
    """A captured update replayed: each replay goes on from the state that the last one left."""
    bs, mbps, nb = 16, 8, 40
    lens, new = [20, 0, 64], [40, 16, 0]
    table, ring, state = batch(3, lens, bs, mbps, nb)
    t, r, s, c, n = cuda(table, ring, state, lens, new)
    slots, cu = torch.empty(40, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        capi.oasr_block_table_update(t, c, n, r, s, bs, 40, slot_map=slots, cu_seqlens=cu)
        c.copy_(n)
    for step in ([40, 16, 0], [56, 32, 8], [0, 0, 0], [3, 70, 100]):
        n.copy_(torch.tensor(step, dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        table, ring, state, want, offsets = walk(table, lens, step, ring, state, bs, 40)
        assert [x.tolist() for x in (t, r, s, slots)] == [table, ring, state, want]
        assert cu.tolist() == offsets
        lens = step
        capi.oasr_device_status()


@pytest.mark.gpu
def test_update_captured_flags_only_what_is_out_of_range():
    """Replays whose rows fit `total` raise nothing; those with more rows do, and the next ones nothing again."""
    bs, mbps, nb, total = 16, 8, 40, 40
    lens = [20, 0, 64]
    table, ring, state = batch(3, lens, bs, mbps, nb)
    t, r, s, c, n = cuda(table, ring, state, lens, lens)
    slots = torch.empty(total, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    capi.oasr_device_status()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        capi.oasr_block_table_update(t, c, n, r, s, bs, total, slot_map=slots)
        c.copy_(n)
    for step in ([40, 16, 0], [56, 32, 8], [0, 0, 0], [3, 70, 100], [0, 70, 110], [128, 128, 128], [0, 0, 0]):
        n.copy_(torch.tensor(step, dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        fits = sum(max(0, b - a) for a, b in zip(lens, step)) <= total
        table, ring, state, want, _ = walk(table, lens, step, ring, state, bs, total)
        assert [x.tolist() for x in (t, r, s, slots)] == [table, ring, state, want]
        assert capi.oasr_device_status() == (0 if fits else capi.STATUS_BOUNDS_BIT)
        lens = step


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,H,D,bs", [(1, 1, 64, 16), (7, 4, 64, 8), (333, 8, 64, 32), (40, 3, 64, 5), (65, 5, 8, 16),
                                         (12, 20, 128, 7)])
def test_append_slots(rows, H, D, bs, dtype):
    g = torch.Generator().manual_seed(rows)
    nb = rows // bs + 3
    kv = torch.randn(rows, 2, H, D, generator=g).to(dtype).cuda()
    slots = torch.randperm(nb * bs, generator=g)[:rows].to(torch.int32)
    slots[rows // 2] = -1 if rows > 1 else slots[0]
    pools = [torch.randn(nb, bs, H, D, generator=g).to(dtype).cuda() for _ in range(2)]
    want = [p.clone() for p in pools]
    keep = slots >= 0
    for i, w in enumerate(want):
        w.view(-1, H, D)[slots[keep].long().cuda()] = kv[keep.cuda(), i]
    for k, v in ((kv[:, 0], kv[:, 1]), (kv[:, 0].contiguous(), kv[:, 1].contiguous())):
        out = [p.clone() for p in pools]
        capi.oasr_paged_append_slots(k, v, *out, slots.cuda())
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out, want))
    assert capi.oasr_device_status() == 0


@pytest.mark.gpu
def test_append_slots_named_twice():
    """Each 16 bytes of such a slot are one of its rows', the slots beside it are not touched."""
    k = torch.arange(1, 65, device="cuda").view(64, 1, 1).expand(64, 16, 64).to(torch.bfloat16).contiguous()
    pools = [torch.zeros(3, 1, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = torch.full((64,), 1, dtype=torch.int32, device="cuda")
    capi.oasr_paged_append_slots(k, -k, *pools, slots)
    for p, sign in zip(pools, (1, -1)):
        got = sign * p[1].view(-1, 8).float()
        assert bool((got == got[:, :1]).all()) and bool(((got >= 1) & (got <= 64)).all())
        assert not p[0].any() and not p[2].any()
    assert capi.oasr_device_status() == 0


@pytest.mark.gpu
def test_append_slots_out_of_range():
    k = torch.randn(6, 2, 64, device="cuda")
    pools = [torch.zeros(2, 4, 2, 64, device="cuda") for _ in range(2)]
    capi.oasr_paged_append_slots(k, -k, *pools, torch.tensor([8, -2, 3, -1, 0, 2 ** 31 - 1], dtype=torch.int32, device="cuda"))
    assert capi.oasr_device_status() == capi.STATUS_BOUNDS_BIT
    want = torch.zeros(8, 2, 64, device="cuda")
    want[3], want[0] = k[2], k[4]
    assert torch.equal(pools[0].view(8, 2, 64), want) and torch.equal(pools[1].view(8, 2, 64), -want)


@pytest.mark.gpu
def test_append_slots_past_4_gb():
    """Rows whose byte offsets pass 2^32 in the pools."""
    nb, bs, H = 140000, 64, 4
    pools = [torch.zeros(nb, bs, H, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k = torch.randn(5, H, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([nb * bs - 1, 0, nb * bs // 2, 1, nb * bs - 2], dtype=torch.int32, device="cuda")
    capi.oasr_paged_append_slots(k, 2 * k, *pools, slots)
    for i, p in enumerate(pools):
        p = p.view(-1, H, 64)
        assert torch.equal(p[slots.long()], (i + 1) * k)
        assert int((p[nb * bs // 4:] != 0).any(-1).any(-1).sum()) == 3
    assert capi.oasr_device_status() == 0
