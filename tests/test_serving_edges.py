"""The cache and cross-attention calls where a server meets their edges: offsets past 32 bits, one page under several
tables, captured calls of every kind replayed together, large batches, many rows, a table far longer than the
sequences (needs a B200)."""
import math

import numpy as np
import pytest
import torch

from kv_cases import Cache, bf16, check, decode_want, f64, gen
from oracle import attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tiled_attention_forward_03_b200 as mod
    return mod


def settled(attn):
    torch.cuda.synchronize()
    st, site = attn.device_status()
    assert st == attn.ATTN_OK, f"kernel wait gave up at site {site}"


def same(a, b):
    """Bit for bit (NaN included)."""
    return all(x.shape == y.shape and torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for x, y in zip(a, b, strict=True))


@pytest.mark.parametrize("f8", [False, True])
def test_offsets_past_32_bits(attn, f8):
    """The pages of a small cache at the end of one whose element (bf16: and byte) offsets pass 2^32."""
    small = Cache(51, [150, 33, 0], 2, 128, 64, f8, prefix=130)
    k, v, table, lens, sc = small.on_gpu()
    n = k.shape[0]
    pages = (1 << 32) // k[0].numel() + n + 3 if f8 else (1 << 31) // k[0].numel() + n + 3
    at = pages - n
    big = [torch.empty((pages, *k.shape[1:]), dtype=k.dtype, device="cuda") for _ in "kv"]
    for b, x in zip(big, (k, v)):
        b.view(torch.uint8)[at:].copy_(x.view(torch.uint8))
    scb = {}
    for name, s in sc.items():
        if s is not None:
            scb[name] = torch.zeros((pages, *s.shape[1:]), dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
            scb[name].view(torch.uint8)[at:].copy_(s.view(torch.uint8))
    if not f8:
        sc = {}
    far, prefix = table + at, small.prefix_table.cuda()
    q = bf16(gen(1), 3, 8, 2, 128).cuda()
    assert same(attn.forward_decode(q, *big, far, lens, **scb), attn.forward_decode(q, k, v, table, lens, **sc))
    assert same(attn.cache_read(*big, far, lens, 151, **scb), attn.cache_read(k, v, table, lens, 151, **sc))
    many = q.repeat(30, 1, 1, 1)   # 720 rows a KV head: the prefix on the many-row kernel
    for x, t, m in ((q, 1, lens), (many, 30, lens.repeat(30))):
        a = attn.forward_shared_prefix(x, *big, prefix + at, 130, far.repeat(t, 1), m, **scb)
        b = attn.forward_shared_prefix(x, k, v, prefix, 130, table.repeat(t, 1), m, **sc)
        assert same(a, b)
    new = bf16(gen(2), 3, 2, 5, 128).cuda()
    attn.cache_append(new, new, *big, far, lens, **scb)
    attn.cache_append(new, new, k, v, table, lens, **sc)
    settled(attn)
    for b, x in zip(big, (k, v)):
        assert torch.equal(b.view(torch.uint8)[at:], x.view(torch.uint8))
    for name, s in scb.items():
        assert torch.equal(s.view(torch.uint8)[at:], sc[name].view(torch.uint8))


@pytest.mark.parametrize("f8", [False, True])
def test_one_page_under_several_tables(attn, f8):
    """Sequences that share pages (and one that has the same page twice), and a prefix whose pages are a sequence's own."""
    c = Cache(52, [96, 96, 96], 2, 64, 32, f8, prefix=64)
    c.table[1] = c.table[0]
    c.table[2, 1] = c.table[2, 0]
    c.prefix_table[:] = c.table[0, :2]
    q = bf16(gen(3), 3, 4, 1, 64)
    k, v, table, lens, sc = c.on_gpu()
    o, lse = attn.forward_shared_prefix(q.cuda(), k, v, c.prefix_table.cuda(), 64, table, lens, **sc)
    settled(attn)
    for b in range(3):
        check(f64(o[b]), f64(lse[b]), decode_want(c, f64(q[b]), b, 1 / 8), 64, 1 / 8, 160)


@pytest.mark.parametrize("f8", [False, True])
def test_a_serving_step_captured_twice(attn, f8):
    """Append, decode, decode behind a prefix of many rows, and the cache read back: in two graphs over caches of their
    own, replayed at once, then again with other lengths (the last time past positions that were never written and hold
    NaN); each as the calls made one by one."""
    B = 40   # 320 rows a KV head see the prefix
    make = lambda seed: Cache(seed, [50 + 3 * (i % 5) for i in range(B)], 1, 64, 16, f8, prefix=700)
    q = bf16(gen(4), B, 8, 1, 64).cuda()
    new = bf16(gen(5), B, 1, 1, 64).cuda()
    def step(s):
        attn.cache_append(new, new, s["k"], s["v"], s["table"], s["lens"], **s["sc"])
        n = s["lens"] + 1
        return [*attn.forward_decode(q, s["k"], s["v"], s["table"], n, **s["sc"]),
                *attn.forward_shared_prefix(q, s["k"], s["v"], s["pre"], 700, s["table"], n, **s["sc"]),
                *attn.cache_read(s["k"], s["v"], s["table"], n, 80, **s["sc"])]
    def state(seed):
        c = make(seed)
        k, v, table, lens, sc = c.on_gpu()
        return dict(k=k, v=v, table=table, lens=lens, sc=sc, pre=c.prefix_table.cuda())
    ahead, alone = [state(61), state(62)], [state(61), state(62)]
    step(state(63))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in ahead:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step(s))
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in graphs]
    for by in (0, 1, 5):
        for s in (*ahead, *alone):
            s["lens"] += by
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for s, out in zip(alone, outs):
            assert same(step(s), out)
        settled(attn)


def test_cross_captured_twice_and_replayed_together(attn):
    g = gen(6)
    q = [bf16(g, 2, 8, 300, 64).cuda() for _ in "ab"]
    k, v, do = bf16(g, 2, 2, 500, 64).cuda(), bf16(g, 2, 2, 500, 64).cuda(), bf16(g, 2, 8, 300, 64).cuda()
    lens = torch.tensor([500, 77], dtype=torch.int32).cuda()
    def step(x):
        o, lse = attn.forward_cross(x, k, v, lens)
        return [o, lse, *attn.backward_cross(x, k, v, o, lse, do, lens)]
    want = [step(x) for x in q]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in q:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step(x))
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        step(q[0])   # and an eager one beside them
        settled(attn)
        assert all(same(a, b) for a, b in zip(outs, want))


def test_many_short_sequences(attn):
    """70,000 sequences: past 16 bits in every index of the batch."""
    B, hkv, d, page = 70000, 1, 32, 16
    g = gen(7)
    k, v, q = bf16(g, B, hkv, page, d).cuda(), bf16(g, B, hkv, page, d).cuda(), bf16(g, B, 2, 1, d).cuda()
    table = torch.randperm(B, generator=g).to(torch.int32).view(B, 1).cuda()
    lens = (torch.arange(B, dtype=torch.int32) % 17).cuda()
    o, lse = attn.forward_decode(q, k, v, table, lens)
    settled(attn)
    for b in (0, 1, 16, 32768, 65535, 65536, 65537, 69999):
        n, pg = int(lens[b]), int(table[b, 0])
        check(f64(o[b]), f64(lse[b]), attend(f64(q[b]), f64(k[pg, :, :n]), f64(v[pg, :, :n]), [n], d ** -0.5), d, d ** -0.5, n)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("B,hkv,top,d", [(80, 2, 1200, 64), (50, 4, 900, 128), (230, 2, 400, 96), (3, 2, 500, 32)])
def test_whole_units(attn, f8, B, hkv, top, d):
    """Batches whose units are not split: one to a CTA, one to a warp, and a few short ones."""
    r = np.random.default_rng(12)
    lens = [int(x) for x in r.integers(0, top + 1, B)]
    lens[0], lens[1], lens[-1] = top, 0, top - 1
    c = Cache(56, lens, hkv, d, 32, f8)
    q = bf16(gen(13), B, 4 * hkv, 2, d)
    k, v, table, n, sc = c.on_gpu()
    o, lse = attn.forward_decode(q.cuda(), k, v, table, n, **sc)
    settled(attn)
    for b in (0, 1, 2, B // 2, B - 2, B - 1):
        check(f64(o[b]), f64(lse[b]), decode_want(c, f64(q[b]), b, d ** -0.5), d, d ** -0.5, lens[b])


def test_what_follows_waits_for_unsplit_units(attn):
    """No unit is split, so the joining kernels have nothing to do: a copy of the result behind the call still gets it
    whole."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator(device="cuda").manual_seed(14)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    # decode: as many equal units as CTAs (three an SM)
    B, hkv, d, page, n = 3 * sms // 4, 4, 128, 64, 2560
    k, v, q = rand(B * n // page, hkv, page, d), rand(B * n // page, hkv, page, d), rand(B, 8, 1, d)
    table = torch.arange(B * n // page, dtype=torch.int32, device="cuda").view(B, n // page)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    # cross: a unit for each SM
    qc, kc, vc = rand(sms, 1, 128, d), rand(sms, 1, 8192, d), rand(sms, 1, 8192, d)
    for _ in range(5):
        for call, shape in ((lambda out: attn.forward_decode(q, k, v, table, lens, out=out), q.shape),
                            (lambda out: attn.forward_cross(qc, kc, vc, out=out), qc.shape)):
            out = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
            call(out)
            behind = out.clone()
            settled(attn)
            assert not (out == 7).all(-1).any() and same([behind], [out])


@pytest.mark.parametrize("f8", [False, True])
def test_many_tokens_at_once(attn, f8):
    """2,400 rows a KV head through the decode, most of which see nothing."""
    c = Cache(53, [40, 700], 1, 64, 16, f8)
    q = bf16(gen(8), 2, 8, 300, 64)
    k, v, table, lens, sc = c.on_gpu()
    o, lse = attn.forward_decode(q.cuda(), k, v, table, lens, **sc)
    settled(attn)
    for b in range(2):
        check(f64(o[b]), f64(lse[b]), decode_want(c, f64(q[b]), b, 1 / 8), 64, 1 / 8, c.lens[b])


@pytest.mark.parametrize("f8", [False, True])
def test_a_table_far_longer_than_the_sequences(attn, f8):
    """max_pages * page past 2^31: lengths are what they are, and those past every table clamp."""
    c = Cache(54, [70, 5], 1, 64, 1024, f8)
    q = bf16(gen(9), 2, 4, 1, 64)
    k, v, table, lens, sc = c.on_gpu()
    long = torch.full((2, (1 << 21) + 5), -1, dtype=torch.int32)
    long[:, : table.shape[1]] = c.table
    a = attn.forward_decode(q.cuda(), k, v, long.cuda(), lens, **sc)
    settled(attn)
    for b in range(2):
        check(f64(a[0][b]), f64(a[1][b]), decode_want(c, f64(q[b]), b, 1 / 8), 64, 1 / 8, 70)
    out = attn.cache_read(k, v, long.cuda(), lens, 71, **sc)
    settled(attn)
    assert same(out, attn.cache_read(k, v, table, lens, 71, **sc))


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("short", [0, 1, 40, 70])
def test_the_longest_sequence(attn, f8, prefix, short):
    """2^31 - 1 positions (less a few), all on one page but for the last, whose position 2^31 - 1 is no key and whose key
    there would outweigh all others.  Keys are 0 and values 0 or 1: every sum of a part is exact, the joining adds fewer
    than 1000 of them, and o is the values' mean, rounded to bf16."""
    page, d, n = 1024, 64, (1 << 31) - 1 - short
    g = gen(15)
    k = torch.zeros(2, 1, page, d)
    v = torch.randint(0, 2, (1, 1, page, d), generator=g).float().repeat(2, 1, 1, 1)
    k[1, 0, -1] = 16.0
    counts = ((1 << 21) * v[0, 0].double().sum(0) - v[0, 0, page - 1 - short :].double().sum(0)) / n
    if short:
        k[1, 0, -1 - short :] = 16.0
    dt = torch.float8_e4m3fn if f8 else torch.bfloat16
    k, v = k.to(dt).cuda(), v.to(dt).cuda()
    sc = {x: torch.full((2, 1, page), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
          for x in ("k_scale", "v_scale")} if f8 else {}
    table = torch.zeros(1 << 21, dtype=torch.int32, device="cuda")
    table[-1] = 1
    q = torch.ones(1, 2, 1, d, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    if prefix:
        o, lse = attn.forward_shared_prefix(q, k, v, table, n, table[:1].view(1, 1), lens * 0, **sc)
    else:
        o, lse = attn.forward_decode(q, k, v, table.view(1, -1), lens, **sc)
    settled(attn)
    assert np.all(np.abs(f64(o[0, :, 0]) - counts.numpy()) <= (2.0 ** -8 + 2000 * 2.0 ** -24) * counts.numpy())
    assert np.all(np.abs(f64(lse) - math.log(n)) <= 2000 * 2.0 ** -24 + 2.0 ** -21 * (1 + math.log(n)))


@pytest.mark.parametrize("f8", [False, True])
def test_outputs_beside_others_are_left_alone(attn, f8):
    """Outputs handed in as parts of larger buffers: nothing outside them is written."""
    c = Cache(55, [90, 0, 17], 1, 96, 16, f8, prefix=50)
    k, v, table, lens, sc = c.on_gpu()
    for hq, T in ((3, 1), (7, 3), (20, 3)):
        q = bf16(gen(10), 3, hq, T, 96).cuda()
        room = torch.full((5, hq, T, 96), 7.0, dtype=torch.bfloat16, device="cuda")
        room_l = torch.full((5, hq, T), 7.0, device="cuda")
        attn.forward_shared_prefix(q, k, v, c.prefix_table.cuda(), 50, table, lens, out=room[1:4], lse=room_l[1:4], **sc)
        settled(attn)
        assert (room[::4] == 7).all() and (room_l[::4] == 7).all()
        qn = f64(q)
        for b in range(3):
            check(f64(room[1 + b]), f64(room_l[1 + b]), decode_want(c, qn[b], b, 96 ** -0.5), 96, 96 ** -0.5, 140)


@pytest.mark.parametrize("nq,nk", [(1, 40), (3, 4000), (70, 90), (1000, 33)])
def test_cross_outputs_beside_others_are_left_alone(attn, nq, nk):
    g = gen(11)
    q, k, v, do = bf16(g, 2, 4, nq, 64).cuda(), bf16(g, 2, 2, nk, 64).cuda(), bf16(g, 2, 2, nk, 64).cuda(), bf16(g, 2, 4, nq, 64).cuda()
    lens = torch.tensor([nk, nk // 3], dtype=torch.int32).cuda()
    o, lse = attn.forward_cross(q, k, v, lens)
    grads = attn.backward_cross(q, k, v, o, lse, do, lens)
    room = [torch.full((4, *t.shape[1:]), 7.0, dtype=t.dtype, device="cuda") for t in (o, lse, *grads)]
    attn.forward_cross(q, k, v, lens, out=room[0][1:3], lse=room[1][1:3])
    attn.backward_cross(q, k, v, o, lse, do, lens, dq=room[2][1:3], dk=room[3][1:3], dv=room[4][1:3])
    settled(attn)
    for r, t in zip(room, (o, lse, *grads)):
        assert torch.equal(r[1:3], t) and (r[::3] == 7).all()
