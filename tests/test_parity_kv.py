"""The paged cache and the attention over it against the fp64 oracle (needs a B200)."""
import math

import numpy as np
import pytest
import torch

from kv_cases import Cache, bf16, check, decode_want, f64, gen
from oracle import gather, page_row, quantise_row

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


# ---------------------------------------------------------------- cache_append, cache_read

def _special_rows(x):
    """Rows at the borders of the quantiser, over the first rows of x [.., D]."""
    r = x.view(-1, x.shape[-1])
    for i, v in enumerate((0.0, 448.0, 450.0, 1.75, 1.7578125, 3.3895313892515355e38, 2.0 ** -130, 9.1835e-41,
                           math.inf, -math.inf, math.nan)):
        if i < r.shape[0]:
            r[i] = r[i] * 0.01
            r[i, i % r.shape[1]] = v
    return x


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("B,hkv,T,d,page,lens,new", [
    (1, 1, 1, 32, 16, [0], None),
    (3, 2, 1, 64, 16, [15, 16, 31], None),
    (2, 3, 37, 96, 48, [0, 100], [37, 5]),
    (4, 2, 20, 128, 32, [5, 0, 63, 1], [0, 20, 1, 19]),
    (2, 5, 70, 128, 64, [3, 60], [69, 0]),
])
def test_append_writes_these_rows_and_no_others(attn, f8, B, hkv, T, d, page, lens, new):
    g = gen(7)
    per = -(-(max(lens) + T) // page)
    pages = B * per + 2
    table = torch.randperm(pages, generator=g)[: B * per].view(B, per).to(torch.int32)
    k, v = _special_rows(bf16(g, B, hkv, T, d)), _special_rows(bf16(g, B, hkv, T, d).flip(0).contiguous())
    shape = (pages, hkv, page)
    if f8:
        caches = [torch.randint(0, 256, (*shape, d), generator=g).to(torch.uint8).view(torch.float8_e4m3fn) for _ in "kv"]
        scales = [torch.randint(0, 256, shape, generator=g).to(torch.uint8).view(torch.float8_e8m0fnu) for _ in "kv"]
    else:
        caches, scales = [bf16(g, *shape, d) for _ in "kv"], [None, None]
    gc = [c.cuda() for c in caches]
    gs = [None if s is None else s.cuda() for s in scales]
    counts = None if new is None else torch.tensor(new, dtype=torch.int32).cuda()
    attn.cache_append(k.cuda(), v.cuda(), *gc, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                      new_lens=counts, k_scale=gs[0], v_scale=gs[1])
    settled(attn)
    bits = torch.uint8 if f8 else torch.int16
    for x, cache, scale, gcache, gscale in zip((k, v), caches, scales, gc, gs):
        want = cache.clone()
        want_scale = scale.view(torch.uint8).clone() if f8 else None
        for b in range(B):
            for t in range(T if new is None else new[b]):
                i, row = page_row(table[b].tolist(), page, pages, lens[b] + t)
                for h in range(hkv):
                    if f8:
                        codes, byte = quantise_row(f64(x[b, h, t]))
                        want[i, h, row] = torch.tensor(codes, dtype=torch.float32).to(torch.float8_e4m3fn)
                        want_scale[i, h, row] = byte
                    else:
                        want[i, h, row] = x[b, h, t]
        # zeros may carry either sign; NaN payloads of untouched bytes must stay: compare values, then bits elsewhere
        same = gcache.cpu().view(bits) == want.view(bits)
        zero = (gcache.cpu().float() == 0) & (want.float() == 0)
        assert bool((same | zero).all())
        if f8:
            assert torch.equal(gscale.cpu().view(torch.uint8), want_scale)


@pytest.mark.parametrize("f8", [False, True])
def test_append_skips_what_has_no_place(attn, f8):
    """Bad page ids, negative and far positions, lengths past the table: nothing is written, nothing faults."""
    g = gen(3)
    hkv, d, page, pages, T = 2, 64, 16, 5, 8
    table = torch.tensor([[0, -1], [5, 1], [2147483647, 2], [-2147483648, 3], [0, 4]], dtype=torch.int32)
    lens = [12, 12, 14, 16, 30]
    caches = [torch.zeros((pages, hkv, page, d), dtype=torch.float8_e4m3fn if f8 else torch.bfloat16).cuda() for _ in "kv"]
    scales = [torch.zeros((pages, hkv, page), dtype=torch.uint8).view(torch.float8_e8m0fnu).cuda() if f8 else None for _ in "kv"]
    k, v = bf16(g, 5, hkv, T, d), bf16(g, 5, hkv, T, d)
    attn.cache_append(k.cuda(), v.cuda(), *caches, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                      k_scale=scales[0], v_scale=scales[1])
    for far in (-5, -2147483648, 2147483647, 2147483640):
        attn.cache_append(k.cuda(), v.cuda(), *caches, table.cuda(),
                          torch.tensor([far] * 5, dtype=torch.int32).cuda(), new_lens=torch.tensor([5] * 5, dtype=torch.int32).cuda(),
                          k_scale=scales[0], v_scale=scales[1])
    settled(attn)
    wrote = caches[0].cpu().float().abs().sum(-1).ne(0).any(1)   # [pages, page]
    want = torch.zeros(pages, page, dtype=torch.bool)
    for b in range(5):
        for t in range(T):
            at = page_row(table[b].tolist(), page, pages, lens[b] + t)
            if at:
                want[at] = True
    assert torch.equal(wrote, want)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("lens,hkv,d,page,N", [
    ([0], 1, 32, 16, 1), ([1, 16, 17], 2, 64, 16, 33), ([100, 0, 47], 3, 96, 48, 101), ([130, 1], 2, 128, 64, 129),
    ([300], 1, 128, 256, 256),
])
def test_read_back(attn, f8, lens, hkv, d, page, N):
    c = Cache(11, lens, hkv, d, page, f8)
    c.table[0, -1] = -7   # a page that is none, behind the first sequence
    lens_in = [n if n else -3 for n in lens]
    k, v, table, _, scales = c.on_gpu()
    out = attn.cache_read(k, v, table, torch.tensor(lens_in, dtype=torch.int32).cuda(), N, **scales)
    settled(attn)
    for b, n in enumerate(lens):
        n = min(n, N)
        for got, want in zip(out, c.rows(c.table[b], n)):
            assert np.array_equal(f64(got[b, :, :n]), want)
            assert not got[b, :, n:].any()


def test_read_past_the_table_and_bad_pages_is_zero(attn):
    c = Cache(12, [60, 60], 2, 64, 16, False, spare=0)
    c.table[0, 1], c.table[1, 2] = -1, 2147483647
    k, v, table, _, _ = c.on_gpu()
    out = attn.cache_read(k, v, table, torch.tensor([2147483647, 60], dtype=torch.int32).cuda(), 200)
    settled(attn)
    assert not out[0][0, :, 16:32].any() and not out[0][0, :, 64:].any() and not out[1][1, :, 32:48].any()
    assert torch.equal(out[0][1, :, :32].cpu(), torch.cat([c.k[int(i)] for i in c.table[1, :2]], 1))


def test_rows_that_are_not_finite_read_as_nan(attn):
    k = torch.ones((1, 1, 3, 32), dtype=torch.bfloat16)
    k[0, 0, 1, 5] = math.inf
    cache = [torch.zeros((1, 1, 16, 32), dtype=torch.float8_e4m3fn).cuda() for _ in "kv"]
    scale = [torch.zeros((1, 1, 16), dtype=torch.uint8).view(torch.float8_e8m0fnu).cuda() for _ in "kv"]
    table, lens = torch.zeros((1, 1), dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    attn.cache_append(k.cuda(), k.cuda(), *cache, table, lens, k_scale=scale[0], v_scale=scale[1])
    out, _ = attn.cache_read(*cache, table, lens + 3, 3, k_scale=scale[0], v_scale=scale[1])
    o, lse = attn.forward_decode(torch.ones((1, 1, 1, 32), dtype=torch.bfloat16).cuda(), *cache, table, lens + 3,
                                 k_scale=scale[0], v_scale=scale[1])
    settled(attn)
    assert out[0, 0, 1].isnan().all() and torch.equal(out[0, 0, ::2].cpu(), k[0, 0, ::2])
    assert o.isnan().all() and lse.isnan().all()


# ---------------------------------------------------------------- forward_decode, forward_shared_prefix

def run_decode(attn, c, q, scale=None, **kw):
    k, v, table, lens, scales = c.on_gpu()
    if c.prefix_len:
        o, lse = attn.forward_shared_prefix(q.cuda(), k, v, c.prefix_table.cuda(), c.prefix_len, table, lens,
                                            scale=scale, **scales, **kw)
    else:
        o, lse = attn.forward_decode(q.cuda(), k, v, table, lens, scale=scale, **scales, **kw)
    settled(attn)
    return o, lse


def check_decode(attn, c, hq, T, scale=None, seed=5, which=None):
    q = bf16(gen(seed), len(c.lens), hq, T, c.d)
    o, lse = run_decode(attn, c, q, scale)
    s = 1 / math.sqrt(c.d) if scale is None else scale
    for b in range(len(c.lens)) if which is None else which:
        check(f64(o[b]), f64(lse[b]), decode_want(c, f64(q[b]), b, s), c.d, s, c.lens[b] + c.prefix_len)
    return o, lse


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("lens,hq,hkv,T,page", [
    ([1], 1, 1, 1, 16),
    ([0, 1, 15, 16, 17, 64, 65, 130], 4, 2, 1, 16),
    ([200, 3, 0, 129], 6, 2, 3, 48),
    ([700, 64, 5], 8, 1, 5, 64),             # 40 rows: four row tiles
    ([257, 0, 90], 12, 1, 7, 32),            # 84 rows: two row blocks
    ([1500], 2, 2, 1, 256),
])
def test_decode(attn, f8, d, lens, hq, hkv, T, page):
    check_decode(attn, Cache(21, lens, hkv, d, page, f8), hq, T)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_decode_scales(attn, f8, scale):
    check_decode(attn, Cache(22, [300, 2], 2, 64, 16, f8), 4, 2, scale)


@pytest.mark.parametrize("f8", [False, True])
def test_decode_long_sequences_are_split_and_joined(attn, f8):
    c = Cache(23, [9000, 1, 4000], 1, 64, 64, f8)
    check_decode(attn, c, 4, 1)


def test_decode_more_sequences_than_threads(attn):
    r = np.random.RandomState(0)
    lens = [int(n) for n in r.randint(0, 90, 300)]
    check_decode(attn, Cache(24, lens, 2, 32, 16, True), 4, 1, which=range(0, 300, 7))


@pytest.mark.parametrize("f8", [False, True])
def test_decode_bad_pages_read_as_zeros(attn, f8):
    c = Cache(25, [100, 70], 2, 64, 16, f8)
    c.table[0, 2], c.table[1, 0], c.table[1, 4] = -1, 2147483647, -2147483648
    check_decode(attn, c, 4, 1)


def test_decode_lengths_outside_the_table(attn):
    c = Cache(26, [64, 64], 1, 64, 16, False, spare=0)
    q = bf16(gen(1), 2, 2, 1, 64)
    k, v, table, _, _ = c.on_gpu()
    o, lse = attn.forward_decode(q.cuda(), k, v, table, torch.tensor([2147483647, -2147483648], dtype=torch.int32).cuda())
    settled(attn)
    check(f64(o[0]), f64(lse[0]), decode_want(c, f64(q[0]), 0, 1 / 8), 64, 1 / 8, 64)
    assert not o[1].any() and bool(torch.isneginf(lse[1]).all())


def test_decode_large_scores_move_the_maximum(attn):
    """Keys that grow along the sequence: the running maximum moves at almost every step, far past the lazy limit."""
    c = Cache(27, [400], 1, 64, 16, False)
    ramp = torch.linspace(0.1, 30, 400)
    for p in range(400):
        i, row = page_row(c.table[0].tolist(), 16, c.k.shape[0], p)
        c.k[i, 0, row] = (c.k[i, 0, row].float() * ramp[p]).to(torch.bfloat16)
    check_decode(attn, c, 4, 2)


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("lo,hi", [(127, 127), (100, 150), (20, 230), (60, 71), (60, 72)])
def test_decode_value_scales_far_apart(attn, d, lo, hi):
    """V exponents that do not fit one pass of the kernel's probabilities, and K exponents against them."""
    c = Cache(43, [333, 70, 1], 2, d, 16, True)
    r = np.random.RandomState(lo + hi)
    vs = c.vs.view(torch.uint8)
    new = torch.tensor(r.randint(lo, hi + 1, tuple(vs.shape)), dtype=torch.uint8)
    new[:, :, ::3] = lo
    new[:, :, 5] = hi
    vs[vs != 255] = new[vs != 255]
    check_decode(attn, c, 4, 3)


def test_decode_weights_spread_over_many_small_ones(attn):
    """One key far above the rest, whose weights sum to as much: small probabilities must not vanish."""
    for f8 in (False, True):
        c = Cache(44, [6000], 1, 64, 64, f8)
        if f8:
            c.ks.view(torch.uint8)[c.ks.view(torch.uint8) != 255] = 127
        q = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
        q[0, 0, 0, 0] = 1.0
        for p in range(6000):
            i, row = page_row(c.table[0].tolist(), 64, c.k.shape[0], p)
            c.k[i, 0, row, 0] = torch.tensor(9.0 if p == 777 else 0.0).to(c.k.dtype)
        o, lse = run_decode(attn, c, q, 1.0)
        check(f64(o[0]), f64(lse[0]), decode_want(c, f64(q[0]), 0, 1.0), 64, 1.0, 6000)


@pytest.mark.parametrize("power", [-120, -60, 60, 110])
def test_decode_queries_of_any_size(attn, power):
    """Query rows far from 1, each with elements far apart."""
    for f8 in (False, True):
        c = Cache(45, [200, 31], 2, 64, 16, f8)
        q = bf16(gen(4), 2, 4, 2, 64)
        q[..., ::2] *= 2.0 ** -9
        q = (q.double() * 2.0 ** power).to(torch.bfloat16)
        scale = 2.0 ** -power / 8
        k, v, table, lens, sc = c.on_gpu()
        o, lse = attn.forward_decode(q.cuda(), k, v, table, lens, scale=scale, **sc)
        settled(attn)
        for b in range(2):
            check(f64(o[b]), f64(lse[b]), decode_want(c, f64(q[b]), b, scale), 64, scale, c.lens[b])


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("what", ["k", "v", "both"])
@pytest.mark.parametrize("lens,hq,hkv,T,prefix", [
    ([5], 2, 2, 5, 0),                        # the first tokens see next to nothing
    ([300, 3, 77, 128, 1], 4, 2, 4, 0),       # 8 rows; some tokens see nothing
    ([300, 77], 12, 3, 4, 0),                 # 16
    ([140, 33, 64], 16, 2, 7, 0),             # 56
    ([9000, 600], 4, 2, 3, 0),                # split and joined
    ([40, 0, 3] * 30, 8, 2, 2, 260),          # behind a prefix
])
def test_decode_what_later_tokens_hold_stays_theirs(attn, lens, hq, hkv, T, prefix, what, f8, d):
    """The last tokens' keys and values are not finite (E4M3: marked): tokens before them are as if nothing stood there,
    those that see them are NaN or infinite where the sum is (a key in every column and in lse, a value in its own
    columns, a marked value in all)."""
    c = Cache(46, lens, hkv, d, 16, f8, prefix=prefix)
    for b, n in enumerate(lens):
        for p in range(max(0, n - T + 1), n):   # seen by some tokens, not by the first
            i, row = page_row(c.table[b].tolist(), 16, c.k.shape[0], p)
            for t, sc, name in ((c.k, c.ks, "k"), (c.v, c.vs, "v")):
                if what not in (name, "both") or (n - 1 - p) % 3 == 2:
                    continue
                if f8:
                    t[i, 0, row] = 0
                    sc.view(torch.uint8)[i, 0, row] = 255
                else:
                    t[i, 0, row, (p * 5) % d] = (math.nan, math.inf, -math.inf)[p % 3]
    q = bf16(gen(7), len(lens), hq, T, d)
    o, lse = run_decode(attn, c, q)
    s = d ** -0.5
    for b in range(len(lens)) if len(lens) <= 6 else (0, 1, 2, 45, 89):
        with np.errstate(invalid="ignore"):
            want = decode_want(c, f64(q[b]), b, s)
        got, got_l = f64(o[b]), f64(lse[b])
        # a score of minus infinity leaves the row as it would be without that key: the oracle's |q k| is no bound there
        fine = np.isfinite(want[0]).all(-1) & ~np.isnan(want[1]) & np.isfinite(want[3])
        for h in range(hq):
            rows = np.nonzero(fine[h])[0]
            check(got[h : h + 1, rows], got_l[h : h + 1, rows], tuple(w[h : h + 1, rows] for w in want), d, s, lens[b] + prefix)
        nan = np.isnan(want[1])
        assert np.isnan(got_l[nan]).all() and np.isnan(got[nan]).all() and not np.isnan(got_l[~nan]).any()
        ok = np.isfinite(want[0]) & ~nan[..., None]
        assert np.isfinite(got[ok]).all()
        assert not np.isfinite(got[~np.isfinite(want[0])]).any()


def test_decode_is_deterministic(attn):
    c = Cache(28, [2000, 77, 0, 513], 2, 128, 64, True)
    q = bf16(gen(9), 4, 8, 1, 128)
    a, b = run_decode(attn, c, q), run_decode(attn, c, q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("lens,prefix,hq,hkv,T,page", [
    ([0, 1, 40], 1, 2, 1, 1, 16),
    ([3, 0], 100, 4, 2, 2, 16),              # 8 rows a KV head see the prefix
    ([70, 1, 200, 0, 9], 333, 8, 1, 1, 64),  # 40
    ([5] * 30, 500, 6, 2, 1, 48),            # 90
    ([20, 0, 3] * 14, 260, 16, 2, 1, 32),    # 336: several 128-row tiles
    ([9, 4], 200, 12, 1, 11, 32),            # 132 rows of one sequence
    ([9, 4, 7], 1300, 7, 1, 9, 256),         # 63 a sequence: tiles of two sequences, two rows short
])
def test_shared_prefix(attn, f8, d, lens, prefix, hq, hkv, T, page):
    c = Cache(31, lens, hkv, d, page, f8, prefix=prefix)
    n = len(lens)
    check_decode(attn, c, hq, T, which=None if n <= 5 else [0, 1, 2, n // 2, n - 1])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d,hq,T", [(32, 8, 1), (64, 8, 1), (96, 8, 1), (128, 8, 1), (64, 8, 2), (128, 4, 3), (128, 20, 1)])
def test_shared_prefix_as_a_server_has_it(attn, d, hq, T, f8):
    """Many short sequences behind a long prefix with a page that is none: several sequences in a 128-row tile (E4M3:
    converted ahead), the prefix's parts over many CTAs, joined by the warp that has the sequence's own keys (up to 16
    rows; 20: by the joining kernel)."""
    lens = [(37 * b) % 97 for b in range(128)]
    lens[5] = lens[64] = 0
    c = Cache(36, lens, 1, d, 32, f8, prefix=3001)
    c.prefix_table[40] = -1
    assert c.table.shape[1] * 32 == 128
    check_decode(attn, c, hq, T, which=[0, 1, 5, 17, 64, 126, 127])


def test_shared_prefix_of_nothing_is_decode(attn):
    c = Cache(32, [50, 0, 300], 2, 64, 16, False)
    q = bf16(gen(2), 3, 4, 2, 64)
    k, v, table, lens, _ = c.on_gpu()
    o, lse = attn.forward_shared_prefix(q.cuda(), k, v, torch.empty(0, dtype=torch.int32).cuda(), 0, table, lens)
    settled(attn)
    for b in range(3):
        check(f64(o[b]), f64(lse[b]), decode_want(c, f64(q[b]), b, 1 / 8), 64, 1 / 8, 300)


@pytest.mark.parametrize("B", [3, 60])
@pytest.mark.parametrize("page", [16, 48, 32])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
def test_shared_prefix_without_pages_of_its_own(attn, d, f8, page, B):
    """A table of no pages (its pointer is null): the prefix's pages are pages all the same, of fewer rows than a step
    of the kernel or not a multiple of it."""
    c = Cache(34, [0] * B, 2, d, page, f8, prefix=100)
    c.table = c.table[:, :0].contiguous()
    check_decode(attn, c, 4, 2, which=[0, B - 1])


@pytest.mark.parametrize("B", [3, 60])
@pytest.mark.parametrize("f8", [False, True])
def test_shared_prefix_bad_page_reads_as_zeros(attn, f8, B):
    c = Cache(33, [10] * B, 1, 64, 16, f8, prefix=100)
    c.prefix_table[1], c.prefix_table[6] = -1, 1 << 30
    check_decode(attn, c, 4, 1, which=[0, B - 1])


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("B", [4, 25, 150])   # 16 rows a KV head: the decode kernel; 100: one tile; 600: E4M3 converted ahead
def test_shared_prefix_keys_that_are_not_finite(attn, B, f8):
    """A prefix key that is NaN (E4M3: marked), at each position mod 16: every row of its head is NaN in o and lse, the
    other head's rows are bit for bit as without it."""
    c = Cache(35, [(7 * b) % 40 for b in range(B)], 2, 64, 16, f8, prefix=300)
    q = bf16(gen(6), B, 8, 1, 64)
    clean = run_decode(attn, c, q)
    for p in range(130, 146):
        i, row = page_row(c.prefix_table.tolist(), 16, c.k.shape[0], p)
        keep = c.k[i, 0, row].clone(), None if c.ks is None else c.ks.view(torch.uint8)[i, 0, row].clone()
        if f8:
            c.k[i, 0, row] = 0
            c.ks.view(torch.uint8)[i, 0, row] = 255
        else:
            c.k[i, 0, row, 5] = math.nan
        o, lse = run_decode(attn, c, q)
        assert o[:, :4].isnan().all() and lse[:, :4].isnan().all(), p
        assert torch.equal(o[:, 4:], clean[0][:, 4:]) and torch.equal(lse[:, 4:], clean[1][:, 4:]), p
        c.k[i, 0, row] = keep[0]
        if f8:
            c.ks.view(torch.uint8)[i, 0, row] = keep[1]


# ---------------------------------------------------------------- together, as a server uses them

@pytest.mark.parametrize("f8", [False, True])
def test_a_dialogue(attn, f8):
    """Prompts computed by forward(), appended, then tokens decoded one by one and appended; the whole cache read back
    and the last step repeated by forward() on it."""
    g = gen(77)
    B, hq, hkv, d, page, steps = 2, 4, 2, 64, 16, 5
    n0 = [37, 20]
    dt = torch.float8_e4m3fn if f8 else torch.bfloat16
    cache = [torch.zeros((12, hkv, page, d), dtype=dt).cuda() for _ in "kv"]
    sc = {}
    if f8:
        sc = {n: torch.zeros((12, hkv, page), dtype=torch.uint8).view(torch.float8_e8m0fnu).cuda() for n in ("k_scale", "v_scale")}
    table = torch.randperm(12, generator=g).to(torch.int32).view(2, 6).contiguous().cuda()
    lens = torch.zeros(B, dtype=torch.int32).cuda()
    new = torch.tensor(n0, dtype=torch.int32).cuda()
    attn.cache_append(bf16(g, B, hkv, 40, d).cuda(), bf16(g, B, hkv, 40, d).cuda(), *cache, table, lens, new_lens=new, **sc)
    lens += new
    for _ in range(steps):
        q = bf16(g, B, hq, 1, d).cuda()
        attn.cache_append(bf16(g, B, hkv, 1, d).cuda(), bf16(g, B, hkv, 1, d).cuda(), *cache, table, lens, **sc)
        lens += 1
        o, lse = attn.forward_decode(q, *cache, table, lens, **sc)
    settled(attn)
    for b in range(B):
        n = n0[b] + steps
        k, v = attn.cache_read(*cache, table, lens, n, **sc)
        whole = q[b : b + 1].expand(1, hq, n, d).contiguous()
        o2, lse2 = attn.forward(whole, k[b : b + 1].contiguous(), v[b : b + 1].contiguous(), causal=True)
        settled(attn)
        # two kernels, each within its own tolerance of the same value: P and O rounded to bf16 in each
        assert (o[b, :, 0].float() - o2[0, :, -1].float()).abs().max() <= 4 * 2.0 ** -8 * v[b].float().abs().max()
        assert (lse[b, :, 0] - lse2[0, :, -1]).abs().max() <= 2e-3


def test_captured_calls_see_new_lengths_and_tables(attn):
    c = Cache(41, [100, 50, 3], 2, 64, 16, False)
    q = bf16(gen(3), 3, 4, 1, 64).cuda()
    k, v, table, lens, _ = c.on_gpu()
    o, lse = attn.forward_decode(q, k, v, table, lens)   # warm-up, and shapes
    out = []
    graphs = []
    for _ in range(2):   # two graphs, replayed at once on two streams below
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out.append(attn.forward_decode(q, k, v, table, lens))
        graphs.append(gr)
    for new in ([100, 50, 3], [64, 0, 1], [99, 17, 2]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        settled(attn)
        for o, lse in out:
            for b, n in enumerate(new):
                c.lens[b] = n
                check(f64(o[b]), f64(lse[b]), decode_want(c, f64(q[b]), b, 1 / 8), 64, 1 / 8, 100)


def test_calls_on_two_streams_at_once(attn):
    c = Cache(42, [3000, 10], 2, 128, 64, True)
    q = [bf16(gen(i), 2, 8, 1, 128).cuda() for i in range(2)]
    k, v, table, lens, sc = c.on_gpu()
    want = [attn.forward_decode(x, k, v, table, lens, **sc) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    got = []
    for _ in range(10):
        got = [attn.forward_decode(x, k, v, table, lens, stream=s, **sc) for x, s in zip(q, streams)]
    settled(attn)
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
