"""Cross attention, forward and backward, against the fp64 oracle (needs a B200)."""
import math

import numpy as np
import pytest
import torch

from kv_cases import bf16, check, f64, gen
from oracle import attend, cross_backward

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


def case(seed, B, hq, hkv, nq, nk, d, lens, poison=True):
    """q, k, v, do on the CPU; the padding holds NaN and infinities."""
    g = gen(seed)
    q, k, v, do = bf16(g, B, hq, nq, d), bf16(g, B, hkv, nk, d), bf16(g, B, hkv, nk, d), bf16(g, B, hq, nq, d)
    for b, n in enumerate(lens) if poison and lens else ():
        n = max(0, min(n, nk))
        k[b, :, n:], v[b, :, n:] = float("nan"), float("inf")
        k[b, :, n + 1 :: 3], v[b, :, n + 1 :: 2] = float("-inf"), float("nan")
    return q, k, v, do


def counts(lens, B, nk):
    return [nk] * B if lens is None else [max(0, min(n, nk)) for n in lens]


def gpu_lens(lens):
    return None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()


SIZES = [
    # B, Hq, Hkv, Nq, Nk, lens
    (1, 1, 1, 1, 1, None),
    (2, 2, 2, 1, 50, [50, 0]),
    (3, 4, 2, 2, 130, [128, 1, 129]),
    (2, 4, 4, 16, 300, None),
    (2, 2, 1, 33, 64, [64, 63]),
    (3, 2, 2, 130, 257, [257, 100, 0]),
    (2, 6, 2, 77, 333, [332, 17]),
    (1, 8, 1, 40, 200, [200]),
    (4, 2, 2, 300, 7, [7, 3, 9, -5]),
    (2, 1, 1, 513, 640, [640, 385]),
    (2, 2, 2, 5, 0, None),
]


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("B,hq,hkv,nq,nk,lens", SIZES)
def test_forward(attn, d, B, hq, hkv, nq, nk, lens):
    q, k, v, _ = case(3, B, hq, hkv, nq, nk, d, lens)
    o, lse = attn.forward_cross(q.cuda(), k.cuda(), v.cuda(), k_lens=gpu_lens(lens))
    settled(attn)
    s = 1 / math.sqrt(d)
    for b, n in enumerate(counts(lens, B, nk)):
        want = attend(f64(q[b]), f64(k[b, :, :n]), f64(v[b, :, :n]), [n] * nq, s)
        check(f64(o[b]), f64(lse[b]), want, d, s, n)


@pytest.mark.parametrize("lens", [[0] * 9, [0, 0, 0, 0, 0, 0, 0, 0, 130], [130] + [0] * 8, [0, 0, 0, 0, 200, 0, 0, 0, 1],
                                  [1, 1, 1, 1, 1, 1, 1, 1, 1]])
def test_forward_runs_of_batch_rows_without_keys(attn, lens):
    """More tiles without a key in a row than the kernel's ring of units holds, before, behind and between others."""
    q, k, v, _ = case(7, 9, 6, 3, 150, 260, 32, lens)
    o, lse = attn.forward_cross(q.cuda(), k.cuda(), v.cuda(), k_lens=gpu_lens(lens))
    settled(attn)
    for b, n in enumerate(lens):
        check(f64(o[b]), f64(lse[b]), attend(f64(q[b]), f64(k[b, :, :n]), f64(v[b, :, :n]), [n] * 150, 32 ** -0.5), 32,
              32 ** -0.5, n)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.5])
@pytest.mark.parametrize("nq", [3, 200])
def test_forward_scales(attn, scale, nq):
    q, k, v, _ = case(4, 2, 2, 1, nq, 190, 64, [190, 65])
    o, lse = attn.forward_cross(q.cuda(), k.cuda(), v.cuda(), k_lens=gpu_lens([190, 65]), scale=scale)
    settled(attn)
    for b, n in enumerate([190, 65]):
        check(f64(o[b]), f64(lse[b]), attend(f64(q[b]), f64(k[b, :, :n]), f64(v[b, :, :n]), [n] * nq, scale), 64, scale, n)


def test_forward_few_rows_many_keys_is_split_and_joined(attn):
    q, k, v, _ = case(5, 2, 2, 1, 150, 9001, 64, [9001, 4000])
    o, lse = attn.forward_cross(q.cuda(), k.cuda(), v.cuda(), k_lens=gpu_lens([9001, 4000]))
    settled(attn)
    for b, n in enumerate([9001, 4000]):
        check(f64(o[b]), f64(lse[b]), attend(f64(q[b]), f64(k[b, :, :n]), f64(v[b, :, :n]), [n] * 150, 1 / 8), 64, 1 / 8, n)


def test_forward_large_scores_move_the_maximum(attn):
    q, k, v, _ = case(6, 1, 2, 2, 140, 700, 64, None)
    k = (k.float() * torch.linspace(0.1, 25, 700)[:, None]).to(torch.bfloat16)
    o, lse = attn.forward_cross(q.cuda(), k.cuda(), v.cuda())
    settled(attn)
    check(f64(o[0]), f64(lse[0]), attend(f64(q[0]), f64(k[0]), f64(v[0]), [700] * 140, 1 / 8), 64, 1 / 8, 700)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nk", [(1, 150), (200, 150), (200, 16), (130, 1200), (2000, 700)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_forward_keys_that_are_not_finite(attn, bad, nq, nk, d):
    """A key that is NaN or infinite, at each position mod 16 (one a batch row): NaN wherever the score is NaN or plus
    infinity, the key's weight 0 where it is minus infinity; the other batch rows bit for bit as without it."""
    B, s = 18, d ** -0.5
    q, k, v, _ = case(8, B, 2, 1, nq, nk, d, None)
    clean = attn.forward_cross(q.cuda(), k.cuda(), v.cuda())
    at = [nk // 2 // 16 * 16 + b for b in range(16)]
    for b, p in enumerate(at):
        k[b, 0, p, 3] = bad
    o, lse = attn.forward_cross(q.cuda(), k.cuda(), v.cuda())
    settled(attn)
    for got, want in zip((o, lse), clean):
        assert torch.equal(got[16:], want[16:])
    for b, p in enumerate(at):
        nan = torch.isnan(q[b, ..., 3].float() * bad) | (q[b, ..., 3].float() * bad > 0)   # [Hq, Nq]
        assert torch.equal(lse[b].isnan().cpu(), nan) and torch.equal(o[b].isnan().all(-1).cpu(), nan)
        rows = (~nan).any(0).nonzero().flatten()[:40]
        if len(rows):
            keep = [j for j in range(nk) if j != p]
            want = attend(f64(q[b][:, rows]), f64(k[b, :, keep]), f64(v[b, :, keep]), [nk - 1] * len(rows), s)
            live = f64(~nan[:, rows].unsqueeze(-1)) > 0
            w = (*(np.where(live if x.ndim == 3 else live[..., 0], x, -np.inf if i == 1 else 0.0) for i, x in enumerate(want)),)
            go, gl = f64(o[b][:, rows]), f64(lse[b][:, rows])
            check(np.where(live, go, 0.0), np.where(live[..., 0], gl, -np.inf), w, d, s, nk)


@pytest.mark.parametrize("nq", [1, 200])
@pytest.mark.parametrize("nk", [1, 64, 70, 300, 5000])
def test_forward_no_key_is_finite(attn, nq, nk):
    q, k, v, _ = case(9, 2, 2, 1, nq, nk, 64, None)
    k[0] = math.nan
    o, lse = attn.forward_cross(q.cuda(), k.cuda(), v.cuda())
    settled(attn)
    assert o[0].isnan().all() and lse[0].isnan().all()
    check(f64(o[1]), f64(lse[1]), attend(f64(q[1]), f64(k[1]), f64(v[1]), [nk] * nq, 1 / 8), 64, 1 / 8, nk)


def backward_bounds(q, k, v, do, n, scale, o, lse):
    """Element-wise tolerances of dq, dk, dv for one batch row, from the roundings of the kernel: P and dS to bf16 (half
    a step, 2^-8, of each), the gradients to bf16, and the given o (bf16) in delta; scores, dP and exponentials in fp32
    (their relative error of P is `rel`, as in kv_cases.check, with the fp32 rounding of the given lse)."""
    Hq, group, D = q.shape[0], q.shape[0] // k.shape[0], q.shape[2]
    half, u = 2.0 ** -8, 2.0 ** -24
    tq, tk, tv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for h in range(Hq) if n else ():
        g = h // group
        kk, vv = k[g, :n], v[g, :n]
        p = np.exp(scale * (q[h] @ kk.T) - lse[h][:, None])
        rel = (D + 4) * u * abs(scale) * (np.abs(q[h]) @ np.abs(kk).T) + 7.5e-5 + 4 * u * (1 + np.abs(lse[h]))[:, None]
        dp, adp = do[h] @ vv.T, np.abs(do[h]) @ np.abs(vv).T
        delta, adelta = (do[h] * o[h]).sum(1), (np.abs(do[h]) * np.abs(o[h])).sum(1)
        ds = p * (dp - delta[:, None])
        t_diff = (D + 4) * u * (adp + adelta[:, None]) + half * adelta[:, None]
        t_ds = p * (1 + rel) * t_diff + (rel + half * (1 + rel)) * np.abs(ds) + half * p * t_diff
        t_p = (rel + half * (1 + rel)) * p
        rows = q.shape[1] * group + 64
        for t, w, x, acc, rows_n in ((t_ds, ds, kk, tq[h], n + 64),):
            acc += abs(scale) * (t @ np.abs(x) + rows_n * u * (np.abs(w) @ np.abs(x)))
        tk[g, :n] += abs(scale) * (t_ds.T @ np.abs(q[h]) + rows * u * (np.abs(ds).T @ np.abs(q[h])))
        tv[g, :n] += t_p.T @ np.abs(do[h]) + rows * u * (p.T @ np.abs(do[h]))
    return tq, tk, tv


BWD_SIZES = [s for s in SIZES if s[4] > 0] + [(2, 4, 2, 1, 200, [200, 5]), (1, 4, 1, 260, 1100, [1025])]


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("B,hq,hkv,nq,nk,lens", BWD_SIZES)
def test_backward(attn, d, B, hq, hkv, nq, nk, lens):
    q, k, v, do = case(13, B, hq, hkv, nq, nk, d, lens)
    s = 1 / math.sqrt(d)
    ns = counts(lens, B, nk)
    ref = [attend(f64(q[b]), f64(k[b, :, :n]), f64(v[b, :, :n]), [n] * nq, s) for b, n in enumerate(ns)]
    o = torch.tensor(np.stack([r[0] for r in ref])).to(torch.bfloat16)
    lse = torch.tensor(np.stack([r[1] for r in ref])).to(torch.float32)
    got = attn.backward_cross(q.cuda(), k.cuda(), v.cuda(), o.cuda(), lse.cuda(), do.cuda(), k_lens=gpu_lens(lens))
    settled(attn)
    for b, n in enumerate(ns):
        kb, vb = f64(k[b]).copy(), f64(v[b]).copy()
        kb[:, n:], vb[:, n:] = 0, 0
        want = cross_backward(f64(q[b]), kb, vb, f64(do[b]), n, s)
        tols = backward_bounds(f64(q[b]), kb, vb, f64(do[b]), n, s, f64(o[b]), ref[b][1])
        for name, x, w, t in zip(("dq", "dk", "dv"), got, want, tols):
            x = f64(x[b])
            tol = t + 2.0 ** -8 * (np.abs(w) + t) + 1e-30
            assert np.all(np.isfinite(x)), name
            worst = np.max(np.abs(x - w) / tol) if x.size else 0.0
            assert worst <= 1, f"{name} of row {b}: {worst:.3f} of the tolerance"
            if name != "dq":
                assert not x[:, n:].any(), f"{name} at the padding"
        if n == 0:
            assert not f64(got[0][b]).any()


@pytest.mark.parametrize("nq,nk", [(0, 5), (5, 0)])
def test_backward_with_one_side_empty_is_zero(attn, nq, nk):
    q, k, v, do = case(14, 2, 2, 1, nq, nk, 64, None)
    lse = torch.full((2, 2, nq), -math.inf)
    grads = [torch.ones_like(x).cuda() for x in (q, k, v)]
    attn.backward_cross(q.cuda(), k.cuda(), v.cuda(), torch.zeros_like(q).cuda(), lse.cuda(), do.cuda(), dq=grads[0],
                        dk=grads[1], dv=grads[2])
    settled(attn)
    assert not any(bool(g.any()) for g in grads)


def test_step_against_differences(attn):
    """Forward and backward together: the gradient's directional derivative against differences of the oracle's loss
    at the same bf16 inputs."""
    B, hq, hkv, nq, nk, d, lens = 2, 4, 2, 140, 150, 64, [150, 70]
    q, k, v, do = case(15, B, hq, hkv, nq, nk, d, lens, poison=False)
    gl = gpu_lens(lens)
    o, lse = attn.forward_cross(q.cuda(), k.cuda(), v.cuda(), k_lens=gl)
    grads = attn.backward_cross(q.cuda(), k.cuda(), v.cuda(), o, lse, do.cuda(), k_lens=gl)
    settled(attn)
    r = np.random.RandomState(0)
    x = [f64(t) for t in (q, k, v)]
    dirs = [r.randn(*t.shape) for t in x]

    def loss(y):
        return sum(float((attend(y[0][b], y[1][b], y[2][b], [n] * nq, 1 / 8)[0] * f64(do[b])).sum()) for b, n in enumerate(lens))

    for i in range(3):
        h = 1e-5
        plus, minus = [t.copy() for t in x], [t.copy() for t in x]
        plus[i] += h * dirs[i]
        minus[i] -= h * dirs[i]
        slope = (loss(plus) - loss(minus)) / (2 * h)
        terms = f64(grads[i]) * dirs[i]
        # each element is off by a few half steps of roundings that do not add up in one direction: 2^-6 of their root sum of squares, sixfold
        assert abs(terms.sum() - slope) <= 6 * 2.0 ** -6 * math.sqrt((terms ** 2).sum()) + 1e-6


@pytest.mark.parametrize("d,nq,nk", [(32, 40, 30), (64, 300, 130), (96, 128, 500), (128, 700, 900)])
def test_backward_row_sums_are_this_calls(attn, d, nq, nk):
    """Calls in turn whose row sums differ in every row and lie in the same workspace, without a pause between them:
    the dQ pass, which starts before the dK/dV pass has ended, reads those of its own call."""
    q, k, v, do = (t.cuda() for t in case(18, 2, 4, 2, nq, nk, d, None))
    o, lse = attn.forward_cross(q, k, v)
    dos = [do, (-3 * do).contiguous(), (do * do).contiguous()]
    want = []
    for x in dos:
        want.append(attn.backward_cross(q, k, v, o, lse, x))
        torch.cuda.synchronize()
    got = [attn.backward_cross(q, k, v, o, lse, dos[i % 3]) for i in range(30)]
    settled(attn)
    for i, grads in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(grads, want[i % 3])), i


def test_backward_captured_beside_an_eager_one(attn):
    B, hq, hkv, nq, nk, d, lens = 2, 2, 1, 100, 150, 64, [150, 33]
    q, k, v, do = (t.cuda() for t in case(16, B, hq, hkv, nq, nk, d, lens))
    gl = gpu_lens(lens)
    o, lse = attn.forward_cross(q, k, v, k_lens=gl)
    want = attn.backward_cross(q, k, v, o, lse, do, k_lens=gl)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        o2, lse2 = attn.forward_cross(q, k, v, k_lens=gl)
        got = attn.backward_cross(q, k, v, o2, lse2, do, k_lens=gl)
    for _ in range(2):
        for g in got:
            g.fill_(7)
        gr.replay()
        settled(attn)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(o, o2)


def test_forward_is_deterministic_and_streams_do_not_meet(attn):
    q, k, v, _ = (t.cuda() for t in case(17, 2, 4, 2, 300, 1000, 128, [1000, 444]))
    gl = gpu_lens([1000, 444])
    want = attn.forward_cross(q, k, v, k_lens=gl)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        got = [attn.forward_cross(q, k, v, k_lens=gl, stream=s) for s in streams]
        settled(attn)
        assert all(torch.equal(a[0], want[0]) and torch.equal(a[1], want[1]) for a in got)
