"""Seeded caches and batches for the cache and cross-attention tests, and the tolerances they are held to."""
import numpy as np
import torch

from oracle import attend, gather


def gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def bf16(g, *shape):
    return torch.randn(shape, generator=g, dtype=torch.float32).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy() if t.dtype != torch.float8_e4m3fn else t.detach().cpu().float().double().numpy()


class Cache:
    """A paged cache on the CPU with random rows, pages in shuffled order, every row behind a sequence's last holding
    NaN (bf16) or the NaN exponent (E4M3): nothing may read them."""

    def __init__(self, seed, lens, hkv, d, page, f8, spare=1, prefix=0):
        g = gen(seed)
        self.lens, self.hkv, self.d, self.page, self.f8 = list(lens), hkv, d, page, f8
        per = max(1, -(-max(max(lens), 1) // page)) + spare
        pre = -(-prefix // page)
        total = len(lens) * per + pre + 1
        order = torch.randperm(total, generator=g).to(torch.int32)
        self.table = order[: len(lens) * per].view(len(lens), per).contiguous()
        self.prefix_table, self.prefix_len = order[len(lens) * per : len(lens) * per + pre].contiguous(), prefix
        self.k, self.v = bf16(g, total, hkv, page, d), bf16(g, total, hkv, page, d)
        self.ks = self.vs = None
        live = torch.zeros((total, page), dtype=torch.bool)
        rows = [(self.table[b], n) for b, n in enumerate(lens)] + [(self.prefix_table, prefix)]
        for table, n in rows:
            for p in range(max(n, 0)):
                live[int(table[p // page]), p % page] = True
        if f8:
            self.k, self.v = self.k.to(torch.float8_e4m3fn), self.v.to(torch.float8_e4m3fn)
            shape = (total, hkv, page)
            self.ks = torch.randint(125, 130, shape, generator=g).to(torch.uint8)
            self.vs = torch.randint(120, 131, shape, generator=g).to(torch.uint8)
            dead = ~live[:, None].expand(shape)
            self.ks[dead] = 255
            self.vs[dead] = 255
            self.ks, self.vs = self.ks.view(torch.float8_e8m0fnu), self.vs.view(torch.float8_e8m0fnu)
        else:
            dead = ~live[:, None, :, None].expand(self.k.shape)
            self.k[dead] = float("nan")
            self.v[dead] = float("nan")

    def on_gpu(self):
        """Keyword arguments of the cache's tensors, positional table and lens, on the GPU."""
        c = lambda t: None if t is None else t.cuda()
        lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        return c(self.k), c(self.v), self.table.cuda(), lens, {"k_scale": c(self.ks), "v_scale": c(self.vs)}

    def rows(self, table, n):
        """fp64 k, v [Hkv, n, D] of the first n positions behind a table row."""
        byte = lambda s: None if s is None else s.view(torch.uint8).numpy()
        return (gather(f64(self.k), byte(self.ks), table.numpy(), n), gather(f64(self.v), byte(self.vs), table.numpy(), n))


def check(o, lse, want, d, scale, n):
    """o [Hq, T, D], lse [Hq, T] of the kernel (fp64 arrays) against oracle.attend's answer, element by element.

    The kernels round the probabilities to bf16 (at most half a step, 2^-8 of each) and then O (2^-8 again), and
    otherwise work in fp32 (2^-24 a step):
      scores   the sum of D products: at most (D + 4) steps of sum |q k| * scale, which shifts every exponent; an
               exponential turns that into a relative error of p, once in the numerator and once in the sum;
      exp      2 * 2.4e-7, the largest relative error of the hardware's 2^x (2^-22) and of the polynomial that
               stands in for part of it, numerator and sum;
      sums     n + 64 additions at most, numerator and sum.
    """
    o_ref, lse_ref, a, top = want
    half = 2.0 ** -8
    rel = 2 * ((d + 4) * 2.0 ** -24 * abs(scale) * top + 2.4e-7 + (n + 64) * 2.0 ** -24)
    tol = (half * (1 + half) + rel[..., None]) * a + half * (np.abs(o_ref) + half * a) + 1e-30
    live = np.isfinite(lse_ref)
    assert np.array_equal(np.isneginf(lse), ~live), "rows without keys"
    assert not o[~live].any(), "rows without keys"
    bad = np.abs(o - o_ref) > tol
    assert np.all(np.isfinite(o)) and not bad.any(), (
        f"{bad.sum()} of {bad.size} outside: worst {np.nanmax(np.abs(o - o_ref) / tol):.3f} of the tolerance")
    dl = np.abs(lse[live] - lse_ref[live])
    tol_l = rel[live] + 2.0 ** -21 * (1 + np.abs(lse_ref[live]))
    assert np.all(dl <= tol_l), f"lse: worst {np.max(dl / tol_l):.3f} of the tolerance"


def decode_want(c, q, b, scale, causal=True):
    """oracle.attend for sequence b of cache c behind its shared prefix, with q [Hq, T, D]."""
    n, T = max(c.lens[b], 0), q.shape[1]
    k, v = c.rows(c.table[b], n)
    lims = [n - T + 1 + t for t in range(T)]
    if c.prefix_len:
        pk, pv = c.rows(c.prefix_table, c.prefix_len)
        k, v = np.concatenate([pk, k], 1), np.concatenate([pv, v], 1)
        lims = [c.prefix_len + max(0, x) for x in lims]
    return attend(q, k, v, lims, scale)
