"""The entry points of the key/value cache and of attention over keys of another length: what they refuse, and the
empty problems they accept, before any CUDA call (no GPU needed); and what needs a device to be refused (gpu)."""
import math

import pytest

import tiled_attention_forward_03_b200 as attn

OK, INVALID, UNSUPPORTED, MISALIGNED = (attn.ATTN_OK, attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED,
                                        attn.ATTN_ERR_MISALIGNED)
P = 0x10000  # a 256-byte aligned fake device address; never dereferenced by a rejected call

CACHE = dict(k_cache=P, v_cache=P, k_scale=None, v_scale=None, block_table=P, lens=P)
SIZES = dict(D=64, num_pages=8, page_size=16, max_pages=4)
APPEND = dict(k=P, v=P, **CACHE, new_lens=None, B=2, Hkv=2, T=3, **SIZES, stream=None)
READ = dict(**CACHE, k=P, v=P, B=2, Hkv=2, N=3, **SIZES, stream=None)
DECODE = dict(q=P, **CACHE, o=P, lse=P, B=2, Hq=4, Hkv=2, T=1, **SIZES, scale=0.125, workspace=P,
              workspace_bytes=1 << 40, stream=None)
PREFIX = dict(q=P, **{k: CACHE[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale")}, prefix_table=P, prefix_len=20,
              block_table=P, lens=P, o=P, lse=P, B=2, Hq=4, Hkv=2, T=1, **SIZES, scale=0.125, workspace=P,
              workspace_bytes=1 << 40, stream=None)
CROSS = dict(q=P, k=P, v=P, k_lens=None, o=P, lse=P, B=2, Hq=4, Hkv=2, Nq=5, Nk=7, D=64, scale=0.125, workspace=P,
             workspace_bytes=1 << 40, stream=None)
CROSS_BWD = dict(q=P, k=P, v=P, k_lens=None, o=P, lse=P, dout=P, dq=P, dk=P, dv=P, B=2, Hq=4, Hkv=2, Nq=5, Nk=7, D=64,
                 scale=0.125, workspace=P, workspace_bytes=1 << 40, stream=None)
CALLS = {"append": (attn.attn_cache_append, APPEND), "read": (attn.attn_cache_read, READ),
         "decode": (attn.attn_fwd_decode, DECODE), "prefix": (attn.attn_fwd_shared_prefix, PREFIX),
         "cross": (attn.attn_fwd_cross, CROSS), "cross_bwd": (attn.attn_bwd_cross, CROSS_BWD)}
CACHED = ("append", "read", "decode", "prefix")
HEADS = ("decode", "prefix", "cross", "cross_bwd")


def call(which, **kw):
    fn, args = CALLS[which]
    assert set(kw) <= set(args)
    return fn(*{**args, **kw}.values())


def each(names, *rows):
    return [(n, kw, want) for n in names for kw, want in rows]


@pytest.mark.parametrize("which,kw,want", [
    *each(CALLS, (dict(B=-1), INVALID), (dict(Hkv=0), INVALID), (dict(D=256), UNSUPPORTED), (dict(D=0), UNSUPPORTED),
          (dict(D=40), UNSUPPORTED), (dict(B=1 << 30, Hkv=4), UNSUPPORTED)),
    *each(CACHED, (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID), (dict(lens=None), INVALID),
          (dict(block_table=None), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID),
          (dict(page_size=-16), INVALID), (dict(max_pages=-1), INVALID), (dict(page_size=24), UNSUPPORTED),
          (dict(k_scale=P), INVALID), (dict(v_scale=P), INVALID), (dict(k_cache=P + 8), MISALIGNED),
          (dict(v_cache=P + 8), MISALIGNED), (dict(k_scale=P, v_scale=P + 8), MISALIGNED),
          (dict(k_scale=P + 8, v_scale=P), MISALIGNED), (dict(block_table=P + 2), MISALIGNED),
          (dict(lens=P + 2), MISALIGNED), (dict(num_pages=1 << 30, Hkv=4), UNSUPPORTED)),
    *each(("append", "read"), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=P + 8), MISALIGNED),
          (dict(v=P + 8), MISALIGNED)),
    *each(("append",), (dict(T=-1), INVALID), (dict(new_lens=P + 2), MISALIGNED),
          (dict(B=1 << 16, T=1 << 15), UNSUPPORTED)),
    *each(("read",), (dict(N=-1), INVALID), (dict(B=1 << 16, N=1 << 15), UNSUPPORTED)),
    *each(HEADS, (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(lse=None), INVALID), (dict(Hq=0), INVALID),
          (dict(Hq=3), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
          (dict(q=P + 8), MISALIGNED), (dict(o=P + 8), MISALIGNED), (dict(lse=P + 2), MISALIGNED),
          (dict(workspace=P + 16), MISALIGNED)),
    *each(("decode", "prefix"), (dict(T=-1), INVALID), (dict(B=1 << 20, T=1 << 12), UNSUPPORTED)),
    *each(("prefix",), (dict(prefix_len=-1), INVALID), (dict(prefix_table=None), INVALID),
          (dict(prefix_table=P + 2), MISALIGNED)),
    *each(("cross", "cross_bwd"), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(Nq=-1), INVALID),
          (dict(Nk=-1), INVALID), (dict(k=P + 8), MISALIGNED), (dict(v=P + 8), MISALIGNED),
          (dict(k_lens=P + 2), MISALIGNED), (dict(B=1 << 20, Nk=1 << 20), UNSUPPORTED),
          (dict(B=1 << 20, Nq=1 << 20), UNSUPPORTED)),
    *each(("cross_bwd",), *[(dict([(n, None)]), INVALID) for n in ("dout", "dq", "dk", "dv", "workspace")],
          *[(dict([(n, P + 8)]), MISALIGNED) for n in ("dout", "dq", "dk", "dv")],
          (dict(workspace_bytes=0), INVALID)),
])
def test_rejected_before_any_cuda_call(which, kw, want):
    assert call(which, **kw) == want


@pytest.mark.parametrize("which,kw", [
    *[(n, dict(B=0)) for n in CALLS], ("append", dict(T=0)), ("read", dict(N=0)), ("decode", dict(T=0)),
    ("prefix", dict(T=0)), ("cross", dict(Nq=0)), ("cross_bwd", dict(Nq=0, Nk=0)),
    ("append", dict(B=0, k=None, v=None, k_cache=None, v_cache=None, lens=None, block_table=None)),
    ("cross", dict(Nq=0, q=None, o=None, lse=None, workspace=None, workspace_bytes=0)),
])
def test_empty_problem_is_ok_without_launch(which, kw):
    assert call(which, **kw) == OK


def test_workspace_queries_refuse_what_the_calls_refuse():
    assert attn.attn_fwd_decode_workspace_bytes(2, 3, 2, 1, 64, 16, 4) == -1
    assert attn.attn_fwd_decode_workspace_bytes(2, 4, 2, 1, 64, 24, 4) == -1
    assert attn.attn_fwd_decode_workspace_bytes(2, 4, 2, 0, 64, 16, 4) == 0
    assert attn.attn_fwd_shared_prefix_workspace_bytes(2, 4, 2, 1, 64, 16, 4, -1, 0) == -1
    assert attn.attn_fwd_shared_prefix_workspace_bytes(0, 4, 2, 1, 64, 16, 4, 20, 0) == 0
    assert attn.attn_fwd_cross_workspace_bytes(2, 4, 2, 5, -1, 64) == -1
    assert attn.attn_fwd_cross_workspace_bytes(2, 4, 2, 0, 7, 64) == 0
    assert attn.attn_bwd_cross_workspace_bytes(2, 3, 2, 5) == -1
    assert attn.attn_bwd_cross_workspace_bytes(2, 4, 2, 5) > 0


def test_a_failed_workspace_query_is_asked_again(monkeypatch):
    """A CUDA error during the query does not stay: the next call of those sizes gets its workspace, and that is kept."""
    answers = [-1, -1, 4096]

    class Lib:
        def attn_fwd_decode_workspace_bytes(self, *sizes):
            return answers.pop(0)

    monkeypatch.setattr(attn, "lib", Lib())
    sizes = ("attn_fwd_decode_workspace_bytes", 77, 2, 4, 2, 1, 64, 16, 4)
    assert [attn._workspace_bytes(*sizes) for _ in range(4)] == [-1, -1, 4096, 4096]


def test_host_tensors_are_refused():
    import torch

    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    cache = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for f in (lambda: attn.forward_cross(q, q, q), lambda: attn.backward_cross(q, q, q, q, q[..., 0].float(), q),
              lambda: attn.forward_decode(q, cache, cache, table, lens),
              lambda: attn.forward_shared_prefix(q, cache, cache, table[0], 16, table, lens),
              lambda: attn.cache_append(q, q, cache, cache, table, lens),
              lambda: attn.cache_read(cache, cache, table, lens, 3)):
        with pytest.raises(ValueError, match="CUDA"):
            f()


# ---------------------------------------------------------------- with a device: the calls' own checks

@pytest.fixture(scope="module")
def paged():
    import torch

    dev = torch.device("cuda", torch.cuda.current_device())

    def make(f8=False):
        kind = torch.float8_e4m3fn if f8 else torch.bfloat16
        c = dict(k_cache=torch.zeros(8, 2, 16, 64, device=dev).to(kind), v_cache=torch.zeros(8, 2, 16, 64, device=dev).to(kind),
                 block_table=torch.zeros(2, 4, dtype=torch.int32, device=dev),
                 lens=torch.zeros(2, dtype=torch.int32, device=dev))
        if f8:
            c.update({n: torch.full((8, 2, 16), 127, dtype=torch.uint8, device=dev).view(torch.float8_e8m0fnu)
                      for n in ("k_scale", "v_scale")})
        return c
    return make


@pytest.mark.gpu
@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
def test_cache_calls_check_their_tensors(paged, f8):
    import torch

    c = paged(f8)
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(2, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    pre = torch.zeros(2, dtype=torch.int32, device="cuda")
    calls = [lambda c: attn.forward_decode(q, **c), lambda c: attn.cache_append(kv, kv, **c),
             lambda c: attn.cache_read(N=5, **c), lambda c: attn.forward_shared_prefix(q, prefix_table=pre, prefix_len=17, **c)]
    wrong = [dict(v_cache=c["v_cache"][:4]), dict(lens=c["lens"].long()), dict(lens=c["lens"][:1]), dict(lens=c["lens"].cpu()),
             dict(block_table=c["block_table"][0]), dict(block_table=c["block_table"].t()),
             dict(k_cache=c["k_cache"].transpose(1, 2)), dict(k_cache=c["k_cache"].to(torch.float16)),
             dict(v_cache=torch.zeros(8, 2, 16, 64, dtype=torch.float16, device="cuda"))]
    if f8:
        wrong += [dict(k_scale=None), dict(v_scale=None), dict(k_scale=None, v_scale=None),
                  dict(k_scale=c["k_scale"].view(torch.uint8)), dict(v_scale=c["v_scale"][:4])]
    else:
        s = paged(True)
        wrong += [dict(k_scale=s["k_scale"], v_scale=s["v_scale"])]
    for f in calls:
        f(c)
        for w in wrong:
            with pytest.raises((ValueError, TypeError, attn.AttnError)):
                f({**c, **w})
    for n in (-1, 33):
        with pytest.raises(ValueError, match="prefix_len"):
            attn.forward_shared_prefix(q, prefix_table=pre, prefix_len=n, **c)
    for bad in (q.float(), q[:1], q[..., :32], q.cpu()):
        with pytest.raises((ValueError, TypeError)):
            attn.forward_decode(bad, **c)
    for out in (q.float(), q[:1]):
        with pytest.raises((ValueError, TypeError)):
            attn.forward_decode(q, out=out, **c)
    with pytest.raises(attn.AttnError):   # three query heads over two
        attn.forward_decode(q[:, :3].contiguous(), **c)
    with pytest.raises((ValueError, TypeError)):
        attn.cache_append(kv, kv[:1], **c)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_a_prefix_past_32_bits_is_refused():
    """(The C entry point takes an int: 2^32 + 5 would arrive there as 5.)"""
    import torch

    page = 1 << 20
    cache = torch.zeros(1, 1, page, 32, dtype=torch.bfloat16, device="cuda")
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    pre, q = torch.zeros(4097, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, 1, 32, dtype=torch.bfloat16, device="cuda")
    for n in (1 << 31, (1 << 32) + 5):
        with pytest.raises(ValueError, match="prefix_len"):
            attn.forward_shared_prefix(q, cache, cache, pre, n, table, lens)


@pytest.mark.gpu
def test_cross_calls_check_their_tensors():
    import torch

    q = torch.zeros(2, 4, 40, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(2, 2, 9, 64, dtype=torch.bfloat16, device="cuda")
    lens = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    o, lse = attn.forward_cross(q, k, k, lens)
    good = dict(q=q, k=k, v=k, k_lens=lens)
    for w in (dict(k_lens=lens.long()), dict(k_lens=lens[:1]), dict(k_lens=lens.cpu()), dict(v=k[:, :, :8]), dict(k=k.float()),
              dict(k=k[:1]), dict(q=q[:, :3].contiguous()), dict(q=q[0]), dict(v=k.cpu()), dict(scale=math.nan)):
        with pytest.raises((ValueError, TypeError, attn.AttnError)):
            attn.forward_cross(**{**good, **w})
        with pytest.raises((ValueError, TypeError, attn.AttnError)):
            attn.backward_cross(o=o, lse=lse, dout=o, **{**good, **w})
    for w in (dict(o=o.float()), dict(lse=lse[..., None]), dict(dout=o[:1])):
        with pytest.raises((ValueError, TypeError)):
            attn.backward_cross(**{**good, **dict(o=o, lse=lse, dout=o), **w})
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_workspaces_that_are_too_small_are_refused(paged):
    """Long sequences (so that units are split), a prefix for many rows, cross attention of many rows."""
    import torch

    torch.zeros(1, device="cuda")
    kinds = {
        "decode": attn.attn_fwd_decode_workspace_bytes(2, 4, 2, 1, 64, 16, 4000),
        "prefix": attn.attn_fwd_shared_prefix_workspace_bytes(64, 4, 2, 1, 64, 16, 4, 4000, 0),
        "cross": attn.attn_fwd_cross_workspace_bytes(2, 4, 2, 500, 700, 64),
        "cross_bwd": attn.attn_bwd_cross_workspace_bytes(2, 4, 2, 500),
    }
    sizes = {"decode": dict(max_pages=4000), "prefix": dict(B=64, prefix_len=4000),
             "cross": dict(Nq=500, Nk=700), "cross_bwd": dict(Nq=500, Nk=700)}
    for which, need in kinds.items():
        assert need > 0
        assert call(which, workspace_bytes=need - 1, **sizes[which]) == INVALID
        assert call(which, workspace=None, **sizes[which]) == INVALID
        assert call(which, workspace=None, workspace_bytes=0, **sizes[which]) == INVALID
