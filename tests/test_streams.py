"""Calls on another stream than the current one: the memory of their outputs is neither still in use by the current
stream when they write it, nor taken by a later call while the current stream still reads it (needs a B200)."""
import pytest
import torch

from kv_cases import Cache, bf16, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tiled_attention_forward_03_b200 as mod
    return mod


def calls(attn):
    """name -> a call of each entry point that allocates its outputs, as a function of the stream."""
    g = gen(1)
    q, k, v, do = (bf16(g, 2, h, 200, 64).cuda() for h in (4, 2, 2, 4))
    f8 = [x.to(torch.float8_e4m3fn) for x in (q, k, v)]
    cos_t, sin_t = attn.rope_tables(200, 64, device="cuda")
    o, lse = attn.forward(q, k, v)
    ro, rlse = attn.forward_rope(q, k, v, cos_t, sin_t)
    c = Cache(2, [100, 37], 2, 64, 16, True, prefix=50)
    kc, vc, table, lens, sc = c.on_gpu()
    pre, new = c.prefix_table.cuda(), bf16(g, 2, 4, 3, 64).cuda()
    many = q[:, :, :40].contiguous()
    return {
        "forward": lambda s: attn.forward(q, k, v, stream=s),
        "backward": lambda s: attn.backward(q, k, v, o, lse, do, stream=s),
        "forward_fp8": lambda s: attn.forward_fp8(*f8, 1.0, 1.0, 1.0, stream=s),
        "rope_tables": lambda s: attn.rope_tables(200, 64, device="cuda", stream=s),
        "rope": lambda s: attn.rope(q, k, cos_t, sin_t, stream=s),
        "rope_inverse": lambda s: attn.rope_inverse(q, k, cos_t, sin_t, stream=s),
        "forward_rope": lambda s: attn.forward_rope(q, k, v, cos_t, sin_t, stream=s),
        "backward_rope": lambda s: attn.backward_rope(q, k, v, cos_t, sin_t, ro, rlse, do, stream=s),
        "cache_read": lambda s: attn.cache_read(kc, vc, table, lens, 90, stream=s, **sc),
        "forward_decode": lambda s: attn.forward_decode(new, kc, vc, table, lens, stream=s, **sc),
        "forward_shared_prefix": lambda s: attn.forward_shared_prefix(many, kc, vc, pre, 50, table, lens, stream=s, **sc),
        "forward_cross": lambda s: attn.forward_cross(many, k, v, stream=s),
        "backward_cross": lambda s: attn.backward_cross(q, k, v, o, lse, do, stream=s),
    }


NAMES = ["forward", "backward", "forward_fp8", "rope_tables", "rope", "rope_inverse", "forward_rope", "backward_rope",
         "cache_read", "forward_decode", "forward_shared_prefix", "forward_cross", "backward_cross"]


@pytest.fixture(scope="module")
def made(attn):
    made = calls(attn)
    assert list(made) == NAMES
    return made


@pytest.mark.parametrize("name", NAMES)
def test_outputs_on_another_stream(made, name):
    call, side = made[name], torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    # blocks of the outputs' sizes, freed while the current stream has yet to read them
    held = [torch.full_like(t, 7) for t in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    kept = [t.clone() for t in held]
    del held
    got = call(side)
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in kept), "written while the current stream still used the memory"
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # and outputs that the current stream has yet to read, freed before the next call
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(100_000_000)
    kept = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):
        over = [torch.full_like(t, 9) for t in want for _ in range(2)]
    call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want)), "taken again while the current stream still read it"
    del over
