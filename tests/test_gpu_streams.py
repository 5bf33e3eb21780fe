"""Calls on a stream given by name (stream=): what they allocate belongs to it."""
import pytest
import torch

import bf16_causal_prefill_fwd_b200 as b2

pytestmark = pytest.mark.gpu


def bf16(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def qkv(seed, *lead):
    return [bf16(3 * seed + i, *lead, h, 128) for i, h in enumerate((8, 2, 2))]


LENS = [0, 300, 301, 900]
CALLS = {
    "attn": lambda x, **kw: b2.attn_func(*x, return_lse=True, **kw),
    "fp8": lambda x, **kw: b2.attn_func(*x, fp8=True, return_lse=True, **kw),
    "fp8 per head": lambda x, **kw: b2.attn_func(*x, fp8=True, granularity="head", return_lse=True, **kw),
    "fp8 fused q": lambda x, **kw: b2.attn_func(*x, fp8=True, fused_q=True, return_lse=True, **kw),
    "varlen": lambda x, **kw: b2.attn_varlen_func(*(t[0] for t in x), LENS, return_lse=True, **kw),
    "varlen fp8": lambda x, **kw: b2.attn_varlen_func(*(t[0] for t in x), LENS, fp8=True, return_lse=True, **kw),
    "quantize": lambda x, **kw: b2.quantize_fp8(x[0], **kw),
    "quantize kv": lambda x, **kw: b2.quantize_kv_fp8(*x[1:], **kw),
    "quantize qkv": lambda x, **kw: b2.quantize_qkv_fp8(*x, hadamard=True, **kw),
}


def owner(t):
    """Handle of the stream whose pool t's memory is in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


def same(got, want):
    return all(torch.equal(g.view(torch.uint8), w.view(torch.uint8)) for g, w in zip(got, want, strict=True))


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_calls_on_streams_given_by_name_share_no_memory(name, raw):
    """Two busy streams with other inputs each, and memory taken and filled on the current stream once a call has
    returned."""
    xs = [qkv(i, 1, 900) for i in range(2)]
    want = [CALLS[name](x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for s, x in zip(streams * 2, xs * 2):
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        got.append(CALLS[name](x, stream=s.cuda_stream if raw else s))
        for n in (64, 512, 8192, *(t.numel() * t.element_size() for t in got[-1])):
            torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
        assert all(owner(t) == s.cuda_stream for t in got[-1])
    torch.cuda.synchronize()
    assert b2.check() == 0
    assert all(same(g, w) for g, w in zip(got, want * 2))


def test_the_default_stream_and_given_outputs():
    x = qkv(5, 1, 900)
    want = CALLS["attn"](x)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for handle in (0, 1):
            got = CALLS["attn"](x, stream=handle)
            assert all(owner(t) == 0 for t in got)
            torch.cuda.synchronize()
            assert same(got, want)
    out, side = torch.empty_like(want[0]), torch.cuda.Stream()
    assert b2.attn_fwd(q=x[0], k=x[1], v=x[2], out=out, stream=side) is out
    side.synchronize()
    assert torch.equal(out, want[0]) and b2.check() == 0
