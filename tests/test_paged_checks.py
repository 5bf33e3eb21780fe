"""Argument checks of the paged-cache operators, on the host: what the binding
refuses before the library is called (the library's functions replaced by
stand-ins that launch nothing, so these tests run on CPU tensors and reach no
GPU), and what
the C entry points refuse before they touch a device."""
import ctypes
import struct

import pytest
import torch

from bf16_causal_prefill_fwd_b200 import _binding as b
from bf16_causal_prefill_fwd_b200 import _paged as p

E4M3 = torch.float8_e4m3fn


class Stub:
    """Stands for the library: records the calls, launches nothing."""

    def __init__(self):
        self.calls = []
        i, vp, sz, f = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
        types = {"slots": [vp, sz, i, vp, vp, i, i, i, vp, i] + [vp] * 7, "append": [vp, vp, sz, sz, i, vp, vp, vp],
                 "fwd": [vp, sz, vp, vp, sz, i, vp, vp, i, i, i, i, i, f, vp, vp, vp, sz, vp]}
        self.fns = [ctypes.CFUNCTYPE(i, *t)(self._record(n)) for n, t in types.items()]
        self.fns.append(ctypes.CFUNCTYPE(sz, i, i, i, i)(lambda *a: 64))
        self.addresses = [ctypes.cast(x, ctypes.c_void_p).value for x in self.fns]

    def _record(self, name):
        def fn(*args):
            cache = {"append": 5, "fwd": 2}.get(name)
            args = list(args)
            if cache is not None:
                args[cache] = CACHE.unpack(ctypes.string_at(args[cache], CACHE.size))
            self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture(scope="module")
def real():
    from bf16_causal_prefill_fwd_b200 import build
    build.build()
    return b.load_library()


@pytest.fixture
def lib(real):
    stub, native = Stub(), p._load()
    native.bind(*stub.addresses, True)
    yield stub
    p._bind(native)


CACHE = struct.Struct("@2P6q6i2P")  # b200attn_paged_cache
P, PS, HQ, HKV, D, T, B, W = 6, 16, 8, 2, 128, 5, 3, 4


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def attn(lib, q=None, kc=None, vc=None, table=None, cu=None, kv=None, **kw):
    kc = bf16(P, PS, HKV, D) if kc is None else kc
    return p.attn_paged_fwd(bf16(T, HQ, kc.shape[-1]) if q is None else q, kc, bf16(P, PS, HKV, D) if vc is None else vc,
                            ints(B, W) if table is None else table, ints(B + 1) if cu is None else cu,
                            ints(B) if kv is None else kv, stream=0, **kw)


def append(lib, k=None, v=None, kc=None, vc=None, slots=None, **kw):
    return p.paged_append_kv(bf16(T, HKV, D) if k is None else k, bf16(T, HKV, D) if v is None else v,
                             bf16(P, PS, HKV, D) if kc is None else kc, bf16(P, PS, HKV, D) if vc is None else vc,
                             ints(T) if slots is None else slots, stream=0, **kw)


def slots(lib, table=None, ctx=None, new=None, total=T, ps=PS, **kw):
    return p.paged_slots(ints(B, W) if table is None else table, ints(B) if ctx is None else ctx,
                         ints(B) if new is None else new, total, ps, stream=0, **kw)


def test_documented_calls_reach_the_library(lib):
    o = attn(lib)
    assert o.shape == (T, HQ, 128) and o.dtype == torch.bfloat16
    o, lse = attn(lib, return_lse=True, max_seqlen_q=2, causal=False, softmax_scale=0.5, out=bf16(T, HQ, D))
    assert lse.shape == (HQ, T)
    scale = dict(k_scale=torch.ones(HKV), v_scale=torch.ones(HKV))
    e4m3 = torch.zeros(P, PS, HKV, 192, dtype=torch.uint8), torch.zeros(P, PS, HKV, D, dtype=torch.uint8)
    attn(lib, kc=e4m3[0], vc=e4m3[1], **scale)
    append(lib)
    append(lib, k=bf16(T, HKV, 192), kc=e4m3[0].view(E4M3), vc=e4m3[1].view(E4M3), **scale)
    cu, kv, pos, sl = slots(lib)
    assert [t.numel() for t in (cu, kv, pos, sl)] == [B + 1, B, T, T] and all(t.dtype == torch.int32 for t in (cu, kv, pos, sl))
    head = ints(1)
    out = slots(lib, free_pages=ints(7), free_head=head, free_head_out=head)
    assert out[4] is head
    assert slots(lib, free_pages=ints(0), free_head=head)[4].shape == (1,)
    assert len(lib.calls) == 8


def test_views_the_kernels_take_as_they_are(lib):
    """Slices of a fused projection, a [pages, heads, rows, d] cache, K and V in one buffer, a wider table."""
    qkv = bf16(T, (HQ + 2 * HKV) * D)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([HQ * D, HKV * D, HKV * D], 1))
    hnd = bf16(P, HKV, PS, D).permute(0, 2, 1, 3)
    both = bf16(P, 2, PS, HKV, D)
    attn(lib, q=q, kc=hnd, vc=both[:, 1], table=ints(B, 9)[:, :W])
    append(lib, k=k, v=v, kc=both[:, 0], vc=both[:, 1])
    name, args = lib.calls[0]
    assert name == "fwd" and args[1] == qkv.stride(0) and args[4] == 9 and args[5] == W
    strides = args[2][2:8]
    assert strides == (PS * HKV * D, D, PS * D, 2 * PS * HKV * D, HKV * D, D)


def test_one_layers_call_takes_the_buffers_of_its_halves(lib):
    """What a captured step has to keep alive can be given to attn_paged_func as to attn_paged_fwd."""
    out, ws = bf16(T, HQ, D), torch.zeros(64, dtype=torch.uint8)
    got = p.attn_paged_func(bf16(T, HQ, D), bf16(T, HKV, D), bf16(T, HKV, D), bf16(P, PS, HKV, D), bf16(P, PS, HKV, D),
                            ints(B, W), ints(B + 1), ints(B), ints(T), max_seqlen_q=2, out=out, workspace=ws, stream=0)
    assert got is out and [name for name, _ in lib.calls] == ["append", "fwd"]
    assert lib.calls[1][1][14] == out.data_ptr() and lib.calls[1][1][16:18] == [ws.data_ptr(), 64]


def test_no_new_tokens_is_no_work(lib):
    o = attn(lib, q=bf16(0, HQ, D))
    assert o.shape == (0, HQ, D) and lib.calls == []


@pytest.mark.parametrize("bad", [
    dict(q=torch.zeros(T, HQ, D)), dict(q=bf16(T, HQ, 64)), dict(q=bf16(T, 7, D)), dict(q=bf16(T, HQ * D)),
    dict(q=bf16(T, D, HQ).transpose(1, 2)), dict(q=bf16(T, HQ * D + 4)[:, : HQ * D].unflatten(1, (HQ, D))),
    dict(q=bf16(1, HQ, D).expand(T, HQ, D)), dict(q=bf16(T, HQ, D).as_strided((T, HQ, D), (D, D, 1))),
    dict(kc=bf16(P, PS, HKV, D).float()), dict(kc=bf16(P, PS, 3, D)), dict(vc=bf16(P + 1, PS, HKV, D)),
    dict(kc=bf16(PS, HKV, D)), dict(kc=bf16(P, PS, D, HKV).transpose(2, 3)),
    dict(kc=bf16(P, PS, HKV, D + 4)[..., :D]), dict(kc=bf16(1, PS, HKV, D).expand(P, PS, HKV, D)),
    dict(kc=torch.zeros(P, PS, HKV, D, dtype=E4M3), vc=torch.zeros(P, PS, HKV, D, dtype=E4M3)),
    dict(k_scale=torch.ones(HKV)), dict(table=ints(B + 1, W)), dict(table=ints(B, 0)), dict(table=ints(B, W).long()),
    dict(table=ints(W, B).t()), dict(table=ints(1, W).expand(B, W)), dict(cu=ints(B)), dict(cu=ints(2 * B + 2)[::2]),
    dict(kv=ints(B + 1)), dict(kv=ints(B).long()), dict(kv=ints(0)), dict(kv=[1, 2, 3]), dict(q=None, max_seqlen_q=0),
    dict(out=bf16(T, HQ, 64)), dict(out=torch.zeros(T, HQ, D)), dict(workspace=b"x"),
    dict(workspace=torch.zeros(200, dtype=torch.uint8)[::2])])
def test_attn_refuses(lib, bad):
    with pytest.raises(ValueError):
        attn(lib, **bad)
    assert lib.calls == []


@pytest.mark.parametrize("bad", [
    dict(k=bf16(T, HKV + 1, D)), dict(k=bf16(T + 1, HKV, D)), dict(v=bf16(T, HKV, 64)), dict(v=torch.zeros(T, HKV, D)),
    dict(slots=ints(T + 1)), dict(slots=ints(T).long()), dict(slots=ints(2 * T)[::2]), dict(k=None, v_scale=torch.ones(HKV)),
    dict(kc=torch.zeros(P, PS, HKV, D, dtype=E4M3), vc=torch.zeros(P, PS, HKV, D, dtype=E4M3), k_scale=torch.ones(HKV)),
    dict(kc=torch.zeros(P, PS, HKV, D, dtype=E4M3), vc=torch.zeros(P, PS, HKV, D, dtype=E4M3),
         k_scale=torch.ones(HKV).double(), v_scale=torch.ones(HKV))])
def test_append_refuses(lib, bad):
    with pytest.raises(ValueError):
        append(lib, **bad)
    assert lib.calls == []


@pytest.mark.parametrize("bad", [
    dict(ctx=ints(B).long()), dict(ctx=ints(0)), dict(new=ints(B + 1)), dict(table=ints(B + 1, W)), dict(total=-1), dict(ps=0),
    dict(free_head=ints(1)), dict(free_pages=ints(4)), dict(free_pages=ints(4).long(), free_head=ints(1)),
    dict(free_pages=ints(4), free_head=ints(2)), dict(free_pages=ints(4), free_head=ints(1), free_head_out=ints(0)),
    dict(free_pages=[1, 2], free_head=ints(1))])
def test_slots_refuses(lib, bad):
    with pytest.raises(ValueError):
        slots(lib, **bad)
    assert lib.calls == []


def test_cpu_tensors_are_refused(real):
    for call in (attn, append, slots):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call(None)


def test_arguments_of_other_kinds_are_refused(lib):
    for bad in (dict(q="x"), dict(kc=None, k_scale="x"), dict(max_seqlen_q=1.5), dict(max_seqlen_q=2 ** 70)):
        with pytest.raises(ValueError):
            attn(lib, **bad)
    with pytest.raises(TypeError):
        attn(lib, softmax_scale="x")
    with pytest.raises(ValueError):
        slots(lib, total=2.5)
    assert lib.calls == []


# ------------------------------------------------------------------------------------------- C entry points

FAKE = 0x10000  # 16-byte aligned, never dereferenced


def cache(k=FAKE, v=FAKE, page=PS * HKV * D, token=HKV * D, head=D, pages=P, ps=PS, h=HKV, dqk=D, dv=D, dtype=0, ks=0, vs=0):
    return CACHE.pack(k, v, page, token, head, page, token, head, pages, ps, h, dqk, dv, dtype, ks, vs)


def c_attn(lib, c, q=FAKE, stride=HQ * D, table=FAKE, row=W, width=W, cu=FAKE, kv=FAKE, batch=B, total=T, maxq=T, hq=HQ,
           causal=1, scale=0.0, o=FAKE, lse=None, ws=FAKE, wsb=1 << 40):
    return lib.b200attn_paged_fwd(q, stride, c, table, row, width, cu, kv, batch, total, maxq, hq, causal, scale, o, lse, ws,
                                  wsb, None)


def test_attn_entry_point_refuses(real):
    assert c_attn(real, None) == -1
    for bad in (dict(k=0), dict(v=FAKE + 8), dict(pages=0), dict(ps=0), dict(page=12), dict(token=-8), dict(head=0), dict(dtype=1)):
        assert c_attn(real, cache(**bad)) == -1, bad
    for bad in (dict(ps=24), dict(dqk=64), dict(dv=64), dict(dtype=7), dict(pages=1 << 28)):
        assert c_attn(real, cache(**bad)) == -2, bad
    for bad in (dict(q=None), dict(q=FAKE + 2), dict(stride=4), dict(stride=0), dict(stride=8), dict(table=None), dict(width=0), dict(cu=None), dict(kv=None),
                dict(batch=0), dict(total=-1), dict(maxq=0), dict(hq=3), dict(causal=2), dict(scale=float("nan")), dict(o=None),
                dict(lse=FAKE + 2), dict(cu=FAKE + 1)):
        assert c_attn(real, cache(), **bad) == -1, bad
    assert c_attn(real, cache(h=1), hq=129, stride=129 * D) == -2                     # a group of more than 128 heads
    assert c_attn(real, cache(), width=(1 << 27) + 1) == -2           # keys past 32-bit counts
    assert c_attn(real, cache(), total=1 << 28, hq=HQ) == -2          # rows past 32-bit counts
    assert c_attn(real, cache(h=1, token=D), hq=128, stride=128 * D, total=1 << 20, maxq=1 << 20, width=1 << 17) == -2  # the line of work, too
    assert c_attn(real, cache(), ws=None) == -5
    assert c_attn(real, cache(), wsb=64) == -5
    assert c_attn(real, cache(), o=FAKE + 16) == -1                    # rows leave in stores of 32 bytes
    assert c_attn(real, cache(), ws=FAKE + 4) == -5
    assert c_attn(real, cache(), total=0, q=None, o=None) == 0        # nothing to do


def test_append_entry_point_refuses(real):
    def call(c, k=FAKE, v=FAKE, ks=HKV * D, vs=HKV * D, total=T, s=FAKE):
        return real.b200attn_paged_append(k, v, ks, vs, total, c, s, None)
    assert call(None) == -1
    assert call(cache(dtype=1)) == -1                                 # e4m3 without scales
    assert call(cache(ps=8)) == -2
    for bad in (dict(k=None), dict(v=FAKE + 8), dict(ks=4), dict(total=-1), dict(s=None), dict(s=FAKE + 2)):
        assert call(cache(), **bad) == -1, bad
    assert call(cache(h=1 << 16), ks=D << 16, vs=D << 16, total=1 << 20) == -2                # units past 32 bits
    assert call(cache(), total=0, k=None) == 0


def test_slots_entry_point_refuses(real):
    def call(table=FAKE, row=W, width=W, ctx=FAKE, new=FAKE, batch=B, total=T, ps=PS, free=None, count=0, head=None, hout=None,
             cu=FAKE, kv=FAKE, pos=FAKE, s=FAKE):
        return real.b200attn_paged_slots(table, row, width, ctx, new, batch, total, ps, free, count, head, hout, cu, kv, pos, s,
                                         None)
    for bad in (dict(table=None), dict(width=0), dict(ctx=None), dict(new=FAKE + 1), dict(batch=0), dict(total=-1), dict(ps=0),
                dict(free=FAKE), dict(free=FAKE, head=FAKE), dict(count=-1), dict(cu=None), dict(kv=None), dict(pos=None),
                dict(s=FAKE + 2)):
        assert call(**bad) == -1, bad
    assert call(batch=16385) == -2
    assert call(total=1 << 30) == -2


def test_workspace_sizes(real):
    ws = real.b200attn_paged_fwd_workspace_bytes
    assert ws(0, 1, 8, 2) == ws(1, 0, 8, 2) == ws(1, 1, 7, 2) == 0
    few = ws(64, 1, 32, 8)
    assert 0 < few < 16 << 20 and ws(64, 4, 32, 8) == few             # 16 rows per key/value head
    assert ws(64, 5, 32, 8) > few                                     # the many-rows kernel: 256 rows a slot
    assert ws(5, 5, 32, 8) < ws(64, 64, 32, 8) == ws(5000, 5000, 32, 8) < 64 << 20


def test_a_workspace_for_more_tokens_is_enough_for_fewer(real):
    """As large as the call itself needs with the same arguments, and growing with both."""
    ws = real.b200attn_paged_fwd_workspace_bytes
    sizes = [1, 2, 3, 4, 5, 6, 7, 8, 11, 12, 16, 17, 31, 64, 65, 1000]
    for hq, hkv in ((32, 8), (8, 2), (16, 16), (28, 4), (128, 1), (5, 1)):
        for total in sizes:
            for max_q in sizes:
                assert ws(total, max_q, hq, hkv) == ws(total, min(max_q, total), hq, hkv)
                assert all(ws(t, m, hq, hkv) <= ws(total, max_q, hq, hkv) for t in sizes if t <= total
                           for m in sizes if m <= max_q)


@pytest.mark.parametrize("total,max_q,hq", [(1, 8, 32), (3, 64, 8), (4, 5, 32), (5, 5, 32), (64, 2, 32)])
def test_the_stated_workspace_is_enough_for_the_call(real, total, max_q, hq):
    hkv = hq // 4
    need = real.b200attn_paged_fwd_workspace_bytes(total, max_q, hq, hkv)
    args = dict(stride=hq * D, total=total, maxq=max_q, hq=hq)
    c = cache(h=hkv, token=hkv * D, page=PS * hkv * D)
    assert c_attn(real, c, wsb=need - 1, **args) == -5
    if not torch.cuda.is_available():  # past the checks: no device
        assert c_attn(real, c, wsb=need, **args) == -3


# ------------------------------------------------------------------------------------------- the compiled binding

def test_the_binding_is_rebuilt_for_another_torch_or_python(monkeypatch, tmp_path):
    from bf16_causal_prefill_fwd_b200 import build
    ran = []

    def compiler(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("binary")
        return type("Done", (), {"returncode": 0, "stdout": "", "stderr": ""})

    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "_paged_binding.so"))
    monkeypatch.setattr(build.subprocess, "run", compiler)
    for _ in range(2):
        build.build_binding()
    assert len(ran) == 1
    monkeypatch.setattr(torch, "__version__", "0.0")
    for _ in range(2):
        build.build_binding()
    assert len(ran) == 2
    monkeypatch.setattr(build.sys, "version", "2.7 (old)")
    build.build_binding()
    assert len(ran) == 3
    (tmp_path / "_paged_binding.so.stamp").unlink()   # one that nothing is known of
    build.build_binding()
    assert len(ran) == 4


def test_a_binding_built_for_another_torch_is_not_loaded(monkeypatch, real):
    p._load()
    monkeypatch.setattr(p, "_native", None)
    monkeypatch.setattr(torch, "__version__", "0.0")
    with pytest.raises(RuntimeError, match="was built for torch"):
        p._load()
