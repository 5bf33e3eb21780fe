"""The paged-cache operators on the GPU against their plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import bf16_causal_prefill_fwd_b200 as b2
from paged_reference import Paged, attention, check_attention, make

pytestmark = pytest.mark.gpu

SHAPES = [(32, 8, 128), (16, 16, 192), (8, 1, 128), (28, 4, 128), (6, 2, 192), (16, 1, 128)]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def run(p: Paged, **kw):
    d = p.cuda()
    got = b2.attn_paged_fwd(*d.args(), **d.scales(), return_lse=True, **kw)
    assert b2.check() == 0
    return got


# ------------------------------------------------------------------------------------------- few rows (decoding)

DECODE_LENS = [
    ([1], [1]),
    ([1, 1, 1, 1, 1, 1, 1, 1], [1, 15, 16, 17, 63, 64, 65, 1000]),
    ([1, 0, 1, 0, 1], [300, 5, 0, 0, 129]),          # no new token; a token without keys
    ([1] * 37, [1 + 53 * i for i in range(37)]),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads", SHAPES)
@pytest.mark.parametrize("lens", DECODE_LENS)
def test_decode_matches_the_plain_form(lens, heads, e4m3):
    p = make(*lens, *heads, page_size=16, e4m3=e4m3, seed=len(lens[0]))
    o, lse = run(p, max_seqlen_q=1)
    check_attention(p, o, lse)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page_size", [16, 32, 48, 64, 80, 128, 256])
def test_decode_page_sizes(page_size, e4m3):
    p = make([1, 1, 1], [page_size - 1, 3 * page_size + 5, 777], 8, 2, 128, page_size, e4m3, seed=page_size)
    o, lse = run(p, max_seqlen_q=1)
    check_attention(p, o, lse)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("e4m3", [False, True])
def test_few_new_tokens_of_one_request(e4m3, causal):
    """Up to 16 rows per key/value head; requests with fewer keys than new tokens have rows that see nothing."""
    p = make([4, 2, 3, 0, 4, 4], [200, 64, 2, 9, 0, 1], 8, 2, 128, 32, e4m3, seed=3)
    o, lse = run(p, max_seqlen_q=4, causal=causal)
    check_attention(p, o, lse, causal)
    unseen = lse == -math.inf
    assert bool((o.transpose(0, 1)[unseen] == 0).all())


def test_decode_of_one_long_request_is_split_over_the_gpu():
    p = make([1], [20011], 8, 2, 128, 16, seed=7)
    o, lse = run(p, max_seqlen_q=1)
    check_attention(p, o, lse)


def test_decode_softmax_scale_and_large_scores():
    p = make([1, 1], [500, 77], 8, 2, 128, 16, seed=8, spread=6.0)
    o, lse = run(p, max_seqlen_q=1, softmax_scale=0.3)
    check_attention(p, o, lse, softmax_scale=0.3)


# ------------------------------------------------------------------------------------------- many rows (chunks)

CHUNK_LENS = [
    ([17], [17]),                                        # a prompt's first chunk
    ([33, 1, 0, 64, 5], [33, 700, 40, 64, 1300]),        # chunks and decoding requests together
    ([200, 130], [1000, 130]),
    ([65, 40, 20], [30, 0, 257]),                        # more new tokens than keys: rows that see nothing
]


@pytest.mark.parametrize("B", [32, 33, 64, 91])
def test_chunks_of_many_requests(B):
    """More requests than a warp's lanes, some without new tokens: runs begin in any of them."""
    q_lens = [(5 * i + 3) % 29 if i % 6 else 0 for i in range(B)]
    p = make(q_lens, [n + (37 * i) % 201 for i, n in enumerate(q_lens)], 8, 2, 128, 16, seed=B)
    o, lse = run(p)
    check_attention(p, o, lse)


def test_chunk_of_groups_that_are_no_power_of_two():
    p = make([150, 260], [700, 260], 14, 2, 128, 16, seed=41)   # 18 tokens a row tile, the line's length by Euclid's steps
    o, lse = run(p)
    check_attention(p, o, lse)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads", SHAPES)
@pytest.mark.parametrize("lens", CHUNK_LENS)
def test_chunk_matches_the_plain_form(lens, heads, e4m3):
    p = make(*lens, *heads, page_size=16, e4m3=e4m3, seed=sum(lens[0]))
    o, lse = run(p)
    check_attention(p, o, lse)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page_size", [16, 48, 64, 96, 128, 256])
def test_chunk_page_sizes(page_size, e4m3):
    p = make([70, 9], [3 * page_size + 70, page_size + 1], 8, 2, 128, page_size, e4m3, seed=page_size)
    o, lse = run(p, max_seqlen_q=70)
    check_attention(p, o, lse)


@pytest.mark.parametrize("e4m3", [False, True])
def test_chunk_without_the_causal_mask(e4m3):
    p = make([50, 150, 3], [400, 1, 129], 8, 2, 128, 32, e4m3, seed=5)
    o, lse = run(p, causal=False)
    check_attention(p, o, lse, causal=False)


@pytest.mark.parametrize("heads", [(128, 1, 128), (5, 1, 128), (48, 2, 192)])
def test_large_and_odd_groups(heads):
    """A group of 128 heads is one token per tile; five heads leave rows of a tile unused."""
    p = make([7, 30], [300, 90], *heads, page_size=16, seed=heads[0])
    o, lse = run(p)
    check_attention(p, o, lse)


@pytest.mark.parametrize("e4m3", [False, True])
def test_chunk_of_one_long_request_is_split_over_the_gpu(e4m3):
    p = make([40], [9000], 4, 1, 128, 64, e4m3, seed=17)
    o, lse = run(p)
    check_attention(p, o, lse)


@pytest.mark.parametrize("e4m3", [False, True])
def test_chunk_large_scores(e4m3):
    p = make([130], [700], 4, 2, 128, 16, e4m3, seed=18, spread=6.0)
    o, lse = run(p, softmax_scale=0.3)
    check_attention(p, o, lse, softmax_scale=0.3)


# ------------------------------------------------------------------------------------------- slots

def plain_slots(table, ctx, new, total, ps, free=None, head=0):
    table = [list(r) for r in table]
    cu, kv, pos, slots = [0], [], [], []
    for b, (c, n) in enumerate(zip(ctx, new)):
        cu.append(cu[-1] + n)
        kv.append(c + n)
        if free is not None:
            for j in range(-(-c // ps), -(-(c + n) // ps)):
                table[b][j] = free[head]
                head += 1
        for x in range(c, c + n):
            pos.append(x)
            slots.append(table[b][x // ps] * ps + x % ps)
    pad = total - len(pos)
    return cu, kv, pos + [0] * pad, slots + [-1] * pad, table, head


def slots_case(ctx, new, ps, pad, alloc, seed):
    rng = np.random.default_rng(seed)
    width = max(-(-(c + n) // ps) for c, n in zip(ctx, new)) + 1
    pages = rng.permutation(len(ctx) * width + 50).tolist()
    table = [[-1] * width for _ in ctx]
    for b, (c, n) in enumerate(zip(ctx, new)):
        for j in range(-(-(c if alloc else c + n) // ps)):
            table[b][j] = pages.pop()
    return table, (pages if alloc else None)


@pytest.mark.parametrize("alloc", [False, True])
@pytest.mark.parametrize("ps", [1, 7, 16, 64])
@pytest.mark.parametrize("lens", [([0], [1]), ([5, 0, 16, 31, 100], [1, 0, 1, 17, 40]), ([3] * 700, [1] * 700),
                                  ([i % 90 for i in range(2000)], [i % 4 for i in range(2000)]), ([0, 9], [0, 0])])
def test_slots_match_the_plain_form(lens, ps, alloc):
    ctx, new = lens
    total = sum(new) + 13
    table, free = slots_case(ctx, new, ps, 13, alloc, seed=ps)
    want = plain_slots(table, ctx, new, total, ps, free, 2 if alloc else 0)
    t = ints(table)
    kw = dict(free_pages=ints(free), free_head=ints([2])) if alloc else {}
    got = b2.paged_slots(t, ints(ctx), ints(new), total, ps, **kw)
    assert b2.check() == 0
    for g, w in zip(got[:4], want[:4]):
        assert g.tolist() == w
    assert t.tolist() == want[4]
    if alloc:
        assert got[4].tolist() == [want[5]]


def test_slots_head_in_place_over_steps():
    """Requests grow by steps, the head moving in place: no page is given out twice."""
    ps, B = 16, 9
    table, head = torch.full((B, 20), -1, dtype=torch.int32, device="cuda"), ints([0])
    free = torch.randperm(200, dtype=torch.int32).cuda()
    ctx = ints([0] * B)
    for step in range(6):
        new = ints([(7 * b + 11 * step) % 23 for b in range(B)])
        cu, kv, pos, slots, out = b2.paged_slots(table, ctx, new, 250, ps, free_pages=free, free_head=head, free_head_out=head)
        assert out is head
        ctx = kv
    assert b2.check() == 0
    used = table[table >= 0].tolist()
    assert len(used) == len(set(used)) == int(head)
    assert [int((r >= 0).sum()) for r in table] == [-(-n // ps) for n in ctx.tolist()]


@pytest.mark.parametrize("bad", ["negative_new", "negative_ctx", "total", "width", "both", "pages", "head"])
def test_slots_that_do_not_fit_give_an_empty_step(bad):
    ctx, new, total, free, head = [5, 20], [3, 4], 9, list(range(100, 110)), 1
    code = -1
    if bad == "negative_new":
        new = [3, -1]
    elif bad == "negative_ctx":
        ctx = [-5, 20]
    elif bad == "total":
        total = 6
    elif bad == "width":
        new, total = [3, 45], 60
    elif bad == "both":
        head = 10      # pages of 4 rows: the second request's are more than a table row holds
    elif bad == "pages":
        new, total, head, code = [3, 13], 17, 10, -6
    elif bad == "head":
        head, code = -1, -6
    table = ints([[1, -1, -1, -1], [2, 3, -1, -1]])
    before = table.clone()
    got = b2.paged_slots(table, ints(ctx), ints(new), total, 16 if bad != "both" else 4, free_pages=ints(free),
                         free_head=ints([head]))
    assert b2.check() == code
    assert got[0].tolist() == [0, 0, 0] and got[1].tolist() == [0, 0]
    assert got[3].tolist() == [-1] * total and got[4].tolist() == [head] and torch.equal(table, before)
    assert b2.check() == 0


@pytest.mark.parametrize("ps", [1 << 20, (1 << 31) - 1])
def test_slots_of_lengths_near_32_bits(ps):
    """The last position that 32 bits hold, with a page taken for it, is given; one token more does not fit."""
    last = 2 ** 31 - 1
    held, free, head = -(-(last - 5) // ps), [9, 9, 0, 9, 9], 2
    width = max(2, held + 1)
    for ctx, new, fits in ((last - 5, 5, True), (last, 0, True), (last - 5, 6, False), (last, 1, False)):
        table = torch.full((2, width), -1, dtype=torch.int32)
        table[0] = torch.arange(width)
        before = table.cuda()
        t = before.clone()
        got = b2.paged_slots(t, ints([ctx, 0]), ints([new, 1]), 9, ps, free_pages=ints(free), free_head=ints([head]))
        assert b2.check() == (0 if fits else -1)
        if fits:
            want = before.clone()
            want[1, 0] = free[head]
            page = (last - 1) // ps
            slot = page * ps + (last - 1) % ps
            assert got[0].tolist() == [0, new, new + 1] and got[1].tolist() == [ctx + new, 1]
            assert got[2].tolist() == list(range(ctx, ctx + new)) + [0] * (9 - new)
            assert got[3].tolist()[:new] == [slot - new + 1 + i for i in range(new)] and got[4].tolist() == [head + 1]
            assert got[3].tolist()[new:] == [0] + [-1] * (8 - new)
        else:
            want = before
            assert got[0].tolist() == [0, 0, 0] and got[3].tolist() == [-1] * 9 and got[4].tolist() == [head]
        assert torch.equal(t, want)


def test_slots_of_an_unset_table_entry_are_reported():
    got = b2.paged_slots(ints([[4, -1]]), ints([14]), ints([4]), 4, 16)
    assert b2.check() == -1
    assert got[3].tolist() == [4 * 16 + 14, 4 * 16 + 15, -1, -1]


# ------------------------------------------------------------------------------------------- append

def plain_codes(x, scale):
    """e4m3(x / scale) from the division in fp32: clamp, then round to nearest even."""
    y = (x.float() / scale[None, :, None]).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,d_qk,T,ps", [(8, 128, 1, 16), (8, 128, 333, 16), (3, 192, 70, 48), (1, 128, 5, 16), (16, 192, 129, 64)])
def test_append_matches_the_plain_form(H, d_qk, T, ps, e4m3):
    g = torch.Generator().manual_seed(T)
    pages = T // ps + 4
    k, v = (torch.randn(T, H, d, generator=g).to(torch.bfloat16) for d in (d_qk, 128))
    slots = torch.randperm(pages * ps, generator=g)[:T].to(torch.int32)
    slots[T // 2] = -1  # a padded row
    scales = [torch.rand(H, generator=g) * 0.01 + 0.004 for _ in range(2)]
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    caches = [torch.randn(pages, ps, H, d, generator=g).to(dt) for d in (d_qk, 128)]
    want = []
    for x, c, s in zip((k, v), caches, scales):
        w = c.clone().view(torch.uint8 if e4m3 else dt)
        rows = w.view(pages * ps, H, -1)
        y = plain_codes(x, s).view(torch.uint8) if e4m3 else x
        keep = slots >= 0
        rows[slots[keep].long()] = y[keep]
        want.append(w)
    got = [c.cuda() for c in caches]
    kw = dict(k_scale=scales[0].cuda(), v_scale=scales[1].cuda()) if e4m3 else {}
    b2.paged_append_kv(k.cuda(), v.cuda(), *got, slots.cuda(), **kw)
    assert b2.check() == 0
    for a, w in zip(got, want):
        assert torch.equal(a.cpu().view(w.dtype), w)


def test_append_of_special_values_into_e4m3():
    x = torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    vals = [math.inf, -math.inf, math.nan, 1e30, -1e30, 448.0, 449.0, 464.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -11, -0.0]
    x[0, 0, : len(vals)] = torch.tensor(vals)
    kc, vc = (torch.zeros(1, 16, 1, 128, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    one = torch.ones(1, device="cuda")
    b2.paged_append_kv(x.cuda(), x.cuda(), kc, vc, ints([3]), k_scale=one, v_scale=one)
    assert b2.check() == 0
    got = kc[0, 3, 0, : len(vals)].float().cpu().tolist()
    assert got[:2] == [448.0, -448.0] and math.isnan(got[2])
    assert got[3:] == [448.0, -448.0, 448.0, 448.0, 448.0, 2.0 ** -9, 0.0, 2.0 ** -9, 0.0]
    assert torch.equal(kc.view(torch.uint8), vc.view(torch.uint8))


def test_append_codes_of_every_bf16_value():
    """Bytes, the sign of zero included, from scales of both kinds of division."""
    scales = torch.tensor([1.0, 0.0078, 3.0, 1 / 3, 2.0 ** -60, 1.7e-30, 4.4e31, 0.02373])
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(512, 1, 128).expand(-1, 8, -1).contiguous()
    want = plain_codes(x, scales)
    kc, vc = (torch.zeros(32, 16, 8, 128, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    sc = scales.cuda()
    b2.paged_append_kv(x.cuda(), x.cuda(), kc, vc, ints(list(range(512))), k_scale=sc, v_scale=sc)
    assert b2.check() == 0
    number = ~x.float().isnan()
    for c in (kc, vc):
        got = c.cpu().view(512, 8, 128)
        assert torch.equal(got.view(torch.uint8)[number], want.view(torch.uint8)[number])
        assert bool(got.float()[~number].isnan().all())


def test_append_slots_past_the_cache_are_skipped_and_reported():
    kc, vc = (torch.zeros(2, 16, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x = torch.ones(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    b2.paged_append_kv(x, x, kc, vc, ints([31, 32, 2 ** 31 - 1]))
    assert b2.check() == -1
    assert float(kc.sum()) == 256.0 and bool((kc[1, 15] == 1).all())


# ------------------------------------------------------------------------------------------- layouts

def test_strided_caches_and_slices_of_a_fused_projection():
    """[pages, heads, rows, d] caches, K and V in one buffer, q, k and v slices of one tensor: the results of
    contiguous copies, bit for bit."""
    p = make([1, 1, 1], [40, 130, 333], 8, 2, 128, 16, seed=12).cuda()
    ref = b2.attn_paged_fwd(*p.args(), max_seqlen_q=1)
    P, ps, H, d = p.k_cache.shape
    hnd = [c.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for c in (p.k_cache, p.v_cache)]
    both = torch.stack([p.k_cache, p.v_cache], 1)
    qkv = torch.cat([p.q.flatten(1), torch.zeros(3, 2 * H * d, dtype=torch.bfloat16, device="cuda")], 1)
    q = qkv[:, : 8 * d].view(3, 8, d)
    for kc, vc in (hnd, (both[:, 0], both[:, 1])):
        assert not kc.is_contiguous()
        got = b2.attn_paged_fwd(q, kc, vc, *p.args()[3:], max_seqlen_q=1)
        assert torch.equal(got, ref)
        k, v = (torch.randn(3, H, d, device="cuda").to(torch.bfloat16) for _ in range(2))
        slots = ints([p.table[b, (n - 1) // ps].item() * ps + (n - 1) % ps for b, n in enumerate((40, 130, 333))])
        a, c = kc.clone(), vc.contiguous().clone()
        b2.paged_append_kv(k, v, kc, vc, slots)
        b2.paged_append_kv(k, v, a, c, slots)
        assert torch.equal(torch.nan_to_num(kc), torch.nan_to_num(a)) and torch.equal(torch.nan_to_num(vc), torch.nan_to_num(c))
    assert b2.check() == 0


# ------------------------------------------------------------------------------------------- contents that do not fit

@pytest.mark.parametrize("max_q", [1, None])
def test_contents_that_do_not_fit_are_skipped_and_reported(max_q):
    """A request whose lengths do not fit, or with more new tokens than announced, leaves its rows as they are; the
    others are computed."""
    n = 1 if max_q == 1 else 20
    p = make([n] * 4, [50, 60, 70, 80], 8, 2, 128, 16, seed=21)
    good = p.cuda()
    want = b2.attn_paged_fwd(*good.args(), max_seqlen_q=max_q)
    assert b2.check() == 0
    for kv in (-1, 16 * p.table.shape[1] + 1):
        bad = p.cuda()
        bad.kv_lens[2] = kv
        out = torch.full_like(want, 7.0)
        b2.attn_paged_fwd(*bad.args(), max_seqlen_q=max_q, out=out)
        assert b2.check() == -1
        assert torch.equal(out[: 2 * n], want[: 2 * n]) and torch.equal(out[3 * n:], want[3 * n:])
        assert bool((out[2 * n: 3 * n] == 7.0).all())
    for cu in ([0, n, 2 * n, 99, 4 * n], [0, n, -5, 3 * n, 4 * n], [0, n, 2 * n, n, 4 * n]):
        bad = p.cuda()
        bad.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        out = torch.full_like(want, 7.0)
        b2.attn_paged_fwd(*bad.args(), max_seqlen_q=max_q, out=out)
        assert b2.check() == -1
        assert torch.equal(out[:n], want[:n])
    assert torch.equal(b2.attn_paged_fwd(*good.args(), max_seqlen_q=max_q), want) and b2.check() == 0


def test_requests_that_share_rows_stay_in_bounds():
    """A cu_seqlens that goes back and forth gives every second request all rows: each is computed, rows keep one of
    the results, and a line of work past 32-bit counts is refused."""
    n, B = 64, 8
    p = make([n] * B, [100] * B, 8, 2, 128, 16, seed=33)
    d = p.cuda()
    d.cu.copy_(torch.tensor([0, n] * (B // 2) + [0], dtype=torch.int32))
    out = torch.full((n * B, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    b2.attn_paged_fwd(*d.args(), out=out)
    assert b2.check() == -1
    assert not bool(out.isnan().any()) and bool((out[n:] == 7.0).all())
    # 2000 requests that all have the same 65536 rows, over 1050 key blocks: 2000 * 1024 pairs of row tiles * 1050
    B, T, pages = 4000, 65536, 2100
    kc = torch.zeros(1, 64, 1, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(T, 4, 128, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(B, pages, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, T] * (B // 2) + [0], dtype=torch.int32, device="cuda")
    kv = torch.full((B,), 64 * pages, dtype=torch.int32, device="cuda")
    assert (B // 2) * (T // 64) * (64 * pages // 128) >= 2 ** 31
    out = torch.full((T, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    b2.attn_paged_fwd(q, kc, kc, table, cu, kv, causal=False, out=out)
    assert b2.check() == -1 and bool((out == 7.0).all())


@pytest.mark.parametrize("n,max_q", [(1, 1), (20, 20)])
def test_table_entries_that_are_no_page_read_as_zeros(n, max_q):
    p = make([n, n], [60, 90], 8, 2, 128, 16, seed=22)
    for entry in (-1, p.k_cache.shape[0], 2 ** 31 - 1):
        bad = p.cuda()
        bad.table[1, 2] = entry
        o = b2.attn_paged_fwd(*bad.args(), max_seqlen_q=max_q)
        assert b2.check() == -1
        zero = Paged(**{k: v if v is None else v.clone() for k, v in p.__dict__.items()})
        zero.k_cache[zero.table[1, 2].long()] = 0
        zero.v_cache[zero.table[1, 2].long()] = 0
        check_attention(zero, o)


def test_rows_behind_the_last_request_stay_as_they_are():
    for n, max_q in ((1, 1), (33, 33)):
        p = make([n, 0, n], [100, 5, 60], 8, 2, 128, 16, seed=23, pad_rows=9)
        d = p.cuda()
        out = torch.full((2 * n + 9, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        b2.attn_paged_fwd(*d.args(), max_seqlen_q=max_q, out=out)
        assert b2.check() == 0
        check_attention(p, out)
        assert bool((out[2 * n:] == 7.0).all())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,max_q", [(1, 1), (40, 40)])
def test_nan_reaches_the_rows_that_see_it_and_no_other(n, max_q, e4m3):
    p = make([n, n, n], [90, 200, 150], 8, 2, 128, 16, e4m3, seed=24)
    ref = run(p, max_seqlen_q=max_q)
    for cache in ("k_cache", "v_cache"):
        bad = Paged(**{k: v if v is None else v.clone() for k, v in p.__dict__.items()})
        page = int(bad.table[1, 1])
        getattr(bad, cache).view(torch.uint8 if e4m3 else torch.int16)[page, 3, 1, 5] = 0x7F if e4m3 else 0x7FC0
        o, lse = run(bad, max_seqlen_q=max_q)
        hit = torch.zeros(3 * n, 8, dtype=torch.bool)
        hit[n: 2 * n, 4:] = True  # key 19 of request 1, key/value head 1: seen by all its new tokens
        nan = o.isnan().any(-1).cpu()
        assert torch.equal(nan, hit)
        assert torch.equal(o[~hit.cuda()], ref[0][~hit.cuda()])
        if cache == "k_cache":
            assert bool(lse.T.isnan().cpu()[hit].all())


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
@pytest.mark.parametrize("q_lens,kv_lens,max_q", [([2, 2, 2], [90, 1, 0], 2), ([40, 40, 3], [200, 7, 0], 40)])
def test_nan_scale_gives_nan_in_its_heads_rows_that_see_a_key(q_lens, kv_lens, max_q, which):
    p = make(q_lens, kv_lens, 8, 2, 128, 16, True, seed=26)
    ref = run(p, max_seqlen_q=max_q)
    getattr(p, which)[1] = math.nan
    o, lse = run(p, max_seqlen_q=max_q)
    hit = ref[1] > -math.inf
    hit[:4] = False
    assert bool(hit.any()) and bool((ref[1][4:] == -math.inf).any())
    assert bool(o.transpose(0, 1)[hit].isnan().all()) and torch.equal(o.transpose(0, 1)[~hit], ref[0].transpose(0, 1)[~hit])
    assert torch.equal(lse[~hit], ref[1][~hit])
    if which == "k_scale":
        assert bool(lse[hit].isnan().all())
    else:
        assert torch.equal(lse, ref[1])


@pytest.mark.parametrize("n,max_q", [(1, 1), (40, 40)])
def test_infinite_query_gives_nan_in_its_row_only(n, max_q):
    for e4m3 in (False, True):
        p = make([n, n], [90, 200], 8, 2, 128, 16, e4m3, seed=25)
        ref = run(p, max_seqlen_q=max_q)[0]
        p.q[n, 3, 7] = math.inf
        o = run(p, max_seqlen_q=max_q)[0]
        assert bool(o[n, 3].isnan().all())
        rest = torch.ones(2 * n, 8, dtype=torch.bool)
        rest[n, 3] = False
        assert torch.equal(o[rest.cuda()], ref[rest.cuda()])


# ------------------------------------------------------------------------------------------- sizes

@pytest.mark.parametrize("e4m3", [False, True])
def test_many_short_requests(e4m3):
    """More requests than a block has threads."""
    B = 1300
    kv = [1 + (i * 37) % 45 for i in range(B)]
    p = make([i % 2 for i in range(B)], kv, 4, 2, 128, 16, e4m3, seed=26)
    check_attention(p, *run(p, max_seqlen_q=1))
    p = make([(i * 7) % 12 for i in range(B)], [n + 12 for n in kv], 4, 2, 128, 16, e4m3, seed=27)
    check_attention(p, *run(p, max_seqlen_q=11))


def test_decoding_and_chunk_kernels_agree():
    """The same decoding step with and without a bound on the new tokens."""
    p = make([1, 1, 1, 1], [1, 130, 64, 999], 32, 8, 128, 16, seed=28)
    few, many = run(p, max_seqlen_q=1), run(p)
    check_attention(p, *few)
    check_attention(p, *many)


def test_offsets_past_32_bits():
    """A cache whose last pages begin past 2^32 bytes and 2^31 elements."""
    pages, ps, H = 33000, 64, 8
    kc, vc = (torch.empty(pages, ps, H, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kc.numel() * 2 > 2 ** 32 and kc[:-3].numel() > 2 ** 31
    q_lens, kv_lens = [1, 1], [100, 150]
    p = make(q_lens, kv_lens, 32, H, 128, ps, seed=29)
    n = p.k_cache.shape[0]
    d = p.cuda()
    table = torch.where(d.table >= 0, d.table + (pages - n), d.table)
    slots = torch.arange((pages - n) * ps, pages * ps, dtype=torch.int32, device="cuda")
    b2.paged_append_kv(d.k_cache.flatten(0, 1), d.v_cache.flatten(0, 1), kc, vc, slots)
    for max_q in (1, None):
        o = b2.attn_paged_fwd(d.q, kc, vc, table, d.cu, d.kv_lens, max_seqlen_q=max_q)
        assert b2.check() == 0
        check_attention(p, o)
    del kc, vc


# ------------------------------------------------------------------------------------------- many keys

def repeated(q, k, v, row, kv, scale):
    """64-bit attention of q [n, d] without a mask over kv keys: the pages `row` of k and v [pages, page_size, d], which
    it may name many times. Returns o, lse and sum_j p_j |v_j| / l."""
    ps = k.shape[1]
    full, rest = kv // ps, kv % ps
    times = torch.bincount(row[:full].long(), minlength=k.shape[0])[:, None].expand(-1, ps).clone()
    if rest:
        times[int(row[full]), :rest] += 1
    x = q.double() @ k.flatten(0, 1).double().T * scale
    x[:, times.flatten() == 0] = -math.inf
    m = x.amax(1, keepdim=True)
    w = torch.exp(x - m) * times.flatten()
    l = w.sum(1, keepdim=True)
    vv = v.flatten(0, 1).double()
    return w @ vv / l, (m + l.log())[:, 0], w @ vv.abs() / l


def lost(n_new, G, kv):
    """What the fp16 probabilities of one part of a row may miss of its largest: 2^-25 each, the largest held at 2^15 by
    the decoding kernel, at 2^7 or more by the other, at 2^13 or more above 2^20 keys."""
    return kv * 2.0 ** -(40 if n_new * G <= 16 else (32 if kv <= 1 << 20 else 38))


@pytest.mark.parametrize("n_new,kv,d", [(1, (1 << 18) + 37, 128), (1, (1 << 18) + 37, 192), (8, (1 << 18) + 37, 128),
                                        (8, (1 << 18) + 37, 192), (8, (1 << 20) + 5, 128)])
def test_small_probabilities_of_a_long_e4m3_context_count(n_new, kv, d):
    """A first key 26 binades above all others, which together hold 2^-8 or more of the weight, in units that no block
    shares with another: the columns of V that only they have."""
    G, ps = 4, 64
    B = torch.cuda.get_device_properties(0).multi_processor_count * (3 if n_new == 1 else 1)
    k, v = torch.zeros(2, ps, d), torch.zeros(2, ps, 128)
    k[..., 0], v[..., 1::2] = -0.1875, 1.0
    k[0, 0, 0], v[0, 0] = 18.0, 0.0
    v[0, 0, ::2] = 1.0
    q = torch.randn(n_new, d, generator=torch.Generator().manual_seed(61)).to(torch.bfloat16)
    q[:, 0] = 1.0
    row = torch.ones(kv // ps + 1, dtype=torch.int32)
    row[0] = 0
    o, lse, _ = repeated(q, k, v, row, kv, 1.0)
    one = torch.ones(1, device="cuda")
    got, got_lse = b2.attn_paged_fwd(
        q.cuda()[:, None].expand(-1, G, -1).repeat(B, 1, 1), *(x.to(torch.float8_e4m3fn).cuda()[:, :, None] for x in (k, v)),
        row.cuda().repeat(B, 1), ints([n_new * i for i in range(B + 1)]), ints([kv] * B), max_seqlen_q=n_new, causal=False,
        softmax_scale=1.0, k_scale=one, v_scale=one, return_lse=True)
    assert b2.check() == 0
    # beside what fp16 loses: a half step of fp16 and of bf16, scores (2^-24 of 18 or less) and the exponential, and
    # kv / 16 fp32 accumulations that may cut off
    off = 2.0 ** -11 + 2.0 ** -8 + 18 * 2.0 ** -23 + 2.0 ** -22 + kv / 16 * 2.0 ** -23
    bound = (o.abs() * off + lost(n_new, G, kv))[None, :, None]
    assert bool((bound[..., 1::2] < o[None, :, None, 1::2] / 4).all())
    assert bool(((got.view(B, n_new, G, 128).double().cpu() - o[None, :, None]).abs() <= bound).all())
    assert bool(((got_lse.view(G, B, n_new).double().cpu() - lse).abs() <= 2.0 ** -18 + kv / 64 * 2.0 ** -24).all())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n_new,kv", [(1, (1 << 20) - 9), (1, (1 << 21) + 3), (9, (1 << 20) - 9), (9, (1 << 20) + 1),
                                      (40, (1 << 21) + 3)])
def test_long_contexts_with_a_rising_maximum(n_new, kv, e4m3):
    """Pages named many times, in the order of the first row's largest score, so that its maximum moves by small steps
    over the whole context."""
    H, G, d, ps = 2, 2, 128, 64
    g = torch.Generator().manual_seed(kv % 1000 + n_new)
    q = torch.randn(n_new, H * G, d, generator=g).to(torch.bfloat16)
    k, v = (torch.randn(300, ps, H, d, generator=g) * s for s in (2.0, 1.0))
    kw = {}
    if e4m3:
        kw = dict(k_scale=torch.full((H,), 0.02), v_scale=torch.full((H,), 0.011))
        kc, vc = ((x / s[0]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn) for x, s in zip((k, v), kw.values()))
        k, v = (c.float() * s[0] for c, s in zip((kc, vc), kw.values()))
    else:
        kc, vc = k.to(torch.bfloat16), v.to(torch.bfloat16)
        k, v = kc, vc
    peak = (k[:, :, 0].double() @ q[0, 0].double()).amax(1)
    order = torch.argsort(peak).to(torch.int32)
    pages = kv // ps + 1
    row = order[torch.arange(pages) * 300 // pages]
    got, got_lse = b2.attn_paged_fwd(q.cuda(), kc.cuda(), vc.cuda(), row.cuda()[None], ints([0, n_new]), ints([kv]),
                                     max_seqlen_q=n_new, causal=False, return_lse=True,
                                     **{n: x.cuda() for n, x in kw.items()})
    assert b2.check() == 0
    half = 2.0 ** -11 if e4m3 else 2.0 ** -8
    for h in range(H * G):
        hk = h // G
        o, lse, a = repeated(q[:, h], k[:, :, hk], v[:, :, hk], row, kv, d ** -0.5)
        reach = (q[:, h].double().abs() @ k[:, :, hk].flatten(0, 1).double().abs().T).amax(1) * d ** -0.5
        score = ((d + 2) * 2.0 ** -24 * reach + 2.0 ** -22)[:, None]
        bound = a * (half + 2 * score + kv / 16 * 2.0 ** -23) + o.abs() * 2.0 ** -8 + a.amax(1, keepdim=True).clamp(min=1.0) * (
            lost(n_new, G, kv) if e4m3 else 0.0)
        assert bool(((got[:, h].double().cpu() - o).abs() <= bound).all()), h
        assert bool(((got_lse[h].double().cpu() - lse).abs() <= score[:, 0] + 2.0 ** -22 * (2 + lse.abs()) + kv / 64 * 2.0 ** -24).all())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n_new,kv", [(1, 3000), (2, 700), (40, 3000)])
@pytest.mark.parametrize("power", [14, 16, 17, 18, 19])
def test_very_large_scores_give_the_largest_ones_value(n_new, kv, e4m3, power):
    """Scores of up to 2^25 binades, where fp32 numbers are 0.125 to 4 apart: rows whose largest score stands out by more
    than its rounding give that key's value."""
    p = make([n_new], [kv], 8, 2, 128, 16, e4m3, seed=80 + power)
    scale = 2.0 ** power
    o, _ = run(p, max_seqlen_q=n_new, softmax_scale=scale)
    want, _, _, reach = attention(p, softmax_scale=scale)
    row = p.table[0].long()
    j = torch.arange(kv)
    hits = 0
    for h in range(8):
        k, v = (c[row[j // 16], j % 16, h // 4].double() for c in (p.k_cache, p.v_cache))
        if e4m3:
            k, v = k * p.k_scale[h // 4].double(), v * p.v_scale[h // 4].double()
        x = p.q[:, h].double() @ k.T * scale
        x[j[None, :] > kv - n_new + torch.arange(n_new)[:, None]] = -math.inf
        top, at = x.topk(2, 1)
        clear = top[:, 0] - top[:, 1] > 40 + 2 * (128 + 2) * 2.0 ** -24 * reach[h]  # the score's error, see check_attention
        hits += int(clear.sum())
        # one half step of the probability's type and one of the output's
        lim = v[at[:, 0]].abs() * (2.0 ** -8 + (2.0 ** -11 if e4m3 else 2.0 ** -8)) + 1e-9
        assert bool(((o[:, h].double().cpu() - v[at[:, 0]]).abs() <= lim)[clear].all())
    assert hits >= 4 * n_new and not bool(o.isnan().any())


def test_falling_maxima_of_very_large_scores():
    """Scores of 2^26.9 binades that fall by one or two steps of fp32 a key block: the first block's keys have all the
    weight, and what has been summed up is not scaled up block by block. As many requests as SMs, so that none is split."""
    n, blocks, B = 40, 10, torch.cuda.get_device_properties(0).multi_processor_count
    k, v = torch.zeros(blocks * 8, 16, 1, 128), torch.full((blocks * 8, 16, 1, 128), -1.0)
    k[..., 0], v[:8] = 256.0, 1.0
    k[..., 1] = torch.arange(blocks - 1, -1, -1).repeat_interleave(8)[:, None, None]
    q = torch.zeros(B * n, 4, 128, dtype=torch.bfloat16, device="cuda")
    q[..., 0], q[..., 1] = 1.0, 2.0 ** -15
    one = torch.ones(1, device="cuda")
    o = b2.attn_paged_fwd(q, *(x.to(torch.float8_e4m3fn).cuda() for x in (k, v)),
                          torch.arange(blocks * 8, dtype=torch.int32, device="cuda").repeat(B, 1),
                          ints([n * i for i in range(B + 1)]), ints([blocks * 128] * B), max_seqlen_q=n, causal=False,
                          softmax_scale=2.0 ** 26.9 / 256 / math.log2(math.e), k_scale=one, v_scale=one)
    assert b2.check() == 0
    # the blocks behind the first have 2^-8 of its weight each at most, as far apart as fp32 numbers of this size are
    assert bool(((o.float() - 1).abs() <= 2 * 2.0 ** -7 + 2.0 ** -8).all())


# ------------------------------------------------------------------------------------------- as a server uses them

def dense(q, k, v, n_ctx):
    """64-bit causal attention of one request: q the last rows of a sequence of k, v."""
    nq, G = q.shape[0], q.shape[1] // k.shape[1]
    kk, vv = k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    x = torch.einsum("ihd,jhd->hij", q.double(), kk) / math.sqrt(q.shape[2])
    x.masked_fill_(torch.arange(k.shape[0])[None, :] > n_ctx + torch.arange(nq)[:, None], -math.inf)
    return torch.einsum("hij,jhd->ihd", torch.softmax(x, 2), vv)


@pytest.mark.parametrize("d_qk,e4m3", [(128, False), (128, True), (192, False)])
def test_serving_steps_together(d_qk, e4m3):
    """Prompts read in chunks, decoding, requests of different ages in one step: lengths -> slots and pages -> K and V
    appended -> attention, each step's output against dense attention of each request's whole history."""
    Hq, H, ps, B = 8, 2, 16, 4
    g = torch.Generator().manual_seed(d_qk + e4m3)
    plan = [[30, 17, 1, 0], [30, 1, 1, 0], [1, 1, 1, 90], [1, 3, 0, 1], [1, 1, 1, 1]]
    total = sum(sum(s) for s in plan)
    pages = total // ps + 2 * B
    dt = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kc, vc = (torch.full((pages, ps, H, d), math.nan, device="cuda").to(dt) for d in (d_qk, 128))
    scale = dict(k_scale=torch.full((H,), 0.011, device="cuda"), v_scale=torch.full((H,), 0.012, device="cuda")) if e4m3 else {}
    table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    free, head, ctx = torch.randperm(pages, generator=g).to(torch.int32).cuda(), ints([0]), ints([0] * B)
    history = [(torch.empty(0, H, d_qk), torch.empty(0, H, 128)) for _ in range(B)]
    for new in plan:
        T, pad = sum(new), 3
        q, k, v = (torch.randn(T + pad, h, d, generator=g).to(torch.bfloat16) for h, d in ((Hq, d_qk), (H, d_qk), (H, 128)))
        cu, kv, pos, slots, head = b2.paged_slots(table, ctx, ints(new), T + pad, ps, free_pages=free, free_head=head)
        o = b2.attn_paged_func(q.cuda(), k.cuda(), v.cuda(), kc, vc, table, cu, kv, slots, max_seqlen_q=max(new), **scale)
        assert b2.check() == 0
        t = 0
        for b, n in enumerate(new):
            stored = (k[t:t + n], v[t:t + n])
            if e4m3:
                stored = tuple(plain_codes(x, s.cpu()).float() * s.cpu()[:, None] for x, s in
                               zip(stored, (scale["k_scale"], scale["v_scale"])))
            old = history[b]
            history[b] = tuple(torch.cat([a, x.float()]) for a, x in zip(old, stored))
            if n:
                want = dense(q[t:t + n], *history[b], old[0].shape[0])
                spread = dense(q[t:t + n], history[b][0], history[b][1].abs(), old[0].shape[0])
                # the bounds of check_attention for scores of this size (|q| |k| / sqrt(d) below 32)
                lim = spread * (2.0 ** -8 + 2 * (d_qk * 32 * 2.0 ** -24 + 2.3e-4)) + want.abs() * 2.0 ** -8
                assert bool(((o[t:t + n].double().cpu() - want).abs() <= lim).all())
            t += n
        ctx = kv
    assert int(head) == sum(-(-sum(s[b] for s in plan) // ps) for b in range(B))


@pytest.mark.parametrize("max_q", [1, 24])
def test_captured_steps_replay_on_new_contents(max_q):
    """A padded step captured once -- slots, append, attention -- and replayed with other lengths, tables and values;
    two graphs with workspaces of their own replayed in turn."""
    Hq, H, d, ps, B, T = 8, 2, 128, 16, 5, 5 * max_q
    g = torch.Generator().manual_seed(max_q)
    pages, width = 80, 12
    mk = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    kc, vc = (torch.randn(pages, ps, H, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q, k, v = mk(T, Hq, d), mk(T, H, d), mk(T, H, d)
    table, ctx, new = torch.zeros(B, width, dtype=torch.int32, device="cuda"), ints([1] * B), ints([1] * B)
    q.zero_(), k.zero_(), v.zero_()
    graphs = []
    for _ in range(2):
        out = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(b2.attn_paged_workspace_bytes(T, max_q, Hq, H), dtype=torch.uint8, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            def step():
                cu, kv, pos, slots = b2.paged_slots(table, ctx, new, T, ps)
                b2.paged_append_kv(k, v, kc, vc, slots)
                b2.attn_paged_fwd(q, kc, vc, table, cu, kv, max_seqlen_q=max_q, out=out, workspace=ws)
                return cu, kv
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cu, kv = step()
        graphs.append((graph, out, cu, kv, ws))  # a captured call's buffers live as long as its graph
    for i in range(4):
        n_new = [min(max_q, (i + b) % (max_q + 1)) for b in range(B)]
        n_ctx = [(17 * (b + 1) * (i + 2)) % 150 for b in range(B)]
        order = torch.randperm(pages, generator=g)[: B * width].view(B, width).to(torch.int32)
        table.copy_(order)
        ctx.copy_(torch.tensor(n_ctx)), new.copy_(torch.tensor(n_new))
        for x in (q, k, v):
            x.copy_(torch.randn(*x.shape, generator=g).to(torch.bfloat16))
        graph, out, cu, kv, _ = graphs[i % 2]
        out.fill_(7.0)
        graph.replay()
        assert b2.check() == 0
        assert kv.tolist() == [a + c for a, c in zip(n_ctx, n_new)]
        p = Paged(q.cpu(), kc.cpu(), vc.cpu(), table.cpu(), cu.cpu(), kv.cpu(), None, None)
        check_attention(p, out)
        assert bool((out[sum(n_new):] == 7.0).all())
    for graph, *_ in graphs:
        graph.reset()


@pytest.mark.parametrize("n,max_q", [(1, 1), (40, 40)])
def test_other_streams_and_repeated_calls_give_the_same_bytes(n, max_q):
    p = make([n] * 6, [700 + 31 * i for i in range(6)], 32, 8, 128, 16, seed=30).cuda()
    ref = b2.attn_paged_fwd(*p.args(), max_seqlen_q=max_q, return_lse=True)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s in side * 3:  # overlapping calls, each with a workspace and an output of its own
        with torch.cuda.stream(s):
            outs.append(b2.attn_paged_fwd(*p.args(), max_seqlen_q=max_q, return_lse=True))
    outs.append(b2.attn_paged_fwd(*p.args(), max_seqlen_q=max_q, return_lse=True, stream=side[0]))
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    assert b2.check() == 0


def test_calls_do_not_wait_for_the_stream():
    p = make([1, 1], [100, 60], 8, 2, 128, 16, seed=31).cuda()
    k = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    args = ints([99, 59]), ints([1, 1])
    b2.paged_slots(p.table, *args, 2, 16)
    slots = ints([-1, -1])
    b2.attn_paged_func(p.q, k, k, p.k_cache, p.v_cache, p.table, p.cu, p.kv_lens, slots, max_seqlen_q=1)
    b2.attn_paged_fwd(*p.args())
    torch.cuda.synchronize()
    busy = torch.cuda.Event()
    torch.cuda._sleep(1_000_000_000)
    busy.record()
    b2.paged_slots(p.table, *args, 2, 16)
    b2.attn_paged_func(p.q, k, k, p.k_cache, p.v_cache, p.table, p.cu, p.kv_lens, slots, max_seqlen_q=1)
    b2.attn_paged_fwd(*p.args())
    assert not busy.query()
    assert b2.check() == 0


def owner(t):
    """Handle of the stream whose pool t's memory is in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("n,max_q", [(1, 1), (40, 40)])
def test_calls_on_streams_given_by_name_share_no_memory(n, max_q, raw):
    """stream= on two streams that are busy, with other inputs each, and memory taken and filled on the current stream
    as soon as a call has returned: workspaces and results are each call's own."""
    ps = [make([n] * 6, [900 + 31 * i for i in range(6)], 32, 8, 128, 16, seed=50 + i).cuda() for i in range(2)]
    want = [b2.attn_paged_fwd(*p.args(), max_seqlen_q=max_q, return_lse=True) for p in ps]
    size = b2.attn_paged_workspace_bytes(ps[0].q.shape[0], max_q, 32, 8)
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    got = []
    for _ in range(2):
        for s, p in zip(streams, ps):
            with torch.cuda.stream(s):
                torch.cuda._sleep(20_000_000)
            got.append(b2.attn_paged_fwd(*p.args(), max_seqlen_q=max_q, return_lse=True, stream=s.cuda_stream if raw else s))
            for like in (size, *(t.numel() * t.element_size() for t in got[-1])):
                torch.full((like,), 0x7f, dtype=torch.uint8, device="cuda")
    for s, (o, lse) in zip(streams * 2, got):
        assert owner(o) == owner(lse) == s.cuda_stream
    torch.cuda.synchronize()
    assert b2.check() == 0
    for (o, lse), (a, c) in zip(got, want * 2):
        assert torch.equal(o, a) and torch.equal(lse, c)


def test_slots_on_a_stream_given_by_name():
    lens = ints([5, 0, 16]), ints([1, 3, 20])
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    free, head = ints(list(range(50, 70))), ints([1])
    want = b2.paged_slots(table.clone(), *lens, 30, 16, free_pages=free, free_head=head)
    side, tables = torch.cuda.Stream(), [table.clone() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for t in tables:
        with torch.cuda.stream(side):
            torch.cuda._sleep(10_000_000)
        got.append(b2.paged_slots(t, *lens, 30, 16, free_pages=free, free_head=head, stream=side))
        torch.full((3 * 2 + 2 + 60,), 9, dtype=torch.int32, device="cuda")
        assert all(owner(x) == side.cuda_stream for x in got[-1])
    torch.cuda.synchronize()
    assert b2.check() == 0
    for r in got:
        assert all(torch.equal(a, c) for a, c in zip(r, want))


def test_the_default_stream_given_by_its_handle():
    """0 and 1 both name it; under another current stream it is a stream of its own."""
    p = make([1, 1], [100, 300], 8, 2, 128, 16, seed=52).cuda()
    want = b2.attn_paged_fwd(*p.args(), max_seqlen_q=1)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for handle in (0, 1):
            o = b2.attn_paged_fwd(*p.args(), max_seqlen_q=1, stream=handle)
            assert owner(o) == 0
            torch.cuda.synchronize()
            assert torch.equal(o, want)
    assert b2.check() == 0


@pytest.mark.parametrize("n,max_q", [(1, 8), (5, 8), (2, 100)])
def test_a_workspace_of_the_stated_size_serves_the_call_and_smaller_ones(n, max_q):
    p = make([n], [300], 32, 8, 128, 16, seed=71)
    size = b2.attn_paged_workspace_bytes(n, max_q, 32, 8)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    check_attention(p, *run(p, max_seqlen_q=max_q, workspace=ws))
    p = make([1], [300], 32, 8, 128, 16, seed=72)
    check_attention(p, *run(p, max_seqlen_q=1, workspace=ws))


def test_work_counted_by_the_bound_on_new_tokens():
    """4000 requests of a pair of row tiles each over tables of 2^26 rows: by max_seqlen_q their key blocks are below
    2^31; by the number of rows alone they would not be."""
    B, n, ps, G = 4000, 64, 1 << 20, 4
    kc = torch.ones(1, ps, 1, 128, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(B, 64, dtype=torch.int32, device="cuda")
    blocks = 64 * ps // 128 + 4
    assert B * blocks < 2 ** 31 <= (B * n // (2 * (128 // G)) + B) * blocks
    q = torch.zeros(B * n, G, 128, dtype=torch.bfloat16, device="cuda")
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    o = b2.attn_paged_fwd(q, kc, kc, table, cu, torch.full((B,), 100, dtype=torch.int32, device="cuda"), max_seqlen_q=n)
    assert b2.check() == 0 and bool((o == 1).all())
