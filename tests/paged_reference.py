"""Plain 64-bit forms of the paged-cache operators, and inputs for their tests.
Nothing here calls the library."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@dataclass
class Paged:
    """A paged cache with its requests, on the CPU."""
    q: torch.Tensor          # bf16 [total, Hq, d_qk]
    k_cache: torch.Tensor    # bf16 or e4m3 [pages, page_size, Hkv, d_qk]
    v_cache: torch.Tensor
    table: torch.Tensor      # int32 [B, width]
    cu: torch.Tensor         # int32 [B + 1]
    kv_lens: torch.Tensor    # int32 [B]
    k_scale: torch.Tensor | None
    v_scale: torch.Tensor | None

    def cuda(self):
        return Paged(**{n: t if t is None else t.cuda() for n, t in self.__dict__.items()})

    def args(self):
        return self.q, self.k_cache, self.v_cache, self.table, self.cu, self.kv_lens

    def scales(self):
        return {"k_scale": self.k_scale, "v_scale": self.v_scale}


def make(q_lens, kv_lens, Hq, Hkv, d_qk, page_size, e4m3=False, seed=0, pad_rows=0, spread=1.0, hole=float("nan")):
    """Requests with q_lens new tokens over kv_lens keys; cache rows that belong to no request hold `hole`, table
    entries behind a request's pages -1, pages are in random order."""
    g = torch.Generator().manual_seed(seed)
    B, d_v = len(q_lens), 128
    need = [-(-n // page_size) for n in kv_lens]
    width = max(need) + 2
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    T = sum(q_lens) + pad_rows
    q = (torch.randn(T, Hq, d_qk, generator=g) * spread).to(torch.bfloat16)
    used = torch.zeros(pages, page_size, dtype=torch.bool)
    for b, n in enumerate(kv_lens):
        for j in range(need[b]):
            used[table[b, j], : min(page_size, n - j * page_size)] = True
    out = []
    for d in (d_qk, d_v):
        x = torch.randn(pages, page_size, Hkv, d, generator=g)
        scale = None
        if e4m3:
            scale = x.abs().amax((0, 1, 3)) / 448.0
            x = (x / scale[:, None]).clamp(-448.0, 448.0)
        x[~used] = hole
        out += [x.to(torch.float8_e4m3fn if e4m3 else torch.bfloat16), scale]
    cu = torch.tensor([0] + list(q_lens)).cumsum(0).to(torch.int32)
    return Paged(q, out[0], out[2], table, cu, torch.tensor(kv_lens, dtype=torch.int32), out[1], out[3])


def attention(p: Paged, causal=True, softmax_scale=None):
    """(o, lse, spread, reach) in 64 bits: the result, sum_j p_j |v_j| / l (what a relative error of the
    probabilities is multiplied with), and the largest scaled sum_d |q_d k_d| of each row. Rows of no request: NaN."""
    T, Hq, d = p.q.shape
    Hkv, ps = p.k_cache.shape[2], p.k_cache.shape[1]
    G, s = Hq // Hkv, softmax_scale or 1.0 / math.sqrt(d)
    o = torch.full((T, Hq, 128), math.nan, dtype=torch.float64)
    a, lse, reach = o.clone(), torch.full((Hq, T), math.nan, dtype=torch.float64), torch.zeros(Hq, T, dtype=torch.float64)
    for b in range(p.kv_lens.numel()):
        t0, t1, n = int(p.cu[b]), int(p.cu[b + 1]), int(p.kv_lens[b])
        nq = t1 - t0
        if nq == 0:
            continue
        j = torch.arange(n)
        pages = p.table[b].long()[j // ps]
        for h in range(Hkv):
            k, v = p.k_cache[pages, j % ps, h].double(), p.v_cache[pages, j % ps, h].double()
            if p.k_scale is not None:
                k, v = k * p.k_scale[h].double(), v * p.v_scale[h].double()
            for hq in range(h * G, h * G + G):
                q = p.q[t0:t1, hq].double()
                x = q @ k.T * s
                if causal:
                    x[j[None, :] > n - nq + torch.arange(nq)[:, None]] = -math.inf
                m = x.amax(1, keepdim=True) if n else torch.full((nq, 1), -math.inf, dtype=torch.float64)
                e = torch.exp(x - torch.where(m.isfinite(), m, 0.0))
                l = e.sum(1, keepdim=True)
                w = torch.where(l > 0, e / l, 0.0)
                o[t0:t1, hq], a[t0:t1, hq] = w @ v, w @ v.abs()
                lse[hq, t0:t1] = (m + l.log())[:, 0]
                reach[hq, t0:t1] = (q.abs() @ k.abs().T).amax(1) * s if n else 0.0
    return o, lse, a, reach


def check_attention(p: Paged, got, lse=None, causal=True, softmax_scale=None):
    """Elementwise bounds. A probability carries the half step of its 16-bit type and an exponential of fp32 scores:
    an fp32 sum of d products is off by at most (d + 2) 2^-24 sum |q_d k_d|, which is a relative error of the
    probability; so is the base-2 exponential's 2^-22. Each probability enters numerator and sum, and the output is
    rounded to bf16 once."""
    o, ref_lse, a, reach = attention(p, causal, softmax_scale)
    d = p.q.shape[2]
    half = HALF_STEP[torch.float16 if p.k_scale is not None else torch.bfloat16]
    score = (d + 2) * 2.0 ** -24 * reach + 2.0 ** -22      # [Hq, T]
    # fp16 probabilities below 2^-14 are off by 2^-25 at most, beside a largest one of at least 1
    tiny = p.kv_lens.max().item() * 2.0 ** -25 * (p.k_scale is not None)
    bound = a * (half + 2 * score.T[..., None]) + a.amax(-1, keepdim=True).clamp(min=1.0) * tiny + o.abs() * 2.0 ** -8 + 1e-30
    real = ~o.isnan()
    got = got.double().cpu()
    assert not got[real].isnan().any()
    over = ((got - o).abs() / bound)[real]
    assert over.numel() == 0 or over.max() <= 1.0, f"error {over.max():.3g} times its bound"
    if lse is not None:
        lse = lse.double().cpu()
        real = ~ref_lse.isnan()
        none = real & (ref_lse == -math.inf)
        assert (lse[none] == -math.inf).all()
        some = real & ~none
        # the scores' error and an fp32 logarithm and sum of numbers of the result's size
        lim = score + 2.0 ** -22 * (2 + ref_lse.abs())
        assert ((lse - ref_lse).abs()[some] <= lim[some]).all(), (lse - ref_lse).abs()[some].max()
