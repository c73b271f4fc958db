"""Plain float64 references of the attention-side operators and the 4-bit projection (CPU torch, no kernels)."""

from __future__ import annotations

import math

import numpy as np
import torch

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step, relative
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def frequencies(rot, theta, sections, layout):
    """(f_j, axis_j), straight from the definition."""
    half = rot // 2
    sec = list(sections) if sections is not None else [half]
    f, ax = [], []
    for j in range(half):
        if layout == "interleaved":
            a = j % 3
            a = a if a < len(sec) and j < 3 * sec[a] else 0
            e = j / half
        else:
            a = next(i for i in range(len(sec)) if j < sum(sec[:i + 1]))
            e = (j - sum(sec[:a])) / sec[a] if layout == "per_axis" else j / half
        f.append(theta ** -e)
        ax.append(a)
    return np.array(f), np.array(ax, int)


def cos_sin(positions, f, ax):
    """fp32 cosine and sine [T, half] of float64 angles."""
    ang = np.asarray(positions, np.float64)[ax].T * f
    return torch.from_numpy(np.cos(ang)).float(), torch.from_numpy(np.sin(ang)).float()


def rotate64(x, cs):
    """The rotation in float64 with the given fp32 cosines and sines."""
    c, s = (t.double().unsqueeze(1) for t in cs)
    h = c.shape[-1]
    x = x.double()
    a, b = x[..., :h], x[..., h:2 * h]
    return torch.cat((a * c - b * s, b * c + a * s, x[..., 2 * h:]), -1)


def rotate32(x, cs):
    """The rotation with every product and sum rounded to fp32."""
    c, s = (t.unsqueeze(1) for t in cs)
    h = c.shape[-1]
    x = x.float()
    a, b = x[..., :h], x[..., h:2 * h]
    return torch.cat((a * c - b * s, b * c + a * s, x[..., 2 * h:]), -1)


def quantise(x, group):
    """(codes, scale, bias, values) of fp32 x [..., D], as the header defines them; scale and bias as float64."""
    y = x.float().unflatten(-1, (-1, group))
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    s = ((hi - lo) * torch.tensor(1.0 / 15.0, dtype=torch.float32)).bfloat16().float()
    b = lo.bfloat16().float()
    c = torch.where(s > 0, ((y - b) / s).round().clamp(0, 15), torch.zeros_like(y))
    bad = ~(torch.isfinite(hi - lo) & torch.isfinite(b))
    s, b = s.masked_fill(bad, math.nan), b.masked_fill(bad, math.nan)
    v = s.double() * c.double() + b.double()
    return c.flatten(-2), s.squeeze(-1).double(), b.squeeze(-1).double(), v.flatten(-2)


def v_group(D):
    return min(D, 128)


def attention64(q, k, v, scale, new):
    """One sequence: q [new, Hq, D], k and v [len, Hkv, D] float64 (the cache's values) -> o, lse."""
    n, hq, d = q.shape
    length, hkv, _ = k.shape
    o, lse = torch.zeros(n, hq, d, dtype=torch.float64), torch.full((n, hq), -math.inf, dtype=torch.float64)
    for i in range(n):
        seen = length - new + i + 1
        if seen <= 0:
            continue
        for h in range(hq):
            kh = h // (hq // hkv)
            s = (k[:seen, kh] @ q[i, h].double()) * scale
            lse[i, h] = torch.logsumexp(s, 0)
            o[i, h] = torch.softmax(s, 0) @ v[:seen, kh]
    return o, lse


def attention_bound(q, k_parts, v_parts, o, scale, new, io, long=False):
    """What rounding allows: (|o error|, |lse error|) per query and head.

    Scores: products of the operands are exact, sums lose at most 2^-23 of the running magnitude a step; a warp's chain
    of a score has fewer than 8 steps that see the whole sum, so 2^-20 of the sum of magnitudes (codes around 8, the bias
    moved there) covers them.  A score off by e changes p by a factor within e^{+-2e}.  Values are codes around 8; sums as
    for scores.  The output rounds once.

    fp32 io: queries and p times the value's scale go in three bf16 parts, 2^-20 covers them.
    bf16 io: queries are fp16 between 2^7 and 2^8 at their row's largest, so that the half step below fp16's normal
    numbers, 2^-25, is 2^-32 of it.  p times the scale is off by half a step of fp16, 2^-11, or, where it is under 2^-14,
    by 2^-25 where the largest scale stands at 2^3 at least: 2^-25 of the largest value for each key.
    long: the long row tiles (bf16 io).  Key products are exact in fp16 too; the moved bias and the sums of the query's
    groups go in two parts of 11 bits each, 2^-22 of either, within the 2^-20.  Keys and values have their largest so far
    between 2^7 and 2^12: half a step below the normal numbers is 2^-32 of the largest key.  Values and probabilities are
    off by half a step of fp16, 2^-11 each; a probability under 2^-14 is off by 2^-25 where the largest is 1 at least."""
    n, hq, d = q.shape
    (_, ks, kb, _), (_, vs, vb, _) = k_parts, v_parts
    length, hkv = ks.shape[:2]
    k_mag = (8 * ks + (kb + 8 * ks).abs()).repeat_interleave(64, -1)
    v_mag = (8 * vs + (vb + 8 * vs).abs()).amax(-1)  # [length, hkv]
    eo, el = torch.zeros(n, hq, dtype=torch.float64), torch.zeros(n, hq, dtype=torch.float64)
    for i in range(n):
        seen = length - new + i + 1
        if seen <= 0:
            continue
        for h in range(hq):
            kh = h // (hq // hkv)
            qa = q[i, h].double().abs()
            ds = abs(scale) * 2.0 ** -20 * (k_mag[:seen, kh] @ qa).max()
            if io == "bf16":
                ds = ds + abs(scale) * 2.0 ** -32 * (qa.max() * k_mag[:seen, kh].sum(-1).max() + k_mag[:, kh].max() * qa.sum())
            el[i, h] = ds
            eo[i, h] = (2 * ds + 2 * 2.0 ** -20) * v_mag[:seen, kh].max()
            if io == "bf16":
                eo[i, h] += ((2 if long else 1) * 2.0 ** -11 + 2.0 ** -32 + seen * 2.0 ** -25) * v_mag[:, kh].max()
    return U[io] * o.abs() + eo.unsqueeze(-1), el


class Case:
    """A packed batch over a shuffled paged cache, on the GPU, with its float64 twin on the CPU."""

    def __init__(self, new, ctx, hq, hkv, d, page, io, seed=0, spare=2, fill=0xFF, outlier=True):
        import linear_attention_recurrence_deltanet_b200 as gdn
        g = torch.Generator().manual_seed(seed)
        self.new, self.lens = list(new), [a + b for a, b in zip(new, ctx)]
        self.hq, self.hkv, self.d, self.page, self.io = hq, hkv, d, page, io
        self.N, self.T = len(new), sum(new)
        self.cfg = gdn.make_attn_config(hq, hkv, d, page_size=page, io_dtype=io)
        self.scale = d ** -0.5
        self.cu = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        need = [-(-n // page) for n in self.lens]
        self.width, self.pages = max(need + [1]), sum(need) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        self.table = torch.full((self.N, self.width), -7, dtype=torch.int32)  # ids past a sequence's end are never read
        for n, m in enumerate(need):
            for j in range(m):
                self.table[n, j] = order.pop()
        self.spare = order
        self.q = torch.randn(self.T, hq, d, generator=g).to(DT[io])
        self.k = [torch.randn(n, hkv, d, generator=g) for n in self.lens]
        self.v = [torch.randn(n, hkv, d, generator=g).to(DT[io]) for n in self.lens]
        for t in self.k:
            if outlier and t.numel():
                t[..., 3::29] *= 5.0
        self.k = [t.to(DT[io]) for t in self.k]
        # every byte of the pool outside the stored tokens is poison: as bf16 scales, NaN
        self.pool = torch.full((self.pages, gdn.kv_page_bytes(self.cfg)), fill, dtype=torch.uint8, device="cuda")
        self.fill_value = fill
        self.d_table, self.d_lens = self.table.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.d_cu, self.d_q = torch.from_numpy(self.cu).cuda(), self.q.cuda()
        self.gdn = gdn

    def fill(self):
        """The whole context into the cache, unrotated, in one append."""
        cu = np.concatenate(([0], np.cumsum(self.lens))).astype(np.int32)
        k, v = torch.cat(self.k).cuda(), torch.cat(self.v).cuda()
        self.gdn.kv_append(self.cfg, None, None, k, v, None, torch.from_numpy(cu).cuda(), cu, self.d_lens, self.pool,
                           self.d_table, None)
        return self

    def outputs(self):
        o = torch.full((self.T, self.hq, self.d), 7.0, dtype=DT[self.io], device="cuda")
        lse = torch.full((self.T, self.hq), 7.0, device="cuda")
        ws = torch.full((max(256, self.gdn.attention_workspace_size(self.cfg, self.T, self.N)),), 0xFF,
                        dtype=torch.uint8, device="cuda")
        return o, lse, ws

    def attention(self, stream=None):
        o, lse, ws = self.outputs()
        self.gdn.attention(self.cfg, self.d_q, self.d_cu, self.cu, self.d_lens, self.pool, self.d_table, o, lse, ws,
                           stream=stream)
        return o, lse

    def check(self, o, lse, skip=()):
        o, lse = o.cpu(), lse.cpu()
        assert torch.isfinite(o).all()
        long = self.io == "bf16" and max(self.new) * (self.hq // self.hkv) > (64 if self.d <= 128 else 128)
        for n in range(self.N):
            a, b = int(self.cu[n]), int(self.cu[n + 1])
            if a == b or n in skip:
                continue
            kp, vp = quantise(self.k[n], 64), quantise(self.v[n], v_group(self.d))
            ref, rl = attention64(self.q[a:b], kp[3], vp[3], self.scale, b - a)
            eo, el = attention_bound(self.q[a:b], kp, vp, ref, self.scale, b - a, self.io, long)
            off = (o[a:b].double() - ref).abs() - eo
            assert off.max() <= 0, f"sequence {n}: o past its bound by {off.max():.3g}"
            seen = torch.isfinite(rl)
            assert torch.equal(torch.isfinite(lse[a:b]), seen) and (lse[a:b][~seen] == -math.inf).all()
            dl = (lse[a:b].double() - rl).abs()[seen] - el[seen] - 2.0 ** -21 * (1 + rl.abs()[seen])
            assert dl.numel() == 0 or dl.max() <= 0, f"sequence {n}: lse past its bound by {dl.max():.3g}"
            assert (o[a:b][~seen] == 0).all()
