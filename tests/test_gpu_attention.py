"""Rotary positions, the 4-bit paged cache and attention over it, through the public calls against float64."""

import math

import numpy as np
import pytest
import torch

import linear_attention_recurrence_deltanet_b200 as gdn
from attn_ref import DT, U, Case, cos_sin, frequencies, quantise, rotate32, rotate64, v_group

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gdn.lib()
    yield
    assert gdn.device_status() == 0


# --------------------------------------------------------------------------------------------------------- rope
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,D,rot,sections,layout", [
    (1, 1, 64, 64, None, "sections"), (5, 24, 128, 64, None, "sections"), (33, 3, 128, 128, [24, 20, 20], "interleaved"),
    (7, 5, 72, 72, [12, 12, 12], "per_axis"), (6, 2, 80, 60, [10, 20], "per_axis"), (9, 2, 256, 256, [64, 32, 32], "sections"),
    (3, 7, 128, 36, [8, 5, 5], "interleaved"), (4, 2, 8, 2, None, "sections"), (2, 2, 64, 0, None, "sections"),
    (2500, 2, 64, 64, [16, 8, 8], "interleaved"),
])
def test_rope_forward_and_inverse(io, T, H, D, rot, sections, layout):
    g = torch.Generator().manual_seed(T * 7 + D)
    axes = len(sections) if sections else 1
    x = torch.randn(T, H, D, generator=g).to(DT[io])
    pos = torch.randint(-5, 262144, (axes, T), generator=g, dtype=torch.int32)
    pos[:, 0] = 2 ** 31 - 1
    plan = gdn.rope_plan(rot, 1e7, sections=sections, layout=layout)
    f, ax = frequencies(rot, 1e7, sections, layout)
    cs = cos_sin(pos.numpy(), f, ax) if rot else (torch.zeros(T, 0), torch.zeros(T, 0))
    # positions near 2^31 in float64: angle error 2^31 * 2^-53, far below an fp32 step of the cosine
    wide = torch.full((T, H + 2, D), 3.0, dtype=DT[io], device="cuda")
    wide[:, 1:H + 1] = x.cuda()
    out = torch.full((T, H, D), 9.0, dtype=DT[io], device="cuda")
    gdn.rope(plan, wide[:, 1:H + 1], pos.cuda(), out)
    ref = rotate64(x, cs)
    # three fp32 roundings of the products and the sum, a step of cosine and sine, one final rounding
    pair = x.double().abs()
    mag = torch.cat((pair[..., :rot // 2] + pair[..., rot // 2:rot],) * 2 + (pair[..., rot:],), -1)
    tol = U[io] * ref.abs() + 6 * 2.0 ** -24 * mag
    assert ((out.cpu().double() - ref).abs() <= tol).all()
    assert torch.equal(out.cpu()[..., rot:], x[..., rot:])
    # in place, inverse: rotates back within the two roundings
    gdn.rope(plan, out, pos.cuda(), out, inverse=True)
    back = rotate64(x, cs)
    tol2 = 2 * U[io] * mag + 12 * 2.0 ** -24 * mag
    assert ((out.cpu().double() - x.double()).abs() <= tol2 + U[io] * back.abs().max() * 0).all()


def test_rope_inverse_is_the_gradient():
    """sum(w * rope(x)) has the gradient rope^-1(w), by the formula and by differences."""
    T, H, D, rot = 3, 2, 64, 64
    g = torch.Generator().manual_seed(3)
    x, w = torch.randn(T, H, D, generator=g).cuda(), torch.randn(T, H, D, generator=g).cuda()
    pos = torch.tensor([[0, 3, 100], [5, 2, 77]], dtype=torch.int32).cuda()
    plan = gdn.rope_plan(rot, 1e4, sections=[20, 12], layout="interleaved")
    grad = torch.empty_like(w)
    gdn.rope(plan, w, pos, grad, inverse=True)
    y0, y1 = torch.empty_like(x), torch.empty_like(x)
    for i in ((0, 0, 0), (1, 1, 37), (2, 0, 63)):
        e = torch.zeros_like(x)
        e[i] = 0.5
        gdn.rope(plan, x + e, pos, y1)
        gdn.rope(plan, x - e, pos, y0)
        num = ((w.double() * (y1.double() - y0.double())).sum()).item()
        # linear in x: the difference is exact up to 128 rounded terms
        assert abs(num - grad[i].item()) <= 128 * 6 * 2.0 ** -24 * 4


def test_rope_custom_frequencies_and_strided_out():
    T, H, D = 6, 2, 64
    f = np.linspace(1.0, 0.01, 16)
    plan = gdn.rope_plan(32, inv_freq=f)
    x = torch.randn(T, H, D, generator=torch.Generator().manual_seed(1))
    pos = torch.arange(T, dtype=torch.int32)
    buf = torch.full((T, H + 1, D), 5.0, device="cuda")
    gdn.rope(plan, x.cuda(), pos.cuda(), buf[:, 1:])
    ref = rotate64(x, cos_sin(pos.view(1, -1).numpy(), f, np.zeros(16, int)))
    assert ((buf[:, 1:].cpu().double() - ref).abs() <= 8 * 2.0 ** -24 * (1 + ref.abs()) * 4).all()
    assert (buf[:, 0] == 5.0).all()


# ------------------------------------------------------------------------------------------------- append, read
APPEND = [
    # new tokens, context, Hq, Hkv, D, page, rot, sections, layout
    ([1], [0], 4, 1, 64, 16, 32, None, "sections"),
    ([1, 1, 1, 1], [0, 15, 16, 200], 24, 2, 128, 64, 64, None, "sections"),
    ([5, 0, 33, 1], [11, 3, 0, 47], 6, 2, 128, 48, 128, [24, 20, 20], "interleaved"),
    ([17, 70], [0, 31], 6, 3, 64, 32, 60, [10, 10, 10], "per_axis"),
    ([40, 3], [1, 16], 2, 2, 256, 16, 256, None, "sections"),
    ([9], [4], 2, 1, 256, 32, 36, [9, 9], "sections"),
    ([3000], [100], 3, 1, 64, 128, 64, None, "sections"),
]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("new,ctx,hq,hkv,d,page,rot,sections,layout", APPEND)
def test_append_then_read(io, new, ctx, hq, hkv, d, page, rot, sections, layout):
    c = Case(new, ctx, hq, hkv, d, page, io, seed=len(new) + d)
    axes = len(sections) if sections else 1
    g = torch.Generator().manual_seed(9)
    T = c.T
    rows = torch.randn(T, hq + 2 * hkv, d, generator=g)
    rows[:, hq:hq + hkv, 2::31] *= 6.0
    rows = rows.to(DT[io])
    pos = torch.randint(0, 70000, (axes, T), generator=g, dtype=torch.int32)
    plan = gdn.rope_plan(rot, 1e6, sections=sections, layout=layout)
    dev = rows.cuda()
    q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]  # slices of a projection's rows
    q_out = torch.full((T, hq, d), 4.0, dtype=DT[io], device="cuda")
    before = c.pool.clone()
    gdn.kv_append(c.cfg, plan, q, k, v, pos.cuda(), c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, q_out)
    k_out, v_out = (torch.full((T, hkv, d), 4.0, dtype=DT[io], device="cuda") for _ in range(2))
    gdn.kv_read(c.cfg, c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, k_out, v_out)
    f, ax = frequencies(rot, 1e6, sections, layout)
    cs = cos_sin(pos.numpy(), f, ax)
    cpu = rows
    ref = rotate64(cpu[:, :hq], cs)
    a = cpu[:, :hq].double().abs()
    mag = torch.cat((a[..., :rot // 2] + a[..., rot // 2:rot],) * 2 + (a[..., rot:],), -1)
    assert ((q_out.cpu().double() - ref).abs() <= U[io] * ref.abs() + 6 * 2.0 ** -24 * mag).all()
    # values: every step is exactly rounded, so they are the definition's bits
    _, _, _, vv = quantise(cpu[:, hq + hkv:], v_group(d))
    assert torch.equal(v_out.cpu(), vv.to(DT[io]))
    # keys: the same, but for cosines whose fp32 rounding sits on a border of the float64 ones
    kr = rotate32(cpu[:, hq:hq + hkv], cs)
    _, ks, _, kv = quantise(kr, 64)
    step = ks.repeat_interleave(64, -1)
    far = (k_out.cpu().double() - kv.to(DT[io]).double()).abs()
    assert (far <= 1.02 * step + 2 * U[io] * kv.abs() + 2.0 ** -7 * kv.abs()).all()
    assert (far > 0).double().mean() <= 1e-3
    # nothing else in the pool changed: clear what the call's tokens occupy in both copies
    mask = touched(c)
    assert torch.equal(c.pool[~mask], before[~mask])
    # appending again is idempotent
    again = c.pool.clone()
    gdn.kv_append(c.cfg, plan, q, k, v, pos.cuda(), c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, q_out)
    assert torch.equal(again, c.pool)


def touched(c):
    """Bytes of the pool that the call's tokens own, from the documented page layout."""
    d, gk, gv = c.d, c.d // 64, c.d // v_group(c.d)
    tile = 16 * (d + 4 * (gk + gv))
    m = torch.zeros(c.pool.shape, dtype=torch.bool)
    for n in range(c.N):
        for p in range(c.lens[n] - c.new[n], c.lens[n]):
            pg, r = int(c.table[n, p // c.page]), p % 16
            vr = (r & 8) | ((r & 1) << 2) | ((r >> 1) & 3)
            for h in range(c.hkv):
                base = (h * (c.page // 16) + p % c.page // 16) * tile
                for b in range(d // 64):
                    m[pg, base + b * 512 + r * 32:base + b * 512 + r * 32 + 32] = True
                    o = base + 16 * d // 2 + b * 512 + vr * 32
                    m[pg, o:o + 32] = True
                for s in range(gk + gv):
                    o = base + 16 * d + s * 64 + r * 4
                    m[pg, o:o + 4] = True
    return m.cuda()


def test_append_in_place_queries_and_cache_positions():
    """q_out may be q; positions None rotates by the cache position."""
    c = Case([3, 2], [10, 0], 4, 2, 128, 16, "f32", seed=5)
    plan = gdn.rope_plan(128, 1e4)
    k, v = torch.randn(5, 2, 128).cuda(), torch.randn(5, 2, 128).cuda()
    q = c.d_q.clone()
    gdn.kv_append(c.cfg, plan, q, k, v, None, c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, q)
    f, ax = frequencies(128, 1e4, None, "sections")
    ref = rotate64(c.q, cos_sin(np.array([[10, 11, 12, 0, 1]]), f, ax))
    assert ((q.cpu().double() - ref).abs() <= 2.0 ** -24 * ref.abs() + 12 * 2.0 ** -24 * 5).all()


def test_append_constant_extreme_and_non_finite_groups():
    c = Case([8], [0], 1, 1, 128, 16, "f32", seed=6)
    k = torch.randn(8, 1, 128)
    k[0] = 0.0
    k[1] = 2.5
    k[2, 0, 5] = math.inf
    k[3, 0, 70] = math.nan
    k[4] *= 1e30
    k[5] *= 1e-40  # subnormals
    k[6, 0, 0], k[6, 0, 1] = 3e38, -3e38  # a range past fp32
    k[7, 0, :64] = -math.inf
    v = k.flip(-1).contiguous()
    gdn.kv_append(c.cfg, None, None, k.cuda(), v.cuda(), None, c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, None)
    ko, vo = torch.empty(8, 1, 128, device="cuda"), torch.empty(8, 1, 128, device="cuda")
    gdn.kv_read(c.cfg, c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, ko, vo)
    for got, x, gr in ((ko.cpu(), k, 64), (vo.cpu(), v, 128)):
        want = quantise(x, gr)[3].float()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(), want.nan_to_num())
    assert torch.isnan(ko[2, 0, :64]).all() and torch.isfinite(ko[2, 0, 64:]).all()


def test_append_padding_rows_and_bad_pages():
    c = Case([1, 1, 1], [4, 0, 8], 2, 1, 64, 16, "bf16", seed=8)
    c.d_lens[1] = 0  # a padding row: nothing to store
    k, v = torch.randn(3, 1, 64).bfloat16().cuda(), torch.randn(3, 1, 64).bfloat16().cuda()
    before = c.pool.clone()
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    gdn.kv_append(c.cfg, None, None, k, v, None, c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, None)
    assert gdn.device_status() == 0
    page1 = int(c.table[1, 0])
    assert torch.equal(c.pool[page1], before[page1])
    gdn.kv_read(c.cfg, c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, ko, vo)
    assert (ko[1] == 0).all() and (vo[1] == 0).all() and (ko[0] != 0).any()
    assert gdn.device_status() == 0
    # a page id outside the pool, and a length past the table's row: skipped and reported
    for bad in ("id", "len"):
        t, lens = c.d_table.clone(), c.d_lens.clone()
        if bad == "id":
            t[2, 0] = c.pages
        else:
            lens[2] = c.width * c.page + 1
        before = c.pool.clone()
        gdn.kv_append(c.cfg, None, None, k, v, None, c.d_cu, c.cu, lens, c.pool, t, None)
        assert gdn.device_status() & 0xFF == 4
        page2 = int(c.table[2, 0])
        assert torch.equal(c.pool[page2], before[page2])
        gdn.kv_read(c.cfg, c.d_cu, c.cu, lens, c.pool, t, ko, vo)
        assert gdn.device_status() & 0xFF == 4 and (ko[2] == 0).all()


# ---------------------------------------------------------------------------------------------------- attention
ATTN = [
    # new, ctx, Hq, Hkv, D, page
    ([1], [0], 1, 1, 64, 16),
    ([1], [1], 8, 1, 128, 16),
    ([1, 1, 1, 1, 1], [0, 14, 15, 16, 63], 24, 2, 128, 64),
    ([1, 1], [777, 130], 16, 2, 256, 32),
    ([1], [2500], 24, 2, 128, 64),
    ([1, 1, 1], [1300, 5, 90], 32, 8, 128, 48),
    ([1, 1], [300, 40], 12, 12, 64, 128),
    ([1, 1], [300, 700], 40, 2, 64, 16),
    ([4, 4, 2], [100, 0, 333], 16, 2, 256, 16),
    ([3, 4], [29, 61], 6, 2, 128, 64),
    ([4], [1000], 24, 2, 128, 64),
    ([0, 7, 0, 1], [3, 20, 0, 0], 6, 3, 64, 32),
    ([50, 1, 19], [0, 200, 64], 6, 1, 128, 64),
    ([130], [70], 4, 2, 64, 16),
    ([37], [150], 6, 2, 256, 64),
    ([129, 65], [0, 31], 3, 1, 128, 48),
    ([300], [212], 2, 1, 128, 64),
    ([1] * 70, list(range(0, 140, 2)), 2, 1, 64, 16),
]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("new,ctx,hq,hkv,d,page", ATTN)
def test_attention_against_float64(io, new, ctx, hq, hkv, d, page):
    c = Case(new, ctx, hq, hkv, d, page, io, seed=hq + d + len(new)).fill()
    o, lse = c.attention()
    c.check(o, lse)
    o2, lse2 = c.attention()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)  # bit-identical on repetition


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attention_rows_that_see_nothing(io):
    """kv_lens 0 (padding) and fewer cached tokens than queries: the rows before the cache see nothing."""
    c = Case([1, 4, 40], [0, 0, 0], 6, 2, 128, 16, io, seed=2).fill()
    c.d_lens[0], c.d_lens[1], c.d_lens[2] = 0, 2, 25
    c.lens = [0, 2, 25]
    c.k, c.v = [t[:n] for t, n in zip(c.k, c.lens)], [t[:n] for t, n in zip(c.v, c.lens)]
    o, lse = c.attention()
    c.check(o, lse)
    assert (o[:3] == 0).all() and (lse[:3] == -math.inf).all() and (o[5:20] == 0).all()
    assert gdn.device_status() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_attention_bad_pages_are_reported_and_skipped(new):
    c = Case([new, new], [100, 60], 6, 2, 128, 16, "bf16", seed=4).fill()
    t = c.d_table.clone()
    t[0, 2] = -1
    t[0, 3] = c.pages + 5
    o, lse, ws = c.outputs()
    gdn.attention(c.cfg, c.d_q, c.d_cu, c.cu, c.d_lens, c.pool, t, o, lse, ws)
    assert gdn.device_status() & 0xFF == 4
    # the other sequence is unaffected; this one attends to what is left
    c.check(o, lse, skip=(0,))
    keep = [j for j in range(c.lens[0]) if j // 16 not in (2, 3)]
    kp, vp = quantise(c.k[0], 64)[3], quantise(c.v[0], 128)[3]
    s = torch.einsum("hd,thd->ht", c.q[0].double(), kp[:c.lens[0] - new + 1].repeat_interleave(3, 1)) * c.scale
    p = torch.zeros_like(s)
    keep = [j for j in keep if j < s.shape[1]]
    p[:, keep] = torch.softmax(s[:, keep], -1)
    ref = torch.einsum("ht,thd->hd", p, vp[:s.shape[1]].repeat_interleave(3, 1))
    assert ((o[0].cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -9).all()
    # a length past the table's row counts the row's tokens
    lens = c.d_lens.clone()
    lens[1] = c.width * c.page + 3
    gdn.attention(c.cfg, c.d_q, c.d_cu, c.cu, lens, c.pool, c.d_table, o, lse, ws)
    assert gdn.device_status() & 0xFF == 4


@pytest.mark.parametrize("new", [1, 33])
def test_attention_non_finite_tokens_reach_only_their_readers(new):
    """A NaN in a token's value reaches the sequences that see it and no other; masked places are not read."""
    c = Case([new, new], [40, 40], 4, 2, 64, 16, "bf16", seed=14)
    c.v[0][3, 0, 5] = math.nan
    c.fill()
    o, lse = c.attention()
    assert torch.isnan(o[:new, :2]).all() and torch.isfinite(o[:new, 2:]).all()
    o[:new] = 0
    c.check(o, lse, skip=(0,))


def test_attention_large_scores_and_shifts():
    """Scores around +-1e4 and equal scores: the softmax neither overflows nor loses its sum."""
    c = Case([1, 1], [90, 90], 2, 2, 64, 16, "f32", seed=15, outlier=False)
    c.q[0] *= 3e3
    c.q[1] = 0.0
    c.d_q = c.q.cuda()
    c.fill()
    o, lse = c.attention()
    kp, vp = quantise(c.k[1], 64), quantise(c.v[1], 64)
    assert ((o[1].cpu().double() - vp[3].mean(0)).abs() <= 2.0 ** -18 * 8).all()
    assert ((lse[1].cpu().double() - math.log(91)).abs() <= 2.0 ** -20).all()
    ref, rl = __import__("attn_ref").attention64(c.q[:1], *(quantise(t[0], 64)[3] for t in (c.k, c.v)), c.scale, 1)
    assert ((lse[0].cpu().double() - rl[0]).abs() <= 2.0 ** -19 * rl[0].abs()).all()
    assert torch.isfinite(o).all()


def test_attention_strided_queries_no_lse_and_scale():
    c = Case([2, 5], [30, 9], 6, 2, 128, 16, "bf16", seed=16).fill()
    o, lse = c.attention()
    wide = torch.full((c.T, 9, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:8] = c.d_q
    o2, _, ws = c.outputs()
    gdn.attention(c.cfg, wide[:, 2:8], c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, o2, None, ws)
    assert torch.equal(o, o2)
    cfg = gdn.make_attn_config(6, 2, 128, page_size=16, softmax_scale=0.0)
    gdn.attention(cfg, c.d_q, c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, o2, lse, ws)
    seen = torch.tensor([31, 32, 10, 11, 12, 13, 14], dtype=torch.float64)
    assert ((lse.cpu().double() - seen.log().unsqueeze(1)).abs() <= 2.0 ** -20).all()


def test_attention_pool_past_two_gigabytes():
    """Page offsets past 2^31 bytes."""
    d, page, hkv = 128, 64, 2
    cfg = gdn.make_attn_config(4, hkv, d, page_size=page)
    pages = (5 << 30) // gdn.kv_page_bytes(cfg)
    c = Case([1], [300], 4, hkv, d, page, "bf16", seed=17)
    pool = torch.empty(pages, gdn.kv_page_bytes(cfg), dtype=torch.uint8, device="cuda")
    c.pool, c.pages = pool, pages
    for j in range(c.width):
        c.table[0, j] = pages - 1 - 3 * j if j % 2 else 2 * j
    c.d_table = c.table.cuda()
    c.fill()
    c.check(*c.attention())


def test_attention_streams_and_concurrent_calls():
    cases = [Case([1] * 8, [900 + 13 * i for i in range(8)], 24, 2, 128, 64, "bf16", seed=s).fill() for s in (1, 2)]
    want = [c.attention() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(5):
        outs = []
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                outs.append(c.attention())
        torch.cuda.synchronize()
        got.append(outs)
    for outs in got:
        for (o, l), (wo, wl) in zip(outs, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


def test_decode_step_captured_and_replayed_with_growing_lengths():
    """One graph holds append and attention; kv_lens moves on the device between replays."""
    N, hq, hkv, d, page, steps = 3, 6, 2, 128, 16, 20
    ctx = [0, 14, 45]
    c = Case([1] * N, [x + steps for x in ctx], hq, hkv, d, page, "bf16", seed=21)
    plan = gdn.rope_plan(64, 1e4)
    lens = torch.tensor(ctx, dtype=torch.int32).cuda()
    pre = np.concatenate(([0], np.cumsum(ctx))).astype(np.int32)
    kc = torch.cat([t[:n] for t, n in zip(c.k, ctx)]).cuda()
    vc = torch.cat([t[:n] for t, n in zip(c.v, ctx)]).cuda()
    gdn.kv_append(c.cfg, plan, None, kc, vc, None, torch.from_numpy(pre).cuda(), pre, lens, c.pool, c.d_table, None)
    q, k, v = (torch.zeros(N, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    q_rot = torch.empty_like(q)
    o, lse, ws = c.outputs()

    def step():
        lens.add_(1)
        gdn.kv_append(c.cfg, plan, q, k, v, None, c.d_cu, c.cu, lens, c.pool, c.d_table, q_rot)
        gdn.attention(c.cfg, q_rot, c.d_cu, c.cu, lens, c.pool, c.d_table, o, lse, ws)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    g = torch.Generator().manual_seed(1)
    f, ax = frequencies(64, 1e4, None, "sections")
    for i in range(steps):
        qi = torch.randn(N, hq, d, generator=g).bfloat16()
        q.copy_(qi.cuda())
        k.copy_(torch.stack([t[n + i] for t, n in zip(c.k, ctx)]).cuda())
        v.copy_(torch.stack([t[n + i] for t, n in zip(c.v, ctx)]).cuda())
        graph.replay()
        torch.cuda.synchronize()
        if i in (0, 1, 2, steps - 1):
            for n in range(N):
                L = ctx[n] + i + 1
                cs = cos_sin(np.arange(L)[None], f, ax)
                kq = quantise(rotate32(c.k[n][:L], cs), 64)
                vq = quantise(c.v[n][:L], 128)
                one = cos_sin(np.array([[L - 1]]), f, ax)
                qr = rotate32(qi[n:n + 1], one).bfloat16()
                from attn_ref import attention64, attention_bound
                ref, _ = attention64(qr, kq[3], vq[3], c.scale, 1)
                eo, _ = attention_bound(qr, kq, vq, ref, c.scale, 1, "bf16")
                assert ((o[n:n + 1].cpu().double() - ref).abs() <= eo + 2.0 ** -10).all(), (i, n)
    assert gdn.device_status() == 0


def test_outputs_past_the_last_token_are_left_alone():
    c = Case([1, 2], [20, 3], 6, 2, 128, 16, "bf16", seed=22).fill()
    o, lse, ws = c.outputs()
    big_o = torch.full((c.T + 5, 6, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    big_l = torch.full((c.T + 5, 6), 7.0, device="cuda")
    gdn.attention(c.cfg, c.d_q, c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, big_o, big_l, ws)
    c.check(big_o[:c.T], big_l[:c.T])
    assert (big_o[c.T:] == 7.0).all() and (big_l[c.T:] == 7.0).all()


# ------------------------------------------------------------------------- the long row tiles (bf16)
@pytest.mark.parametrize("d,hq,hkv,page", [(64, 4, 2, 32), (128, 6, 2, 64)])
def test_long_tiles_masked_nan_values_reach_only_their_readers(d, hq, hkv, page):
    """A token whose value is NaN is seen by the queries from its position on and by no other."""
    new, ctx, at = 90, 37, 80
    c = Case([new], [ctx], hq, hkv, d, page, "bf16", seed=31)
    c.v[0][at, 0, 5] = math.nan  # the whole group stands for NaN
    c.fill()
    o, lse = c.attention()
    group = hq // hkv
    sees = torch.arange(new) + ctx >= at
    assert torch.isnan(o[sees.cuda(), :group]).all()
    assert torch.isfinite(o[~sees.cuda()]).all() and torch.isfinite(o[:, group:]).all() and torch.isfinite(lse).all()
    # the others are what they are without it
    clean = Case([new], [ctx], hq, hkv, d, page, "bf16", seed=31).fill()
    o2, l2 = clean.attention()
    assert torch.equal(o[~sees.cuda()], o2[~sees.cuda()]) and torch.equal(lse, l2)


@pytest.mark.parametrize("k_scale,v_scale,q_scale", [(1e5, 1e-6, 1e-5), (1e-8, 3e6, 1e7), (1e-20, 1e-20, 1.0), (3e4, 1e30, 1e-4)])
def test_long_tiles_magnitudes_past_fp16(k_scale, v_scale, q_scale):
    """Keys, values and queries far outside fp16's range: powers of two over the operands keep them."""
    c = Case([70, 3], [200, 500], 4, 2, 128, 32, "bf16", seed=32)
    c.k = [(t.float() * k_scale).bfloat16() for t in c.k]
    c.v = [(t.float() * v_scale).bfloat16() for t in c.v]
    c.q = (c.q.float() * q_scale).bfloat16()
    c.d_q = c.q.cuda()
    c.fill()
    o, lse = c.attention()
    c.check(o, lse)


def test_long_tiles_values_that_grow_along_the_context():
    """Each 128 tokens ten times the last: the references of keys and values move while rows run."""
    c = Case([80], [1000], 2, 1, 128, 64, "bf16", seed=33, outlier=False)
    grow = 10.0 ** (torch.arange(1080) // 128).float()[:, None, None]
    c.v = [(c.v[0].float() * grow * 1e-4).bfloat16()]
    c.k = [(c.k[0].float() * (1 + torch.arange(1080).float()[:, None, None] / 300)).bfloat16()]
    c.fill()
    o, lse = c.attention()
    c.check(o, lse)


@pytest.mark.parametrize("scale", [-0.05, 0.0, 2.0])
def test_long_tiles_other_scales(scale):
    c = Case([66], [300], 2, 2, 64, 16, "bf16", seed=34, outlier=False)
    c.cfg = gdn.make_attn_config(2, 2, 64, page_size=16, softmax_scale=scale)
    c.scale = scale
    c.fill()
    o, lse = c.attention()
    c.check(o, lse)


def test_long_tiles_batches_of_many_and_empty_sequences():
    """More groups than blocks, groups cut between blocks, sequences without new tokens, one that sees nothing."""
    new = [0, 70, 1, 65, 0, 260, 3, 128, 129] * 3
    ctx = [5, 0, 100, 64, 0, 300, 40, 1, 0] * 3
    c = Case(new, ctx, 4, 4, 64, 16, "bf16", seed=35).fill()
    c.d_lens[2] = 0
    o, lse = c.attention()
    a = int(c.cu[2])
    assert (o[a] == 0).all() and (lse[a] == -math.inf).all()
    c.check(o, lse, skip=(2,))
    assert torch.equal(o, c.attention()[0])


def test_long_tiles_captured_and_on_two_streams():
    cases = [Case([300, 17], [100, 900], 6, 2, 128, 64, "bf16", seed=s).fill() for s in (41, 42)]
    want = [c.attention() for c in cases]
    outs = [c.outputs() for c in cases]
    graphs = []
    for c, (o, l, ws) in zip(cases, outs):
        g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=st):
            gdn.attention(c.cfg, c.d_q, c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, o, l, ws)
        graphs.append((g, st))
    for _ in range(4):
        for (o, l, ws) in outs:
            o.fill_(0)
        torch.cuda.synchronize()
        for g, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (o, l, ws), (wo, wl) in zip(outs, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


# heads of 256 channels: one row tile a block, two buffers of scores, two groups of values
@pytest.mark.parametrize("new,ctx,hq,hkv,page", [([65], [0], 1, 1, 16), ([129, 1, 0, 70], [127, 300, 5, 0], 2, 2, 48),
                                                 ([40], [1000], 16, 2, 64), ([300, 17], [2000, 900], 6, 2, 128),
                                                 ([9, 33], [5000, 3], 8, 1, 32), ([128], [128], 1, 1, 128)])
def test_wide_heads_against_float64(new, ctx, hq, hkv, page):
    c = Case(new, ctx, hq, hkv, 256, page, "bf16", seed=61).fill()
    o, lse = c.attention()
    c.check(o, lse)
    assert torch.equal(o, c.attention()[0])


@pytest.mark.parametrize("channel", [5, 200])
def test_wide_heads_masked_nan_values_reach_only_their_readers(channel):
    """A value group that stands for NaN is half of a head: the other half's outputs are numbers."""
    new, ctx, at = 90, 37, 80
    c = Case([new], [ctx], 6, 2, 256, 64, "bf16", seed=62)
    c.v[0][at, 0, channel] = math.nan
    c.fill()
    o, lse = c.attention()
    sees = (torch.arange(new) + ctx >= at).cuda()
    half = slice(0, 128) if channel < 128 else slice(128, 256)
    other = slice(128, 256) if channel < 128 else slice(0, 128)
    assert torch.isnan(o[sees, :3, half]).all() and torch.isfinite(o[sees, :3, other]).all()
    assert torch.isfinite(o[~sees]).all() and torch.isfinite(o[:, 3:]).all() and torch.isfinite(lse).all()
    o2, l2 = Case([new], [ctx], 6, 2, 256, 64, "bf16", seed=62).fill().attention()
    assert torch.equal(o[~sees], o2[~sees]) and torch.equal(lse, l2)


@pytest.mark.parametrize("k_scale,v_scale,q_scale", [(1e5, 1e-6, 1e-5), (1e-8, 3e6, 1e7), (3e4, 1e30, 1e-4)])
def test_wide_heads_magnitudes_past_fp16(k_scale, v_scale, q_scale):
    c = Case([70, 3], [200, 500], 4, 2, 256, 32, "bf16", seed=63)
    c.k = [(t.float() * k_scale).bfloat16() for t in c.k]
    c.v = [(t.float() * v_scale).bfloat16() for t in c.v]
    c.q = (c.q.float() * q_scale).bfloat16()
    c.d_q = c.q.cuda()
    c.fill()
    o, lse = c.attention()
    c.check(o, lse)


def test_wide_heads_values_that_grow_along_the_context():
    """The references move from tile to tile: every time the output is rescaled behind the product before it."""
    c = Case([80], [1000], 2, 1, 256, 64, "bf16", seed=64, outlier=False)
    grow = 10.0 ** (torch.arange(1080) // 128).float()[:, None, None]
    c.v = [(c.v[0].float() * grow * 1e-4).bfloat16()]
    c.k = [(c.k[0].float() * (1 + torch.arange(1080).float()[:, None, None] / 300)).bfloat16()]
    c.fill()
    o, lse = c.attention()
    c.check(o, lse)


def test_wide_heads_batches_of_many_and_empty_sequences():
    new = [0, 70, 1, 65, 0, 260, 3, 128, 129] * 3
    ctx = [5, 0, 100, 64, 0, 300, 40, 1, 0] * 3
    c = Case(new, ctx, 4, 4, 256, 16, "bf16", seed=65).fill()
    c.d_lens[2] = 0
    o, lse = c.attention()
    a = int(c.cu[2])
    assert (o[a] == 0).all() and (lse[a] == -math.inf).all()
    c.check(o, lse, skip=(2,))


def test_attention_many_sequences():
    """More sequences than a block has threads, with and without new tokens."""
    n = 700
    new = [i % 3 == 0 for i in range(n)]
    c = Case([int(x) for x in new], [1 + (7 * i) % 50 for i in range(n)], 2, 1, 64, 16, "bf16", seed=36).fill()
    o, lse = c.attention()
    c.check(o, lse)
    c = Case([66] + [int(x) for x in new], [3] + [1 + (7 * i) % 50 for i in range(n)], 2, 1, 64, 16, "bf16", seed=37).fill()
    o, lse = c.attention()
    c.check(o, lse)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1184, 2368, 4736, 4737])
def test_rope_at_the_steps_of_its_block_size(io, T):
    """Tokens a block change with T; in place, odd pair counts and a ragged last block."""
    g = torch.Generator().manual_seed(T)
    for H, D, rot in ((3, 64, 64), (5, 80, 60)):
        x = torch.randn(T, H, D, generator=g).to(DT[io])
        pos = torch.randint(0, 300000, (T,), generator=g, dtype=torch.int32)
        plan = gdn.rope_plan(rot, 1e6)
        f, ax = frequencies(rot, 1e6, None, "sections")
        ref = rotate64(x, cos_sin(pos.view(1, -1).numpy(), f, ax))
        out = x.cuda()
        gdn.rope(plan, out, pos.cuda(), out)
        mag = torch.cat((x.double().abs()[..., :rot // 2] + x.double().abs()[..., rot // 2:rot],) * 2 + (x.double().abs()[..., rot:],), -1)
        assert ((out.cpu().double() - ref).abs() <= U[io] * ref.abs() + 6 * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("n", [1000, 1100])
def test_append_many_sequences(n):
    """Sequences are found by a look at all of them, or by bisection where there are more than 1024."""
    c = Case([i % 2 for i in range(n)], [3 + i % 7 for i in range(n)], 1, 1, 64, 16, "bf16", seed=38)
    k, v = torch.randn(c.T, 1, 64).bfloat16().cuda(), torch.randn(c.T, 1, 64).bfloat16().cuda()
    gdn.kv_append(c.cfg, None, None, k, v, None, c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, None)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    gdn.kv_read(c.cfg, c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, ko, vo)
    assert torch.equal(vo.cpu(), quantise(v.cpu(), 64)[3].bfloat16()) and torch.equal(ko.cpu(), quantise(k.cpu(), 64)[3].bfloat16())


@pytest.mark.parametrize("new", [1, 4])
@pytest.mark.parametrize("k_scale,v_scale,q_scale", [(1e5, 1e-6, 1e-5), (1e-8, 3e6, 1e7), (1e-20, 1e-20, 1.0), (3e4, 1e30, 1e-4)])
def test_short_tiles_magnitudes_past_fp16(new, k_scale, v_scale, q_scale):
    c = Case([new, new], [200, 500], 4, 2, 128, 32, "bf16", seed=52)
    c.k = [(t.float() * k_scale).bfloat16() for t in c.k]
    c.v = [(t.float() * v_scale).bfloat16() for t in c.v]
    c.q = (c.q.float() * q_scale).bfloat16()
    c.d_q = c.q.cuda()
    c.fill()
    c.check(*c.attention())


@pytest.mark.parametrize("d", [64, 256])
def test_short_tiles_values_that_grow_and_nan_in_a_draft(d):
    """Scales of the values grow along the context; the last draft token's value is NaN and only its own rows see it."""
    c = Case([3], [1000], 4, 2, d, 64, "bf16", seed=53, outlier=False)
    grow = 10.0 ** (torch.arange(1003) // 128).float()[:, None, None]
    c.v = [(c.v[0].float() * grow * 1e-4).bfloat16()]
    c.fill()
    o, lse = c.attention()
    c.check(o, lse)
    n = Case([3], [1000], 4, 2, d, 64, "bf16", seed=53, outlier=False)
    n.v = [c.v[0].clone()]
    n.v[0][1002, 1, 0] = math.nan
    n.fill()
    o2, l2 = n.attention()
    assert torch.isnan(o2[2, 2:, :min(d, 128)]).all() and torch.equal(o2[:2], o[:2]) and torch.equal(o2[2, :2], o[2, :2])
    assert torch.equal(l2, lse)


@pytest.mark.parametrize("new,ctx,hq,hkv", [
    ([130], [0], 1, 1),                  # groups of one and of two key tiles
    ([129], [127], 1, 1),                # two whole key tiles
    ([140], [200], 2, 2),                # two and three
    ([129, 150, 200], [40, 250, 300], 2, 1),
    ([300], [2000], 16, 1),              # whole groups, and groups cut anywhere
    ([20], [6000], 8, 1),                # one group over many blocks
])
def test_wide_heads_rows_have_all_their_products(new, ctx, hq, hkv):
    """The rows that end a piece wait for its last product, whatever the loads beside it: copies on another stream take
    the memory for some of the passes, and every pass has the first one's bits."""
    c = Case(new, ctx, hq, hkv, 256, 64, "bf16", seed=66).fill()
    o, lse = c.attention()
    c.check(o, lse)
    side, a = torch.cuda.Stream(), torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    b = torch.empty_like(a)
    out, l2, ws = c.outputs()
    torch.cuda.synchronize()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(300):
        if i % 3 == 0:
            with torch.cuda.stream(side):
                b.copy_(a)
        out.fill_(7.0)
        gdn.attention(c.cfg, c.d_q, c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, out, l2, ws)
        differ += (out != o).sum() + (l2 != lse).sum()
    torch.cuda.synchronize()
    assert differ.item() == 0


@pytest.mark.parametrize("q_scale", [1e5, 1e10, 1e27])
@pytest.mark.parametrize("new,d", [(70, 64), (70, 128), (140, 256), (3, 128)])
def test_attention_scores_far_past_the_exponents_range(new, d, q_scale):
    """Scores of 1e6 to 1e28: a row takes the value of its largest score, and lse is that score."""
    c = Case([new], [200], 2, 2, d, 64, "bf16", seed=67, outlier=False)
    c.q = (c.q.float() * q_scale).bfloat16()
    c.d_q = c.q.cuda()
    c.fill()
    o, lse = c.attention()
    c.check(o, lse)
    k, v = quantise(c.k[0], 64)[3], quantise(c.v[0], v_group(d))[3]
    for i in range(0, new, 7):
        for h in range(2):
            qa = c.q[i, h].double()
            s = (k[:201 + i, h] @ qa) * c.scale
            top = s.topk(2).values
            # attention_bound: a score is off by 2^-20 of the sum of its magnitudes, which is under 8 |q|_1; a gap of 2^5
            # leaves e^-32 of the next value, under the bound's own terms
            if top[0] - top[1] <= 2 * 2.0 ** -20 * 8 * qa.abs().sum() * c.scale + 32:
                continue
            want = v[s.argmax(), h]
            tol = 2.0 ** -8 * want.abs() + (2 * 2.0 ** -11 + 2.0 ** -19 + new * 2.0 ** -25 + 201 * 2.0 ** -25) * 2 * v.abs().max()
            assert ((o[i, h].cpu().double() - want).abs() <= tol).all(), (i, h)


@pytest.mark.parametrize("big", [1e9, 1e30])
@pytest.mark.parametrize("by_head", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_tiles_large_neighbours_leave_small_ones_alone(d, by_head, big):
    """Requests, or key/value heads, of one call differ by many powers of two and share blocks (400 groups and more over
    at most 148): each keeps its own bound."""
    n, hkv = (50, 8) if by_head else (400, 1)
    c = Case([70] * n, [60 + i % 3 for i in range(n)], hkv * (1 if d <= 128 else 2), hkv, d, 64, "bf16", seed=71)
    for i in range(n):
        if by_head:
            for t in (c.k[i], c.v[i]):
                t[:, ::3] = (t[:, ::3].float() * big).bfloat16()
        elif i % 3 == 0:
            c.k[i], c.v[i] = ((t.float() * big).bfloat16() for t in (c.k[i], c.v[i]))
    c.fill()
    c.check(*c.attention(), skip=[i for i in range(n) if (i % 25 if by_head else i % 23 > 1)])


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 6, 2), (256, 8, 1)])
@pytest.mark.parametrize("short", [[1, 1, 1, 1, 1], [1, 0, 4, 2, 7]])
def test_attention_short_sequences_beside_prompts(d, hq, hkv, short):
    """Each sequence of a call is rounded as it is alone: the ones and the drafts have the bits of a call without the
    prompts, the prompts those of a call without the others, in any order and captured."""
    longs, at = [150, 40 if d > 64 else 90], (1, 3)
    new = list(short)
    for i, x in zip(at, longs):
        new.insert(i, x)
    ctx = [500, 300, 17, 40, 900, 0, 64]
    c = Case(new, ctx, hq, hkv, d, 32, "bf16", seed=81).fill()
    o, lse = c.attention()
    c.check(o, lse)

    def part(keep):
        cu = np.concatenate(([0], np.cumsum([new[i] for i in keep]))).astype(np.int32)
        rows = torch.cat([torch.arange(int(c.cu[i]), int(c.cu[i + 1])) for i in keep]).cuda()
        q, T = c.d_q[rows].contiguous(), int(cu[-1])
        po = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        pl = torch.full((T, hq), 7.0, device="cuda")
        ws = torch.empty(max(256, gdn.attention_workspace_size(c.cfg, T, len(keep))), dtype=torch.uint8, device="cuda")
        gdn.attention(c.cfg, q, torch.from_numpy(cu).cuda(), cu, c.d_lens[keep].contiguous(), c.pool,
                      c.d_table[keep].contiguous(), po, pl, ws)
        assert torch.equal(po, o[rows]) and torch.equal(pl, lse[rows])

    part([i for i in range(7) if i not in at])
    part(list(at))
    o2, l2, ws = c.outputs()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        gdn.attention(c.cfg, c.d_q, c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, o2, l2, ws)
    for _ in range(3):
        o2.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, o) and torch.equal(l2, lse)


@pytest.mark.parametrize("pad", [-1, -5, -2 ** 31])
@pytest.mark.parametrize("new", [1, 3, 70])
def test_negative_lengths_are_padding(pad, new):
    """A padding row's length may be any number up to 0: nothing is stored, seen or reported."""
    c = Case([new, 2], [20, 9], 2, 2, 64, 16, "bf16", seed=91).fill()
    c.d_lens[0] = pad
    before = c.pool.clone()
    k, v = (torch.randn(c.T, 2, 64, generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in (1, 2))
    k[new:], v[new:] = c.k[1][-2:].cuda(), c.v[1][-2:].cuda()  # what the other sequence holds already
    gdn.kv_append(c.cfg, None, None, k, v, None, c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, None)
    assert torch.equal(c.pool, before)
    ko, vo = torch.full_like(k, 5.0), torch.full_like(v, 5.0)
    gdn.kv_read(c.cfg, c.d_cu, c.cu, c.d_lens, c.pool, c.d_table, ko, vo)
    assert (ko[:new] == 0).all() and (vo[:new] == 0).all() and (ko[new:] != 0).any()
    o, lse = c.attention()
    assert (o[:new] == 0).all() and (lse[:new] == -math.inf).all()
    assert gdn.device_status() == 0
    c.check(o, lse, skip=(0,))
