"""The product with 4-bit weights through the public calls against float64, and a layer's decode step together."""

import numpy as np
import pytest
import torch

import linear_attention_recurrence_deltanet_b200 as gdn
from attn_ref import DT, U, Case, attention64, quantise, v_group

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    gdn.lib()
    yield
    assert gdn.device_status() == 0


def weight(N, K, group, seed):
    """(code [N, K], scale, bias [N, G], packed) with codes past K set, so that reading them would show."""
    g = torch.Generator().manual_seed(seed)
    G = -(-K // group)
    code = torch.randint(0, 16, (N, G * group), generator=g, dtype=torch.uint8)
    scale = ((0.5 + torch.rand(N, G, generator=g)) * 0.05).bfloat16()
    bias = (scale.float() * (-7.5 + torch.randn(N, G, generator=g))).bfloat16()
    packed = gdn.q4_pack((code[:, 0::2] | (code[:, 1::2] << 4)).cuda(), scale.cuda(), bias.cuda(), K, group)
    return code[:, :K].double(), scale.double(), bias.double(), packed


def product(x, code, scale, bias, group):
    """(y, magnitude of what the sums saw for bf16 io, the same for fp32) in float64."""
    K = code.shape[1]
    s, b = (t.repeat_interleave(group, 1)[:, :K] for t in (scale, bias))
    x = x.double()
    return x @ (s * code + b).t(), x.abs() @ (144 * s + b.abs()).t(), x.abs() @ (8 * s + (b + 8 * s).abs()).t()


def run(x, w, fill=9.0):
    M, io = x.shape[0], "bf16" if x.dtype == torch.bfloat16 else "f32"
    y = torch.full((M, w.N), fill, dtype=x.dtype, device="cuda")
    ws = torch.full((max(256, gdn.linear_q4_workspace_size(M, w.N, w.K, w.group, io)),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    gdn.linear_q4(x, w, y, ws)
    return y


SHAPES = [(1, 16, 64), (1, 1, 8), (1, 5120, 640), (2, 33, 200), (3, 100, 5120), (5, 1000, 128), (7, 17, 72),
          (8, 256, 1024), (9, 47, 328), (16, 512, 2048), (17, 130, 264), (31, 64, 512), (33, 200, 1000), (64, 320, 768),
          (65, 70, 136), (100, 257, 512), (200, 129, 640), (300, 520, 1032)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_q4_against_float64(io, group, M, N, K):
    code, scale, bias, w = weight(N, K, group, M + N + K)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(DT[io])
    y = run(x.cuda(), w)
    ref, mag_b, mag_f = product(x, code, scale, bias, group)
    # exact products, sums that lose at most 2^-20 of the magnitudes (see attention_bound); more than 16 rows of bf16 round
    # the weights to fp16 first (half a step, 2^-11 each) and x, scaled to below 2^11 by its row's largest, to steps of
    # 2^-24 at least: 2^-25 / 2^10 of that largest; one final rounding
    if io == "f32":
        tol = U[io] * ref.abs() + 2.0 ** -20 * mag_f
    else:
        s, b = (t.repeat_interleave(group, 1)[:, :K] for t in (scale, bias))
        tol = U[io] * ref.abs() + 2.0 ** -20 * mag_b
        if M > 16:
            w64 = (s * code + b).abs().t()
            tol += 2.0 ** -11 * (x.double().abs() @ w64)
            tol += 2.0 ** -35 * x.double().abs().amax(1, keepdim=True) * w64.sum(0)
    off = (y.cpu().double() - ref).abs() - tol
    assert off.max() <= 0, off.max()
    assert torch.equal(y, run(x.cuda(), w, fill=-3.0))


def test_linear_q4_zero_rows_and_outputs():
    _, _, _, w = weight(64, 128, 64, 1)
    x = torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda")
    gdn.linear_q4(x, w, torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))


def test_linear_q4_ignores_rows_past_the_last_and_reads_no_padding():
    """Rows of y past M stay; K not a multiple of the group: the tail of x is not read past K."""
    code, scale, bias, w = weight(50, 72, 64, 2)
    flat = torch.full((3 * 72 + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = torch.randn(3, 72, generator=torch.Generator().manual_seed(1)).bfloat16()
    flat[:216] = x.flatten().cuda()
    y = torch.full((5, 50), 6.0, dtype=torch.bfloat16, device="cuda")
    gdn.linear_q4(flat[:216].view(3, 72), w, y[:3], torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    assert torch.isfinite(y).all() and (y[3:] == 6.0).all()


def test_linear_q4_non_finite_rows_stay_apart():
    code, scale, bias, w = weight(40, 256, 32, 3)
    x = torch.randn(6, 256, generator=torch.Generator().manual_seed(1)).bfloat16()
    clean = run(x.cuda(), w)
    x[2, 7] = float("inf")
    y = run(x.cuda(), w)
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(y[keep], clean[keep]) and not torch.isfinite(y[2]).any()


def test_linear_q4_captured_on_a_side_stream():
    _, _, _, w = weight(300, 512, 64, 4)
    x = torch.randn(4, 512, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    want = run(x, w)
    y = torch.empty_like(want)
    ws = torch.empty(max(256, gdn.linear_q4_workspace_size(4, 300, 512, 64)), dtype=torch.uint8, device="cuda")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        gdn.linear_q4(x, w, y, ws)
    for _ in range(3):
        y.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_layer_decode_steps_together():
    """linear_q4 (q, k, v rows) -> kv_append -> attention -> linear_q4, three steps of two sequences, against the same
    steps in float64 from each stage's own rounded inputs."""
    hidden, hq, hkv, d, page, N = 192, 6, 2, 64, 16, 2
    rows = (hq + 2 * hkv) * d
    ci, si, bi, w_in = weight(rows, hidden, 64, 5)
    co, so, bo, w_out = weight(hidden, hq * d, 128, 6)
    cfg = gdn.make_attn_config(hq, hkv, d, page_size=page)
    plan = gdn.rope_plan(32, 1e4)
    table = torch.tensor([[1], [3]], dtype=torch.int32).cuda()
    pool = torch.full((4, gdn.kv_page_bytes(cfg)), 0xFF, dtype=torch.uint8, device="cuda")
    cu = np.array([0, 1, 2], np.int32)
    cu_d, lens = torch.from_numpy(cu).cuda(), torch.zeros(2, dtype=torch.int32, device="cuda")
    kept_k, kept_v = [[], []], [[], []]
    g = torch.Generator().manual_seed(2)
    for step in range(3):
        x = torch.randn(N, hidden, generator=g).bfloat16()
        qkv = run(x.cuda(), w_in)
        ref, mag, _ = product(x, ci, si, bi, 64)
        assert ((qkv.cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -20 * mag).all()
        r = qkv.view(N, hq + 2 * hkv, d)
        lens += 1
        q_rot = torch.empty(N, hq, d, dtype=torch.bfloat16, device="cuda")
        gdn.kv_append(cfg, plan, r[:, :hq], r[:, hq:hq + hkv], r[:, hq + hkv:], None, cu_d, cu, lens, pool, table, q_rot)
        ko, vo = (torch.empty(N, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        gdn.kv_read(cfg, cu_d, cu, lens, pool, table, ko, vo)
        o = torch.empty(N, hq, d, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(max(256, gdn.attention_workspace_size(cfg, N, N)), dtype=torch.uint8, device="cuda")
        gdn.attention(cfg, q_rot, cu_d, cu, lens, pool, table, o, None, ws)
        y = run(o.view(N, hq * d), w_out)
        for n in range(N):
            # the cache's values are read back rounded to bf16: half a step of each
            kept_k[n].append(ko[n].cpu().double())
            kept_v[n].append(vo[n].cpu().double())
            k, v = torch.stack(kept_k[n]), torch.stack(kept_v[n])
            want, _ = attention64(q_rot[n:n + 1].cpu(), k, v, d ** -0.5, 1)
            ds = 2.0 ** -8 * (q_rot[n].cpu().double().abs().sum(-1).max() * k.abs().max() * d ** -0.5)
            tol = 2.0 ** -8 * want.abs() + (2 * ds + 2.0 ** -8 + 2.0 ** -12) * v.abs().max()
            assert ((o[n:n + 1].cpu().double() - want).abs() <= tol).all()
        ref, mag, _ = product(o.view(N, -1).cpu(), co, so, bo, 128)
        assert ((y.cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -20 * mag).all()


@pytest.mark.parametrize("M", [1, 20, 300])
@pytest.mark.parametrize("w_scale,x_scale", [(1e-9, 1e6), (1e8, 1e-8), (1.0, 1e35), (1e30, 1e-30)])
def test_linear_q4_magnitudes_past_fp16(M, w_scale, x_scale):
    """Weights and rows of x far outside fp16's range, and rows of one call that differ by 2^40."""
    N, K, group = 150, 200, 64
    g = torch.Generator().manual_seed(7)
    G = -(-K // group)
    code = torch.randint(0, 16, (N, G * group), generator=g, dtype=torch.uint8)
    scale = ((0.5 + torch.rand(N, G, generator=g)) * 0.05 * w_scale).bfloat16()
    bias = (scale.float() * (-7.5 + torch.randn(N, G, generator=g))).bfloat16()
    scale[::3] *= 2.0 ** -40
    bias[::3] *= 2.0 ** -40
    w = gdn.q4_pack((code[:, 0::2] | (code[:, 1::2] << 4)).cuda(), scale.cuda(), bias.cuda(), K, group)
    x = torch.randn(M, K, generator=g) * x_scale
    x[1::2] *= 2.0 ** -40
    x = x.bfloat16()
    y = run(x.cuda(), w)
    code, s, b = code[:, :K].double(), scale.double(), bias.double()
    ref, mag, _ = product(x, code, s, b, group)
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -20 * mag
    if M > 16:
        se, be = (t.repeat_interleave(group, 1)[:, :K] for t in (s, b))
        w64 = (se * code + be).abs().t()
        tol += 2.0 ** -11 * (x.double().abs() @ w64) + 2.0 ** -35 * x.double().abs().amax(1, keepdim=True) * w64.sum(0)
    assert ((y.cpu().double() - ref).abs() <= tol + 2.0 ** -126).all()


@pytest.mark.parametrize("M,N,K,group", [(40, 20000, 128, 32), (2000, 2100, 192, 64), (17, 8, 8, 128), (700, 1300, 1024, 128)])
def test_linear_q4_rounds_and_slices(M, N, K, group):
    """Whole rounds of tiles and a last one cut along K, for calls that share one workspace."""
    code, scale, bias, w = weight(N, K, group, M)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).bfloat16()
    ws = torch.full((gdn.linear_q4_workspace_size(M, N, K, group),), 0xFF, dtype=torch.uint8, device="cuda")
    y = [torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for t in y:
        gdn.linear_q4(x.cuda(), w, t, ws)
    assert torch.equal(y[0], y[1])
    ref, mag, _ = product(x, code, scale, bias, group)
    se, be = (t.repeat_interleave(group, 1)[:, :K] for t in (scale, bias))
    w64 = (se * code + be).abs().t()
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -20 * mag + 2.0 ** -11 * (x.double().abs() @ w64)
    tol += 2.0 ** -35 * x.double().abs().amax(1, keepdim=True) * w64.sum(0)
    assert ((y[0].cpu().double() - ref).abs() <= tol).all()


def test_linear_q4_many_rows_on_two_streams_and_captured():
    _, _, _, w = weight(700, 512, 64, 8)
    xs = [torch.randn(90, 512, generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in range(2)]
    want = [run(x, w) for x in xs]
    ys = [torch.empty_like(t) for t in want]
    ws = [torch.empty(gdn.linear_q4_workspace_size(90, 700, 512, 64), dtype=torch.uint8, device="cuda") for _ in xs]
    graphs = []
    for x, y, s in zip(xs, ys, ws):
        g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=st):
            gdn.linear_q4(x, w, y, s)
        graphs.append((g, st))
    for _ in range(5):
        for y in ys:
            y.fill_(0)
        torch.cuda.synchronize()
        for g, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, t) for y, t in zip(ys, want))


def test_linear_q4_weights_that_are_not_finite_stay_in_their_column():
    for M in (2, 40):
        code, scale, bias, w = weight(130, 128, 64, 9)
        x = torch.randn(M, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
        clean = run(x.cuda(), w)
        scale = scale.float().bfloat16()
        scale[77, 1] = float("nan")
        packed = gdn.q4_pack((code.to(torch.uint8)[:, 0::2] | (code.to(torch.uint8)[:, 1::2] << 4)).cuda(), scale.cuda(),
                             bias.bfloat16().cuda(), 128, 64)
        y = run(x.cuda(), packed)
        keep = torch.arange(130) != 77
        assert torch.isnan(y[:, 77]).all() and torch.equal(y[:, keep.cuda()], clean[:, keep.cuda()])


@pytest.mark.parametrize("M,N,K,group", [(129, 256, 512, 64), (256, 19200, 320, 32), (300, 9600, 640, 128), (600, 2500, 1288, 64),
                                         (128, 18944, 64, 32), (255, 700, 4096, 64)])
def test_products_with_one_and_two_accumulators(M, N, K, group):
    """Tiles of up to 128 rows of x and of more; several tiles a block, ragged last rows and weight rows, slices."""
    test_linear_q4_against_float64("bf16", group, M, N, K)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 130, 72), (5, 40, 264), (8, 1000, 128), (12, 257, 1096), (20, 70, 136), (32, 300, 512)])
def test_linear_q4_infinities_and_the_largest_numbers(io, group, M, N, K):
    """Few rows: an infinity in x gives the formula's infinity or NaN, and a value near the type's largest its product."""
    code, scale, bias, w = weight(N, K, group, M + N)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(DT[io])
    clean = x.clone()
    x[0, 7] = float("inf")
    if M > 2:
        x[1, K - 1] = -float("inf")
        x[2, 3], x[2, 9] = float("inf"), -float("inf")
    if M > 4:
        x[3, 0] = float("nan")
        x[4, K // 2] = 3.3e38  # weights are below 1: the product is within the type
    ref, mag_b, mag_f = product(x, code, scale, bias, group)
    y = run(x.cuda(), w).cpu().double()
    assert torch.equal(torch.isnan(y), torch.isnan(ref))
    assert torch.equal(y[torch.isinf(ref)], ref[torch.isinf(ref)])
    rows = [m for m in range(M) if not (m == 0 or M > 2 and m < 3 or M > 4 and m < 5)]
    assert torch.equal(run(clean.cuda(), w).cpu().double()[rows], y[rows])
    if M > 4:
        # a sum that passes fp32 is formed in fp64 and rounded to fp32 (2^-24 of it) and to the io type; one that does not is
        # the kernel's own, off by 2^-20 of its magnitudes at most (test_linear_q4_against_float64)
        tol = (U[io] + 2.0 ** -23) * ref[4].abs() + 2.0 ** -20 * (mag_f if io == "f32" else mag_b)[4]
        assert ((y[4] - ref[4]).abs() <= tol).all()


def test_q4_pack_on_another_stream_takes_no_memory_in_use():
    """What the current stream has freed may still be in use there: a weight packed on another stream does not lie in it."""
    N, K, group = 2048, 2048, 64
    g = torch.Generator().manual_seed(5)
    args = [torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda(),
            (torch.rand(N, K // group, generator=g) * 0.01).bfloat16().cuda(),
            torch.randn(N, K // group, generator=g).bfloat16().cuda()]
    want = gdn.q4_pack(*args, K, group)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = torch.zeros(want.data.numel(), dtype=torch.uint8, device="cuda")
    at = held.data_ptr()
    big = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(20):
        big.add_(1)
    held.add_(big[:held.numel()])  # pending: behind the passes over `big`
    del held
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        w = gdn.q4_pack(*args, K, group, stream=stream)
        assert not at <= w.data.data_ptr() < at + w.data.numel()
        torch.cuda.synchronize()
        assert torch.equal(w.data, want.data)
    assert torch.equal(gdn.q4_pack(*args, K, group).data, want.data)


@pytest.mark.parametrize("shape", [(), (64,), (2, 4, 32)])
def test_q4_pack_refuses_codes_that_are_no_matrix(shape):
    codes = torch.zeros(shape, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(2, 1, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gdn.GdnError) as e:
        gdn.q4_pack(codes, scales, scales, 64, 64)
    assert e.value.name == "GDN_E_INVAL"


@pytest.mark.parametrize("N,K,group", [(256, 128, 64), (128, 192, 64), (128, 128, 32)])
def test_linear_q4_refuses_a_weight_with_too_few_bytes(N, K, group):
    """Packed bytes that a program has kept, under other sizes than they were packed for."""
    _, _, _, w = weight(128, 128, 64, 10)
    x = torch.zeros(2, K, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gdn.GdnError) as e:
        gdn.linear_q4(x, gdn.Q4Weight(w.data, N, K, group), torch.empty(2, N, dtype=torch.bfloat16, device="cuda"))
    assert e.value.name == "GDN_E_INVAL" and "w has" in str(e.value)
    kept = gdn.Q4Weight(w.data, 128, 128, 64)
    x = torch.randn(2, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    assert torch.equal(run(x, kept), run(x, w))


def test_launches_are_counted_one_by_one():
    """The launch counter and the profiler see every kernel of a call."""
    gdn.profiler_reset()
    gdn.profiler_enable(True)
    before = gdn.launch_count()
    _, _, _, w = weight(300, 256, 64, 11)
    assert gdn.launch_count() - before == 2  # the codes and scales, the rows' powers of two
    run(torch.zeros(1, 256, dtype=torch.bfloat16, device="cuda"), w)
    assert gdn.launch_count() - before == 3
    run(torch.zeros(300, 256, dtype=torch.bfloat16, device="cuda"), w)
    assert gdn.launch_count() - before == 5  # x as the products' operand, the products
    gdn.profiler_enable(False)
    assert [gdn.profiler_read(k)[0] for k in (gdn.K.Q4_PACK, gdn.K.LINEAR_Q4, gdn.K.X_HALF)] == [2, 2, 1]
    gdn.profiler_reset()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(9, 47, 328), (16, 512, 2048), (17, 130, 264), (24, 257, 1096), (31, 64, 512), (32, 300, 520),
                                   (32, 3200, 3840), (24, 3100, 3840)])
def test_linear_q4_exact_rows_keep_their_promise(group, M, N, K):
    """9 to 16 rows of bf16, and to 32 for small weights (no workspace says that they are): nothing but sums is rounded."""
    assert gdn.linear_q4_workspace_size(M, N, K, group) == 0
    code, scale, bias, w = weight(N, K, group, M + N + K)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).bfloat16()
    ref, mag, _ = product(x, code, scale, bias, group)
    assert ((run(x.cuda(), w).cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -20 * mag).all()


@pytest.mark.parametrize("M,N,K", [(17, 3200, 3904), (32, 3300, 3840), (33, 3200, 3840)])
def test_linear_q4_rows_past_the_border_round_weights(M, N, K):
    assert gdn.linear_q4_workspace_size(M, N, K, 64) > 0
    test_linear_q4_against_float64("bf16", 64, M, N, K)
