"""The attention-side entry points and the 4-bit projection on the host: plans, sizes and refusals, before any launch."""

import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import linear_attention_recurrence_deltanet_b200 as gdn
from attn_ref import frequencies


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_attention_recurrence_deltanet_b200 import build
    build.build()
    yield


@pytest.mark.parametrize("rot,sections,layout", [
    (64, None, "sections"), (128, [24, 20, 20], "interleaved"), (128, [24, 20, 20], "sections"),
    (72, [12, 12, 12], "per_axis"), (60, [10, 20], "interleaved"), (256, [64, 0, 64], "per_axis"), (2, None, "sections"),
    (0, None, "sections"), (36, [18, 0], "per_axis"),
])
def test_plan_holds_the_definitions_frequencies(rot, sections, layout):
    plan = gdn.rope_plan(rot, 1e6, sections=sections, layout=layout)
    f, ax = frequencies(rot, 1e6, sections, layout)
    assert plan.rotary_dim == rot and plan.num_axes == (len(sections) if sections else 1)
    assert list(plan.axis[:rot // 2]) == list(ax)
    for j in range(rot // 2):
        turns = f[j] / (2 * math.pi)
        # a turn is an integer: half of 2^-64, besides the float64 steps of this line and of f
        assert abs(plan.turn[j] / 2.0 ** 64 - turns) <= 4 * 2.0 ** -53 * turns + 2.0 ** -65
    # phases by wrap-around: a position times the turn, modulo one turn
    if rot >= 64:
        for pos in (1, 262143, 2 ** 31 - 1, -5):
            for j in (0, 7, rot // 2 - 1):
                got = ((pos * plan.turn[j]) % 2 ** 64) / 2.0 ** 64
                want = (pos * f[j] / (2 * math.pi)) % 1.0
                d = abs(got - want)
                assert min(d, 1 - d) <= 2.0 ** -20 if abs(pos) > 2 ** 30 else 2.0 ** -30


def test_plan_custom_frequencies():
    f = np.array([2 * math.pi, 1.0, 0.0])
    plan = gdn.rope_plan(6, inv_freq=f)
    assert -plan.turn[0] % 2 ** 64 <= 2 ** 11 and plan.turn[2] == 0  # float64's 2 pi is within 2^-53 of a whole turn
    assert abs(plan.turn[1] / 2.0 ** 64 - 1 / (2 * math.pi)) < 1e-15


@pytest.mark.parametrize("args", [
    dict(rotary_dim=63), dict(rotary_dim=258), dict(rotary_dim=-2), dict(rotary_dim=64, theta=0.5),
    dict(rotary_dim=64, theta=float("nan")), dict(rotary_dim=64, theta=float("inf")),
    dict(rotary_dim=64, sections=[16, 15]), dict(rotary_dim=64, sections=[40, -8]),
    dict(rotary_dim=64, sections=[8, 8, 8, 8]), dict(rotary_dim=64, sections=[]), dict(rotary_dim=64, layout="other"),
    dict(rotary_dim=4, inv_freq=[1.0, 7.0]), dict(rotary_dim=4, inv_freq=[1.0, -0.1]),
    dict(rotary_dim=4, inv_freq=[1.0, float("nan")]), dict(rotary_dim=4, inv_freq=[1.0]),
])
def test_plan_refusals(args):
    with pytest.raises(gdn.GdnError) as e:
        gdn.rope_plan(**args)
    assert e.value.name == "GDN_E_INVAL"


def test_page_bytes_from_the_layout():
    for d, groups in ((64, 2), (128, 3), (256, 6)):
        cfg = gdn.make_attn_config(4, 2, d, page_size=48)
        assert gdn.kv_page_bytes(cfg) == 2 * 3 * 16 * (d + 4 * groups)


@pytest.mark.parametrize("args,status", [
    (dict(num_q_heads=5, num_kv_heads=2, head_dim=128), "GDN_E_INVAL"),
    (dict(num_q_heads=0, num_kv_heads=2, head_dim=128), "GDN_E_INVAL"),
    (dict(num_q_heads=4, num_kv_heads=0, head_dim=128), "GDN_E_INVAL"),
    (dict(num_q_heads=8192, num_kv_heads=2, head_dim=128), "GDN_E_UNSUPPORTED"),
    (dict(num_q_heads=4, num_kv_heads=2, head_dim=96), "GDN_E_UNSUPPORTED"),
    (dict(num_q_heads=4, num_kv_heads=2, head_dim=128, page_size=24), "GDN_E_INVAL"),
    (dict(num_q_heads=4, num_kv_heads=2, head_dim=128, page_size=0), "GDN_E_INVAL"),
    (dict(num_q_heads=4, num_kv_heads=2, head_dim=128, page_size=2048), "GDN_E_INVAL"),
    (dict(num_q_heads=4, num_kv_heads=2, head_dim=128, softmax_scale=float("nan")), "GDN_E_INVAL"),
])
def test_config_refusals(args, status):
    cfg = gdn.make_attn_config(**args)
    for call in (lambda: gdn.kv_page_bytes(cfg), lambda: gdn.attention_workspace_size(cfg, 4, 1)):
        with pytest.raises(gdn.GdnError) as e:
            call()
        assert e.value.name == status


def test_config_io_type_refused():
    with pytest.raises(gdn.GdnError) as e:
        gdn.make_attn_config(4, 2, 128, io_dtype=torch.float16)
    assert e.value.name == "GDN_E_UNSUPPORTED"


def test_workspace_size_refusals():
    cfg = gdn.make_attn_config(24, 2, 128)
    for T, N in ((-1, 1), (4, 0), (4, 65536), (1 << 31, 1)):
        with pytest.raises(gdn.GdnError) as e:
            gdn.attention_workspace_size(cfg, T, N)
        assert e.value.name == "GDN_E_INVAL"


class Host:
    """Host memory with a chosen alignment, for calls that are refused before anything reads it."""

    def __init__(self):
        self.buf = np.full(1 << 16, 0x5A, np.uint8)
        self.p = self.buf.ctypes.data + (-self.buf.ctypes.data) % 256

    def untouched(self):
        return (self.buf == 0x5A).all()


def refused(rc, word=None, status=-1):
    assert rc == status, (rc, gdn.last_error())
    assert word is None or word in gdn.last_error(), gdn.last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the last, valid call is for a machine without a GPU")
def test_rope_refusals():
    h = Host()
    plan = gdn.rope_plan(64, 1e4, sections=[16, 16])

    def call(plan=plan, io=1, x=h.p, ldx=256, pos=h.p, T=2, H=2, D=128, out=h.p + 4096, ldo=256):
        return gdn.lib().gdn_rope(None if plan is None else ctypes.byref(plan), io, x, ldx, pos, T, H, D, 0, out, ldo, None)

    refused(call(plan=None), "plan")
    refused(call(io=2), "io_dtype", -2)
    refused(call(x=None), "x is NULL")
    refused(call(x=h.p + 2), "aligned")
    refused(call(out=h.p + 4100), "aligned")
    refused(call(ldx=248), "x:")
    refused(call(ldx=260), "x:")
    refused(call(io=0, ldo=258), "out:")
    refused(call(pos=None), "positions")
    refused(call(pos=h.p + 2), "positions")
    refused(call(T=-1), "num_tokens")
    refused(call(H=0), "num_heads")
    refused(call(D=132, ldx=264, ldo=264), "head_dim", -2)
    refused(call(D=264, ldx=1024, ldo=1024), "head_dim", -2)
    refused(call(D=32), "rotary_dim")
    refused(call(out=h.p, ldo=512), "row pitch")
    bad = gdn.rope_plan(64, 1e4, sections=[16, 16])
    bad.axis[3] = 2
    refused(call(plan=bad), "axis[3]")
    bad.num_axes = 4
    refused(call(plan=bad), "num_axes")
    bad = gdn.rope_plan(64, 1e4)
    bad.rotary_dim = 63
    refused(call(plan=bad), "rotary_dim")
    refused(call(), status=-9)  # valid, but no device here
    assert h.untouched()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the last, valid call of each is for a machine without a GPU")
def test_cache_calls_refusals():
    h = Host()
    L = gdn.lib()
    cfg = gdn.make_attn_config(4, 2, 128, page_size=16)
    cu = np.array([0, 2], np.int32)

    def cache(pool=h.p, table=h.p, lens=h.p, pages=4, width=2):
        return gdn.KvCache(pool, table, lens, pages, width)

    def append(c=cache(), q=h.p, ldq=512, k=h.p, ldk=256, v=h.p, ldv=256, pos=None, cud=h.p, cuh=cu, N=1, qo=h.p,
               ldqo=512, plan=None):
        return L.gdn_kv_append(ctypes.byref(cfg), plan, q, ldq, k, ldk, v, ldv, pos, cud,
                               None if cuh is None else cuh.ctypes.data, N, None if c is None else ctypes.byref(c), qo,
                               ldqo, None)

    def read(c=cache(), ko=h.p, vo=h.p, cuh=cu, N=1):
        return L.gdn_kv_read(ctypes.byref(cfg), h.p, cuh.ctypes.data, N, None if c is None else ctypes.byref(c), ko, vo,
                             None)

    need = gdn.attention_workspace_size(cfg, 2, 1)

    def attn(c=cache(), q=h.p, ldq=512, o=h.p, lse=h.p, ws=h.p, nws=need, cuh=cu, N=1):
        return L.gdn_attention(ctypes.byref(cfg), q, ldq, h.p, cuh.ctypes.data, N,
                               None if c is None else ctypes.byref(c), o, lse, ws, nws, None)

    for call in (append, read, attn):
        refused(call(c=None), "cache")
        refused(call(c=cache(pool=None)), "pool")
        refused(call(c=cache(pool=h.p + 8)), "pool")
        refused(call(c=cache(table=None)), "page_table")
        refused(call(c=cache(table=h.p + 1)), "page_table")
        refused(call(c=cache(lens=None)), "kv_lens")
        refused(call(c=cache(pages=0)), "num_pages")
        refused(call(c=cache(width=0)), "pages_per_seq")
        refused(call(c=cache(width=1 << 28)), "int32")
        refused(call(cuh=np.array([1, 2], np.int32)), "cu_seqlens")
        refused(call(cuh=np.array([0, 2, 1], np.int32), N=2), "decreases")
        refused(call(N=0), "num_seqs")
    refused(append(cuh=None), "cu_seqlens")
    refused(append(q=None), "q_out")
    refused(append(qo=None), "q_out")
    refused(append(k=None), "k is NULL")
    refused(append(v=h.p + 4), "v is not")
    refused(append(ldk=250), "k:")
    refused(append(ldq=256), "q:")
    refused(append(ldqo=520), "row pitch")
    refused(append(pos=h.p + 1), "positions")
    bad = gdn.rope_plan(256, 1e4)
    refused(append(plan=ctypes.byref(bad)), "rotary_dim")
    refused(read(ko=None), "k_out")
    refused(read(vo=h.p + 2), "v_out")
    refused(attn(q=None), "q is NULL")
    refused(attn(ldq=504), "q:")
    refused(attn(o=None), "o is NULL")
    refused(attn(lse=h.p + 2), "lse")
    if need:
        refused(attn(ws=None), "workspace", -3)
        refused(attn(nws=need - 1), "workspace", -3)
        refused(attn(ws=h.p + 16), "aligned", -3)
    for call in (append, read, attn):
        refused(call(), status=-9)
    assert h.untouched()


def test_linear_refusals():
    h = Host()
    L = gdn.lib()

    def lin(io=1, x=h.p, M=2, K=64, w=h.p, N=16, group=64, y=h.p, ws=h.p, nws=1 << 30):
        return L.gdn_linear_q4(io, x, M, K, w, N, group, y, ws, nws, None)

    def pack(c=h.p, s=h.p, b=h.p, N=16, K=64, group=64, out=h.p):
        return L.gdn_q4_pack(c, s, b, N, K, group, out, None)

    for call in (lin, pack):
        refused(call(K=0), "K = 0")
        refused(call(K=60), "K = 60")
        refused(call(N=-1), "N = -1")
        refused(call(group=16), "group", -2)
    refused(lin(io=5), "io_dtype", -2)
    refused(lin(M=-1), "M = -1")
    refused(lin(x=None), "x is NULL")
    refused(lin(x=h.p + 2), "x is not")
    refused(lin(w=h.p + 8), "packed")
    refused(lin(y=None), "y is NULL")
    refused(lin(y=h.p + 1), "y is NULL")
    refused(pack(c=None), "codes")
    refused(pack(s=h.p + 1), "scales")
    refused(pack(out=h.p + 4), "packed")
    size = ctypes.c_size_t()
    assert L.gdn_q4_packed_bytes(16, 60, 64, ctypes.byref(size)) == -1
    assert L.gdn_q4_packed_bytes(16, 64, 64, None) == -1
    with pytest.raises(gdn.GdnError):
        gdn.linear_q4_workspace_size(-1, 16, 64, 64)
    for M in (1, 64, 65, 4096):
        need = gdn.linear_q4_workspace_size(M, 512, 512, 64)
        if need:
            refused(lin(M=M, N=512, K=512, ws=None), "workspace", -3)
            refused(lin(M=M, N=512, K=512, nws=need - 1), "workspace", -3)
            refused(lin(M=M, N=512, K=512, ws=h.p + 128), "aligned", -3)
    assert h.untouched()


def test_packed_bytes_cover_whole_tiles():
    size = ctypes.c_size_t()
    for N, K, group, want in ((16, 64, 64, 4096 + 512 + 512), (129, 72, 64, 2 * (2 * 4096 + 2 * 512 + 512)), (0, 64, 32, 0),
                              (16, 640, 128, 10 * 4096 + 5 * 512 + 512), (16, 72, 32, 2 * 4096 + 4 * 512 + 512)):
        gdn.lib().gdn_q4_packed_bytes(N, K, group, ctypes.byref(size))
        assert size.value == want, (N, K, group)


def test_binding_refuses_host_tensors():
    cfg = gdn.make_attn_config(4, 2, 64, page_size=16)
    x, pos = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32)
    cu, lens = torch.tensor([0, 2], dtype=torch.int32), torch.tensor([2], dtype=torch.int32)
    table, pool = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, gdn.kv_page_bytes(cfg), dtype=torch.uint8)
    for call in (lambda: gdn.rope(gdn.rope_plan(64), x, pos, x),
                 lambda: gdn.kv_append(cfg, None, x, x[:, :2], x[:, 2:], None, cu, [0, 2], lens, pool, table, x),
                 lambda: gdn.kv_read(cfg, cu, [0, 2], lens, pool, table, x, x),
                 lambda: gdn.attention(cfg, x, cu, [0, 2], lens, pool, table, x),
                 lambda: gdn.q4_pack(torch.zeros(4, 32, dtype=torch.uint8), x, x, 64, 64),
                 lambda: gdn.linear_q4(x[0], gdn.Q4Weight(x, 4, 64, 64), x[0])):
        with pytest.raises(gdn.GdnError) as e:
            call()
        assert "CUDA" in str(e.value)


@pytest.mark.parametrize("name", ["attention_prefill.cu", "linear_q4.cu", "tc.cuh"])
def test_aligned_instructions_follow_a_reconvergence(name):
    """All lanes of a warp execute an aligned instruction together: in the source, what only some lanes do (a branch on the
    lane, on rows past the last) is closed by a reconvergence before the next one."""
    path = os.path.join(os.path.dirname(gdn.__file__), "csrc", name)
    lanes = re.compile(r"\b(if|for) \(.*(\blane\b|\btid\b|threadIdx|\(on\)|\bon &&|!on\b|\bn >= a\.N|\bn < a\.N)")
    closed = re.compile(r"__syncwarp|_sync\(0xffffffffu|sync_tc|__syncthreads|mbar_wait_warp|elect_one|"
                        r"tmem_(alloc|dealloc|ld16|ld32|st32)\(")
    aligned = re.compile(r"\b(ld_wait|tmem_ld16_async|tmem_ld32_async|tmem_st16|tmem_st8|tmem_st_16x8|bar_or|bar_sync|"
                         r"group_wait|p_done)\(|\.aligned;")
    since, seen = None, 0
    for i, line in enumerate(open(path), 1):
        line = re.sub(r"//.*|mbar_arrive_if\(.*", "", line)  # (the arrival is predicated, not branched around)
        if "__device__" in line or "__global__" in line:
            since = None
            continue
        if closed.search(line):
            since = None
        if aligned.search(line):
            seen += 1
            assert since is None, f"{name}:{i}: aligned, behind what only some lanes do in line {since}"
        if lanes.search(line) and not aligned.search(line) and "static_assert" not in line:
            since = i
    assert seen >= 3


def test_linear_sizes_past_the_limit_are_refused():
    """Sizes whose rounding up to whole tiles would leave int32."""
    h, L, size = Host(), gdn.lib(), ctypes.c_size_t(7)
    for N, K in ((2 ** 31 - 1, 8), (16, 2 ** 31 - 8), (2 ** 30 + 1, 8), (16, 2 ** 30 + 8)):
        refused(L.gdn_q4_packed_bytes(N, K, 32, ctypes.byref(size)), f"N = {N}", -2)
        refused(L.gdn_q4_pack(h.p, h.p, h.p, N, K, 32, h.p, None), f"N = {N}", -2)
        refused(L.gdn_linear_q4_workspace_size(4, N, K, 32, 1, ctypes.byref(size)), f"N = {N}", -2)
        refused(L.gdn_linear_q4(1, h.p, 4, K, h.p, N, 32, h.p, h.p, 1 << 40, None), f"N = {N}", -2)
    for M in (2 ** 31 - 1, 2 ** 30 + 1):
        refused(L.gdn_linear_q4_workspace_size(M, 16, 64, 64, 1, ctypes.byref(size)), f"M = {M}", -2)
        refused(L.gdn_linear_q4(1, h.p, M, 64, h.p, 16, 64, h.p, h.p, 1 << 40, None), f"M = {M}", -2)
    assert size.value == 7 and h.untouched()
    assert L.gdn_q4_packed_bytes(2 ** 30, 8, 32, ctypes.byref(size)) == 0 and size.value == 2 ** 30 * (32 + 8 + 4)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the valid call is for a machine without a GPU")
def test_table_rows_up_to_the_last_whole_tile_of_int32():
    h, cu = Host(), np.array([0, 1], np.int32)
    cfg = gdn.make_attn_config(1, 1, 64, page_size=16)

    def read(width):
        c = gdn.KvCache(h.p, h.p, h.p, 1, width)
        return gdn.lib().gdn_kv_read(ctypes.byref(cfg), h.p, cu.ctypes.data, 1, ctypes.byref(c), h.p, h.p, None)

    refused(read((2 ** 31 - 16) // 16), "int32")
    refused(read((2 ** 31 - 112) // 16), "int32")
    refused(read((2 ** 31 - 128) // 16), status=-9)  # valid, but no device here


def test_linear_refuses_an_output_over_its_input():
    h = Host()

    def lin(y, io=1, M=4, N=64, K=64):
        return gdn.lib().gdn_linear_q4(io, h.p + 4096, M, K, h.p + 32768, N, 64, h.p + y, h.p, 1 << 30, None)

    for y in (4096, 4096 + 4 * 64 * 2 - 2, 4096 - 4 * 64 * 2 + 2):
        refused(lin(y), "overlaps")
    refused(lin(4096 + 4 * 64 * 4 - 4, io=0), "overlaps")
    if not torch.cuda.is_available():
        for y in (4096 + 4 * 64 * 2, 4096 - 4 * 64 * 2):
            refused(lin(y), status=-9)  # side by side: valid, but no device here
    assert h.untouched()
