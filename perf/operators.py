"""What the attention-side operators and the 4-bit projection do, in plain torch, and the calls that run them.

Four operators: rotary positions over several axes (``rope``), appending rotated keys and values to a paged 4-bit
cache and reading the rows back (``append``), causal attention over that cache (``attention``), and the product with
4-bit weights (``linear``).  ``run`` computes them with elementary torch operations, or, where ``own`` is true,
through ``linear_attention_recurrence_deltanet_b200``.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
THETA = 1e7
LAYOUTS = ("sections", "interleaved", "per_axis")


# ------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of 64 requests: the query heads of one attention layer, text positions
        {"name": "rope decode", "op": "rope", "tokens": 64, "heads": 24, "dim": 128, "rot": 64, "axes": 1,
         "layout": "sections", "io": "bf16", "inverse": False},
        # the gradient through the rotation of a packed batch of video tokens (time, height, width)
        {"name": "rope video gradient", "op": "rope", "tokens": 16384, "heads": 26, "dim": 128, "rot": 128, "axes": 3,
         "layout": "interleaved", "io": "bf16", "inverse": True},
        # the cache write of one decode step of 64 requests at ragged context lengths
        {"name": "append decode", "op": "append", "seqs": 64, "new_min": 1, "new_max": 1, "ctx_min": 1,
         "ctx_max": 8192, "q_heads": 24, "kv_heads": 2, "dim": 128, "page": 64, "rot": 64, "axes": 1,
         "layout": "sections", "io": "bf16", "pick": 1},
        # the cache write of a packed prefill: 16 prompts, 1 .. 2048 tokens, image and text positions
        {"name": "append prefill", "op": "append", "seqs": 16, "new_min": 1, "new_max": 2048, "ctx_min": 0,
         "ctx_max": 1024, "q_heads": 24, "kv_heads": 2, "dim": 128, "page": 64, "rot": 128, "axes": 3,
         "layout": "interleaved", "io": "bf16", "pick": 2},
        # a decode step of one long request (131072 tokens of context): the cache has to be split over the SMs
        {"name": "attention one long", "op": "attention", "seqs": 1, "new_min": 1, "new_max": 1, "ctx_min": 131071,
         "ctx_max": 131071, "q_heads": 24, "kv_heads": 2, "dim": 128, "page": 64, "io": "bf16", "pick": 3},
        # a decode step of 64 requests at ragged context lengths
        {"name": "attention decode batch", "op": "attention", "seqs": 64, "new_min": 1, "new_max": 1, "ctx_min": 17,
         "ctx_max": 16384, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "io": "bf16", "pick": 4},
        # a round of draft tokens, verified against wide heads
        {"name": "attention drafts", "op": "attention", "seqs": 8, "new_min": 4, "new_max": 4, "ctx_min": 1000,
         "ctx_max": 20000, "q_heads": 16, "kv_heads": 2, "dim": 256, "page": 32, "io": "bf16", "pick": 5},
        # a chunk of a long prompt: 2048 new tokens over 6144 that are cached
        {"name": "attention prefill chunk", "op": "attention", "seqs": 1, "new_min": 2048, "new_max": 2048,
         "ctx_min": 6144, "ctx_max": 6144, "q_heads": 24, "kv_heads": 2, "dim": 128, "page": 64, "io": "bf16",
         "pick": 6},
        # fp32 throughout, as the library's small parity configuration
        {"name": "attention fp32", "op": "attention", "seqs": 3, "new_min": 1, "new_max": 7, "ctx_min": 0,
         "ctx_max": 700, "q_heads": 4, "kv_heads": 2, "dim": 64, "page": 16, "io": "f32", "pick": 7},
        # the up projection of a feed-forward layer for one token
        {"name": "linear one token", "op": "linear", "rows": 1, "in": 5120, "out": 17408, "group": 64, "io": "bf16"},
        # the output projection of a layer for a decode batch
        {"name": "linear decode batch", "op": "linear", "rows": 64, "in": 6144, "out": 5120, "group": 128,
         "io": "bf16"},
        # the input projection of a layer for a chunk of a prompt
        {"name": "linear prefill", "op": "linear", "rows": 2048, "in": 5120, "out": 8192, "group": 64, "io": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention", "linear"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "rope":
        dim = rng.choice([64, 72, 80, 128, 256])
        axes = rng.choice([1, 2, 3])
        return {"op": op, "tokens": _log(rng, 1, 12000), "heads": _log(rng, 1, 16 if dim > 128 else 26), "dim": dim,
                "rot": rng.choice([d for d in (32, 64, 72, 128, 256, 60) if d <= dim]), "axes": axes,
                "layout": rng.choice(LAYOUTS), "io": io, "inverse": rng.random() < 0.5}
    if op in ("append", "attention"):
        qh, kvh, dim = rng.choice([(24, 2, 128), (32, 8, 128), (16, 2, 256), (12, 12, 64), (8, 1, 128), (14, 2, 64),
                                   (40, 2, 64), (6, 2, 256)])
        c = {"op": op, "q_heads": qh, "kv_heads": kvh, "dim": dim, "page": rng.choice([16, 32, 48, 64, 128]),
             "io": io, "pick": rng.randrange(1 << 20)}
        if op == "append":
            n = _log(rng, 1, 48)
            top = max(1, 12000 // n if dim < 256 else 6000 // n)
            c |= {"seqs": n, "new_min": rng.choice([0, 1, 1]), "new_max": _log(rng, 1, top), "ctx_min": 0,
                  "ctx_max": _log(rng, 1, 4000), "axes": rng.choice([1, 2, 3]), "layout": rng.choice(LAYOUTS),
                  "rot": rng.choice([0, dim // 4, dim // 2, dim])}
            return c
        n = _log(rng, 1, 64)
        new = rng.choice([1, 1, rng.randint(2, 4), _log(rng, 5, 1200)])
        new = new if new <= 4 else max(5, min(new, 4800 // n))
        # keys: within 64 * 16384 * 8 heads in all, and scores within 24 * 2048 * 8192
        top = min(131072, 64 * 16384 * 8 // (n * kvh), 24 * 2048 * 8192 // (n * qh * new))
        top = top * 128 // max(dim, 128) // (4 if io == "f32" else 1)
        c |= {"seqs": n, "new_min": new if new <= 4 else 1, "new_max": new, "ctx_min": 0,
              "ctx_max": _log(rng, 1, max(2, top))}
        return c
    group = rng.choice([32, 64, 128])
    rows = rng.choice([1, _log(rng, 2, 64), _log(rng, 65, 1500)])
    k = 8 * _log(rng, 8, 2176 if rows < 65 else 640)
    return {"op": op, "rows": rows, "in": k, "out": _log(rng, 48, 17408 if rows < 65 else 6000), "group": group,
            "io": io if rows < 300 else "bf16"}


# ---------------------------------------------------------------------------------------------------- geometry
def _dtype(case):
    return torch.bfloat16 if case["io"] == "bf16" else torch.float32


def _lens(case):
    """(new tokens, tokens in the cache before them) of every sequence: ragged, spread over the logarithm."""
    r = random.Random(case["pick"])
    new, ctx = [], []
    for _ in range(case["seqs"]):
        for lo, hi, to in ((case["new_min"], case["new_max"], new), (case["ctx_min"], case["ctx_max"], ctx)):
            x = int(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 1)))) - 1
            to.append(min(hi, max(lo, x)))
    if case["seqs"] > 1 or max(new) == 0:
        new[-1], ctx[-1] = case["new_max"], case["ctx_max"]
    return new, ctx


def _v_group(dim):
    return min(dim, 128)


def _sections(case):
    """Frequency pairs of each axis: in halves and quarters, the first axis the largest."""
    half, axes = case["rot"] // 2, case["axes"]
    if axes == 1 or half < 4:
        return [half] + [0] * (axes - 1)
    small = half // (axes + 1) if axes == 3 else half // 2
    return [half - small * (axes - 1)] + [small] * (axes - 1)


def _frequencies(case):
    """(inverse frequency, axis) of every pair, as lists."""
    half, sec = case["rot"] // 2, _sections(case)
    inv, axis = [], []
    for j in range(half):
        if case["layout"] == "interleaved" and case["axes"] > 1:
            a = j % 3
            a = a if 0 < a < len(sec) and j < 3 * sec[a] else 0
        else:
            a, edge = 0, sec[0]
            while j >= edge:
                a += 1
                edge += sec[a]
        if case["layout"] == "per_axis":
            local, width = j - sum(sec[:a]), sec[a]
        else:
            local, width = j, half
        inv.append(THETA ** (-local / width))
        axis.append(a)
    return inv, axis


# ------------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _grid_positions(tokens, axes, base):
    """Positions of image and video tokens: frames of 18 rows of 32, behind `base` tokens of text (int32 [axes, tokens])."""
    i = torch.arange(tokens, device=DEV)
    ax = [base + i] if axes == 1 else [base + i // 576, base + i // 32 % 18, base + i % 32][:axes]
    return torch.stack(ax).to(torch.int32).contiguous()


def _quantise(x, group):
    """4-bit codes of x [..., dim] in groups: (codes uint8 [..., dim], scale and bias bf16 [..., dim // group])."""
    y = x.float().unflatten(-1, (-1, group))
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    s, b = ((hi - lo) * (1.0 / 15.0)).bfloat16(), lo.bfloat16()
    code = torch.where(s > 0, ((y - b.float()) / s.float()).round().clamp(0, 15), torch.zeros_like(y))
    return code.to(torch.uint8).flatten(-2), s.squeeze(-1), b.squeeze(-1)


def _nibbles(code):
    """Two codes a byte, the even channel in the low half."""
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _values(packed, s, b):
    """fp32 values of 4-bit codes [..., dim / 2] with the scales and biases of their groups [..., groups]."""
    code = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).float()
    code = code.unflatten(-1, (s.shape[-1], -1))
    return (code * s.float().unsqueeze(-1) + b.float().unsqueeze(-1)).flatten(-2)


def _cache_layout(case, new, ctx, g):
    """Page table int32 [seqs, width] over a shuffled pool, and the pool's size in pages."""
    page = case["page"]
    need = [-(-(a + b) // page) for a, b in zip(new, ctx)]
    width, total = max(1, max(need)), sum(need) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(len(need), width, dtype=torch.int32, device=DEV)
    at = 0
    for n, k in enumerate(need):
        table[n, :k] = order[at:at + k]
        at += k
    return table, total


def _own_attn(case):
    import linear_attention_recurrence_deltanet_b200 as gdn
    return gdn, gdn.make_attn_config(case["q_heads"], case["kv_heads"], case["dim"], page_size=case["page"],
                                     io_dtype=case["io"])


def _own_plan(case):
    import linear_attention_recurrence_deltanet_b200 as gdn
    return gdn.rope_plan(case["rot"], THETA, sections=_sections(case), layout=case["layout"]) if case["rot"] else None


def prepare(case, seed):
    g, dt, op = _gen(seed), _dtype(case), case["op"]
    st = {"case": case}
    if op == "linear":
        m, k, n, gr = case["rows"], case["in"], case["out"], case["group"]
        kp = -(-k // gr) * gr
        st["x"] = _randn(g, m, k).to(dt)
        st["code"] = _nibbles(torch.randint(0, 16, (n, kp), generator=g, device=DEV, dtype=torch.uint8))
        st["scale"] = ((0.5 + torch.rand(n, kp // gr, generator=g, device=DEV)) * (0.6 / math.sqrt(k))).bfloat16()
        st["bias"] = (st["scale"].float() * (-7.5 + 0.5 * _randn(g, n, kp // gr))).bfloat16()
        if own:
            import linear_attention_recurrence_deltanet_b200 as gdn
            st["w"] = gdn.q4_pack(st.pop("code"), st.pop("scale"), st.pop("bias"), k, gr)
            st["y"] = torch.empty(m, n, dtype=dt, device=DEV)
            st["ws"] = torch.empty(max(256, gdn.linear_q4_workspace_size(m, n, k, gr, case["io"])), dtype=torch.uint8,
                                   device=DEV)
        return st
    if op == "rope":
        t, h, d = case["tokens"], case["heads"], case["dim"]
        st["x"] = _randn(g, t, h, d).to(dt)
        st["pos"] = _grid_positions(t, case["axes"], int(torch.randint(0, 100000, (1,), generator=g, device=DEV)))
        inv, axis = _frequencies(case)
        st["inv"] = torch.tensor(inv, dtype=torch.float64, device=DEV)
        st["axis"] = torch.tensor(axis, dtype=torch.int64, device=DEV)
        if own:
            st["plan"], st["out"] = _own_plan(case), torch.empty_like(st["x"])
        return st
    new, ctx = _lens(case)
    qh, kvh, d = case["q_heads"], case["kv_heads"], case["dim"]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    t = cu[-1]
    st["cu_host"], st["cu"] = np.array(cu, np.int32), torch.tensor(cu, dtype=torch.int32, device=DEV)
    st["lens"] = torch.tensor([a + b for a, b in zip(new, ctx)], dtype=torch.int32, device=DEV)
    st["table"], pages = _cache_layout(case, new, ctx, g)
    seq = torch.repeat_interleave(torch.arange(len(new), device=DEV), torch.tensor(new, device=DEV), output_size=t)
    st["seq"], st["at"] = seq, (st["lens"][seq] - st["cu"][1:][seq] + torch.arange(t, device=DEV)).long()
    if op == "append":
        # q, k and v are views of the projection's rows, as the layer has them; keys have some large channels
        rows = _randn(g, t, qh + 2 * kvh, d)
        rows[:, qh:qh + kvh, 5::37] *= 6.0
        rows = rows.to(dt)
        st["q"], st["k"], st["v"] = rows[:, :qh], rows[:, qh:qh + kvh], rows[:, qh + kvh:]
        st["pos"] = _grid_positions(t, case["axes"], int(torch.randint(0, 100000, (1,), generator=g, device=DEV)))
        inv, axis = _frequencies(case)
        st["inv"] = torch.tensor(inv, dtype=torch.float64, device=DEV)
        st["axis"] = torch.tensor(axis, dtype=torch.int64, device=DEV)
        if own:
            gdn, st["cfg"] = _own_attn(case)
            st["plan"] = _own_plan(case)
            st["pool"] = torch.zeros(pages, gdn.kv_page_bytes(st["cfg"]), dtype=torch.uint8, device=DEV)
            st["q_out"] = torch.empty(t, qh, d, dtype=dt, device=DEV)
            st["k_out"], st["v_out"] = (torch.empty(t, kvh, d, dtype=dt, device=DEV) for _ in range(2))
        else:
            slots, gv = pages * case["page"], _v_group(d)
            st["kc"], st["vc"] = (torch.zeros(slots, kvh, d // 2, dtype=torch.uint8, device=DEV) for _ in range(2))
            st["ks"], st["kb"] = (torch.zeros(slots, kvh, d // 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
            st["vs"], st["vb"] = (torch.zeros(slots, kvh, d // gv, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        return st
    # attention: the cache as earlier steps have left it
    st["q"] = _randn(g, t, qh, d).to(dt)
    total = int(st["lens"].sum())
    k, v = _randn(g, total, kvh, d), _randn(g, total, kvh, d)
    k[..., 5::37] *= 4.0  # keys have some large channels
    k, v = k.to(dt), v.to(dt)
    lens = st["lens"].tolist()
    if own:
        gdn, cfg = _own_attn(case)
        st["cfg"] = cfg
        st["pool"] = torch.zeros(pages, gdn.kv_page_bytes(cfg), dtype=torch.uint8, device=DEV)
        all_cu = np.concatenate(([0], np.cumsum(lens))).astype(np.int32)
        gdn.kv_append(cfg, None, None, k, v, None, torch.from_numpy(all_cu).to(DEV), all_cu,
                      st["lens"], st["pool"], st["table"], None)
        st["o"] = torch.empty(t, qh, d, dtype=dt, device=DEV)
        st["lse"] = torch.empty(t, qh, dtype=torch.float32, device=DEV)
        st["ws"] = torch.empty(max(256, gdn.attention_workspace_size(cfg, t, len(new))), dtype=torch.uint8, device=DEV)
    else:
        slots, gv = pages * case["page"], _v_group(d)
        of = torch.repeat_interleave(torch.arange(len(lens), device=DEV), st["lens"].long(), output_size=total)
        begin = torch.cumsum(st["lens"].long(), 0) - st["lens"].long()
        at = torch.arange(total, device=DEV) - begin[of]
        slot = st["table"][of, at // case["page"]].long() * case["page"] + at % case["page"]
        for name, x, gr in (("k", k, 64), ("v", v, gv)):
            code, s, b = _quantise(x, gr)
            for key, y in ((name + "c", _nibbles(code)), (name + "s", s), (name + "b", b)):
                st[key] = torch.zeros(slots, *y.shape[1:], dtype=y.dtype, device=DEV)
                st[key][slot] = y
    return st


# -------------------------------------------------------------------------------------------------- plain forms
def _rotate(x, pos, inv, axis, inverse=False):
    """Pairs (j, j + R/2) of x [tokens, heads, dim] turned by pos * inv; angles in 64 bits, products in 32."""
    half = inv.numel()
    angle = pos[axis].double().t() * inv
    c, s = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)
    s = -s if inverse else s
    x = x.float()
    a, b = x[..., :half], x[..., half:2 * half]
    return torch.cat((a * c - b * s, b * c + a * s, x[..., 2 * half:]), -1)


def _plain_append(st):
    case, dt = st["case"], _dtype(st["case"])
    q, k = (_rotate(st[n], st["pos"], st["inv"], st["axis"]) for n in ("q", "k"))
    slot = st["table"][st["seq"], st["at"] // case["page"]].long() * case["page"] + st["at"] % case["page"]
    kc, ks, kb = _quantise(k, 64)
    vc, vs, vb = _quantise(st["v"], _v_group(case["dim"]))
    st["kc"][slot], st["ks"][slot], st["kb"][slot] = _nibbles(kc), ks, kb
    st["vc"][slot], st["vs"][slot], st["vb"][slot] = _nibbles(vc), vs, vb
    return {"q": q.to(dt), "k": _values(st["kc"][slot], st["ks"][slot], st["kb"][slot]).to(dt),
            "v": _values(st["vc"][slot], st["vs"][slot], st["vb"][slot]).to(dt)}


def _plain_attention(st):
    case, dt = st["case"], _dtype(st["case"])
    qh, kvh, d, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    n, width = st["table"].shape
    lens, new = st["lens"].long(), (st["cu"][1:] - st["cu"][:-1]).long()
    span = width * page
    most = max(int(b - a) for a, b in zip(st["cu_host"][:-1], st["cu_host"][1:]))
    j = torch.arange(span, device=DEV)
    slot = st["table"].long()[:, j // page] * page + j % page
    k = _values(st["kc"][slot], st["ks"][slot], st["kb"][slot]).permute(0, 2, 3, 1)  # [seqs, kv heads, dim, span]
    v = _values(st["vc"][slot], st["vs"][slot], st["vb"][slot]).permute(0, 2, 1, 3)
    i = torch.arange(st["q"].shape[0], device=DEV) - st["cu"].long()[st["seq"]]
    q = torch.zeros(n, most, qh, d, device=DEV)
    q[st["seq"], i] = st["q"].float()
    q = q.view(n, most, kvh, qh // kvh, d).permute(0, 2, 3, 1, 4).reshape(n, kvh, -1, d)
    s = (q @ k).view(n, qh, most, span) * (1.0 / math.sqrt(d))
    at = lens.view(n, 1) - new.view(n, 1) + torch.arange(most, device=DEV)  # position of each query
    seen = (j <= at.unsqueeze(-1)) & (j < lens.view(n, 1, 1))
    s = s.masked_fill(~seen.unsqueeze(1), -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    o = (p.view(n, kvh, -1, span) @ v).view(n, qh, most, d) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (total.log() + top).squeeze(-1)
    return {"o": o.permute(0, 2, 1, 3)[st["seq"], i].to(dt).contiguous(),
            "lse": lse.permute(0, 2, 1)[st["seq"], i].contiguous()}


def _plain_linear(st):
    w = _values(st["code"], st["scale"], st["bias"])[:, :st["case"]["in"]]
    return (st["x"].float() @ w.t()).to(_dtype(st["case"]))


def run(st):
    op = st["case"]["op"]
    if own:
        import linear_attention_recurrence_deltanet_b200 as gdn
        if op == "rope":
            gdn.rope(st["plan"], st["x"], st["pos"], st["out"], inverse=st["case"]["inverse"])
            return st["out"]
        if op == "append":
            gdn.kv_append(st["cfg"], st["plan"], st["q"], st["k"], st["v"], st["pos"], st["cu"], st["cu_host"],
                          st["lens"], st["pool"], st["table"], st["q_out"])
            gdn.kv_read(st["cfg"], st["cu"], st["cu_host"], st["lens"], st["pool"], st["table"], st["k_out"],
                        st["v_out"])
            return {"q": st["q_out"], "k": st["k_out"], "v": st["v_out"]}
        if op == "attention":
            gdn.attention(st["cfg"], st["q"], st["cu"], st["cu_host"], st["lens"], st["pool"], st["table"], st["o"],
                          st["lse"], st["ws"])
            return {"o": st["o"], "lse": st["lse"]}
        gdn.linear_q4(st["x"], st["w"], st["y"], st["ws"])
        return st["y"]
    if op == "rope":
        return _rotate(st["x"], st["pos"], st["inv"], st["axis"], st["case"]["inverse"]).to(_dtype(st["case"]))
    return {"append": _plain_append, "attention": _plain_attention, "linear": _plain_linear}[op](st)


# --------------------------------------------------------------------------------------------------------- work
def work(case):
    es = 2 if case["io"] == "bf16" else 4
    if case["op"] == "linear":
        m, k, n, gr = case["rows"], case["in"], case["out"], case["group"]
        return {"bytes": (m * k + m * n) * es + n * k / 2 + 4 * n * -(-k // gr), "flops": 2.0 * m * n * k}
    if case["op"] == "rope":
        x = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 2 * x * es + 4 * case["axes"] * case["tokens"],
                "flops": 3.0 * case["tokens"] * case["heads"] * case["rot"]}
    new, ctx = _lens(case)
    d, qh, kvh, t = case["dim"], case["q_heads"], case["kv_heads"], sum(new)
    row = kvh * (d + 4 * (d // 64 + d // _v_group(d)))  # one token of the cache
    if case["op"] == "append":
        return {"bytes": t * (2 * qh + 2 * kvh) * d * es + 2 * t * row + t * 2 * kvh * d * es + 4 * case["axes"] * t,
                "flops": 3.0 * t * (qh + kvh) * case["rot"] + 10.0 * t * kvh * d}
    pairs = sum(sum(c + i + 1 for i in range(n)) for n, c in zip(new, ctx))
    cached = sum(a + b for a, b in zip(new, ctx) if a)
    return {"bytes": cached * row + t * qh * (2 * d * es + 4), "flops": 4.0 * d * qh * pairs}


# -------------------------------------------------------------------------------------------------------- exact
def _exact_turn(x, pos, case, inverse):
    """The rotation as a complex product, in 64 bits."""
    inv, axis = _frequencies(case)
    half = len(inv)
    x = x.double()
    ph = torch.stack([pos[a].double() * f for f, a in zip(inv, axis)], -1)
    turn = torch.polar(torch.ones_like(ph), -ph if inverse else ph).unsqueeze(1)
    z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn
    return torch.cat((z.real, z.imag, x[..., 2 * half:]), -1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turn(st["x"], st["pos"], case, case["inverse"])
    if case["op"] == "append":
        q = _exact_turn(st["q"], st["pos"], case, False) if case["rot"] else st["q"].double()
        # what 4 bits stand for steps at the codes' borders, so that only inputs of few bits have one value in 64
        # bits: the values of bf16 rows (their quotients are no nearer to a border than 2^-9, or on it)
        v = None
        if case["io"] == "bf16":
            x = st["v"].double().unflatten(-1, (-1, _v_group(case["dim"])))
            lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
            s = ((hi - lo) * float(torch.tensor(1.0 / 15.0))).float().bfloat16().double()
            code = torch.zeros_like(x)
            torch.div(x - lo, s, out=code)
            code = torch.where(s > 0, torch.clamp(torch.round(code), 0.0, 15.0), torch.zeros_like(code))
            v = (lo + s * code).flatten(-2)
        return {"q": q, "k": None, "v": v}
    if case["op"] == "linear":
        n, gr = case["out"], case["group"]
        y = torch.zeros(case["rows"], n, dtype=torch.float64, device=DEV)
        x = torch.nn.functional.pad(st["x"].double(), (0, -case["in"] % gr)).unflatten(-1, (-1, gr))
        for i in range(0, n, 2048):  # group by group sums: s (x . code) + b sum(x)
            c = st["code"][i:i + 2048]
            c = torch.stack((c % 16, c // 16), -1).flatten(-2).double().unflatten(-1, (-1, gr))
            w = c * st["scale"][i:i + 2048].double().unsqueeze(-1)
            y[:, i:i + 2048] = x.flatten(-2) @ w.flatten(-2).t() + x.sum(-1) @ st["bias"][i:i + 2048].double().t()
        return y
    # attention, one sequence and key head at a time
    d, page, grp = case["dim"], case["page"], case["q_heads"] // case["kv_heads"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    lens = st["lens"].tolist()
    for n, length in enumerate(lens):
        a, b = st["cu_host"][n], st["cu_host"][n + 1]
        if a == b or length == 0:
            continue
        at = torch.arange(length, device=DEV)
        slot = st["table"][n, at // page].long() * page + at % page
        hidden = at.unsqueeze(0) > (length - (b - a) + torch.arange(b - a, device=DEV)).unsqueeze(1)
        for h in range(case["kv_heads"]):
            kv = []
            for c in ("k", "v"):
                code = st[c + "c"][slot, h]
                code = torch.stack((code % 16, code // 16), -1).flatten(-2).double()
                s, bias = st[c + "s"][slot, h].double(), st[c + "b"][slot, h].double()
                w = d // s.shape[-1]
                kv.append(code * s.repeat_interleave(w, -1) + bias.repeat_interleave(w, -1))
            for i in range(h * grp, (h + 1) * grp):
                x = st["q"][a:b, i].double() @ kv[0].t() / math.sqrt(d)
                x[hidden] = -math.inf
                lse[a:b, i] = torch.logsumexp(x, -1)
                o[a:b, i] = torch.softmax(x, -1) @ kv[1]
    return {"o": o, "lse": lse}
