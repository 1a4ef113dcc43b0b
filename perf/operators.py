"""The operators around the paged cache, in their plain form and as the framework calls them.

  norm    h = x + residual, RMS norm of h, out in the input's type or as E4M3 codes with a scale per group
  append  rows into a paged cache (the input's type, or int4 codes with E4M3 scales per 16 dims), rotated on the way
  read    cache rows back as values
  hca     attention over every visible entry of a paged cache + the sliding window + a sink per head
  sparse  the same over a list of selected entries per query

A cache in 4 bits holds 8 dims in a 32-bit word: dims 0, 2, 4, 6 in the nibbles of its low half, dims 1, 3, 5, 7 in those
of its high half; a nibble c and its group's scale s (E4M3) stand for (c - 8) s.
"""
import math

import torch

own = False

GROUP = 16  # dims that share a scale of the int4 cache


def listed():
    d64 = dict(dtype="bf16", D=512, page=64)
    return [
        # the norm in front of an FP8 projection: one decoded token
        dict(name="norm_token", op="norm", rows=1, D=4096, dtype="bf16", residual=True, fp8=True, group=128),
        # the same for a prefill chunk of 4,096 tokens
        dict(name="norm_chunk", op="norm", rows=4096, D=4096, dtype="bf16", residual=True, fp8=True, group=128),
        # the norm of the query latents, unquantised, in 32 bits
        dict(name="norm_latents", op="norm", rows=4097, D=1024, dtype="f32", residual=False, fp8=False, group=0),
        # the entry that each of 32 sequences adds in a decode step at 64K tokens
        dict(name="append_step", op="append", B=32, n=1, fmt="int4", rope=64, pos=65535, stride=4, ragged=False, **d64),
        # the entries of a context of 131,072 tokens at ratio 4
        dict(name="append_context", op="append", B=1, n=32767, fmt="int4", rope=64, pos=7, stride=4, ragged=False, **d64),
        # a ragged batch of prompts into bf16 pages whose size divides nothing
        dict(name="append_ragged", op="append", B=7, n=1021, fmt="bf16", rope=64, pos=1000, stride=1, ragged=True,
             dtype="bf16", D=512, page=48),
        # sequences taken out of the 4-bit cache for the kernels that want bf16 rows
        dict(name="read_context", op="read", B=4, n=8192, fmt="int4", ragged=False, **d64),
        # a few rows, in 32 bits
        dict(name="read_short", op="read", B=3, n=77, fmt="int4", ragged=False, dtype="f32", D=512, page=16),
        # dense attention of one sequence at 1M tokens (8,192 entries of 128 tokens)
        dict(name="hca_token", op="hca", B=1, Q=1, H=64, N=8192, W=128, fmt="int4", ragged=False, **d64),
        # and of a batch of 16
        dict(name="hca_batch", op="hca", B=16, Q=16, H=64, N=8192, W=128, fmt="int4", ragged=False, **d64),
        # the selected 512 of 16,383 entries, 32 sequences at 64K tokens
        dict(name="sparse_step", op="sparse", B=32, Q=32, H=64, N=16383, k=512, W=128, fmt="int4", ragged=False, **d64),
        # the same for 1,024 queries of a prefill chunk over 33,791 entries
        dict(name="sparse_chunk", op="sparse", B=1, Q=1024, H=64, N=33791, k=512, W=128, fmt="int4", ragged=True, **d64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "append", "read", "hca", "sparse"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op == "norm":
        fp8 = rng.random() < 0.5
        group = rng.choice((0, 32, 64, 128, 256)) if fp8 else 0
        D = _log(rng, 2, 64) * 256 if group else _log(rng, 16, 16384)
        rows = _log(rng, 1, max(2, (1 << 24) // D))
        return dict(op=op, rows=rows, D=D, dtype=dtype, residual=rng.random() < 0.6, fp8=fp8, group=group)
    page = rng.choice((1, 16, 17, 48, 64, 64, 128, 256))
    fmt = rng.choice(("int4", "int4", dtype))
    if op in ("append", "read"):
        D = rng.choice((64, 128, 320, 512, 512, 576, 1024))
        B = _log(rng, 1, 64)
        n = _log(rng, 1, max(2, (1 << 24) // (D * B)))
        case = dict(op=op, B=B, n=n, fmt=fmt, ragged=rng.random() < 0.4, dtype=dtype, D=D, page=page)
        if op == "append":
            case |= dict(rope=rng.choice((0, 8, 64)), pos=_log(rng, 1, 1 << 20), stride=rng.choice((1, 4, 128)))
        return case
    small = dtype == "f32"
    D = rng.choice((16, 64, 128, 512)) if small else rng.choice((128, 256, 384, 512, 512, 512))
    H = _log(rng, 1, 16) if small else rng.choice((rng.randint(1, 128), 16, 64, 64, 64, 128))
    B = _log(rng, 1, 64)
    Q = B * rng.choice((1, 1, 1, 2, 3))
    W = rng.choice((0, 1, 128, 128, rng.randint(2, 300)))
    most = 2e9 if small else 8e10  # operations; and the plain form gathers Q (rows + W) D values
    room = int(min(most / (4 * Q * H * D), 3e8 / (Q * D))) - W
    if op == "hca":
        N = min(_log(rng, 1, 16384), max(1, room))
        return dict(op=op, B=B, Q=Q, H=H, N=N, W=W, fmt=fmt, ragged=rng.random() < 0.5, dtype=dtype, D=D, page=page)
    N = min(_log(rng, 8, 40000), int(4e8 / (B * D)))
    k = max(1, min(rng.choice((16, 128, 512, 512, 1024, rng.randint(1, 2048))), room))
    return dict(op=op, B=B, Q=Q, H=H, N=N, k=k, W=W, fmt=fmt, ragged=rng.random() < 0.5, dtype=dtype, D=D, page=page)


_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _layout(c):
    """Entries a sequence's table holds, pages a sequence takes, pages in all (a few spare)."""
    most = c["n"] + 5 if "n" in c else c["N"]
    per = -(-most // c["page"])
    return most, per, c["B"] * per + 3


def _pages(c, g, dev):
    """A cache in use: every page holds rows of unit scale, as a norm leaves them."""
    _, per, total = _layout(c)
    shape = (total, c["page"], c["D"])
    table = torch.randperm(total, generator=g, device=dev)[:c["B"] * per].reshape(c["B"], per).to(torch.int32)
    if c["fmt"] != "int4":
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(_DT[c["fmt"]]), None, table
    codes = torch.randint(0, 256, (*shape[:2], c["D"] // 2), generator=g, device=dev, dtype=torch.uint8)
    # amax / 7 of 16 unit normals: about 0.2 to 0.45
    s = torch.rand((*shape[:2], c["D"] // GROUP), generator=g, device=dev) * 0.25 + 0.2
    return codes, s.to(torch.float8_e4m3fn).view(torch.uint8), table


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(dev)
    g.manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device=dev, dtype=torch.int64).to(torch.int32)

    dt = _DT[c["dtype"]]
    s = dict(case=c)
    if c["op"] == "norm":
        s["x"] = normal(c["rows"], c["D"], dtype=dt)
        s["residual"] = normal(c["rows"], c["D"], dtype=dt) * 2 if c["residual"] else None
        s["weight"] = 1 + 0.1 * normal(c["D"])
        return s
    s["pages"], s["scales"], s["table"] = _pages(c, g, dev)
    B = c["B"]
    if c["op"] in ("append", "read"):
        n = c["n"]
        s["entry0"] = ints(0, 6, B)
        s["n_new"] = ints(0, n + 1, B) if c["ragged"] else None
        if c["op"] == "append":
            s["kv"] = normal(B, n, c["D"], dtype=dt)
            s["pos0"] = (c["pos"] + ints(0, 1000, B)).to(torch.int64)
        s["out"] = torch.zeros((B, n, c["D"]), dtype=dt, device=dev)
        return s
    Q, H, D, N, W = c["Q"], c["H"], c["D"], c["N"], c["W"]
    s["q"] = normal(Q, H, D, dtype=dt)
    s["sink"] = normal(H)
    T = W + 37 if W else 0
    s["kv_win"] = normal(B, T, D, dtype=dt) if W else None
    s["win_end"] = ints(0 if c["ragged"] else W - 1, T, Q) if W else None
    if c["op"] == "hca":
        s["n_cmp"] = ints(0, N + 1, Q) if c["ragged"] else torch.full((Q,), N, dtype=torch.int32, device=dev)
    else:
        k = c["k"]
        # distinct entries, ascending, unused slots (-1) last, as the selection writes them
        pick = torch.rand((Q, N), generator=g, device=dev).topk(min(k, N), dim=1).indices
        if k > N:
            pick = torch.cat([pick, torch.full((Q, k - N), N, device=dev)], dim=1)
        if c["ragged"]:
            pick = torch.where(torch.arange(k, device=dev) < ints(0, k + 1, Q)[:, None], pick, N)
        pick = pick.sort(dim=1).values
        s["idx"] = torch.where(pick < N, pick, -1).to(torch.int32).contiguous()
    return s


# ------------------------------------------------------------------ plain forms

def _over(v, d):
    """v / d, divided: by a plain number torch would multiply by 1 / d, which misses ties by a rounding."""
    return v / torch.full_like(v, d)


def _unpack(codes, scales):
    """int4 codes [..., D / 2] and E4M3 scales [..., D / 16] -> values in 32 bits [..., D]."""
    b = codes.reshape(*codes.shape[:-1], -1, 4)
    lo, hi = b & 15, b >> 4
    # the word's nibbles in the order of their dims 0..7
    nib = torch.stack([lo[..., 0], lo[..., 2], hi[..., 0], hi[..., 2], lo[..., 1], lo[..., 3], hi[..., 1], hi[..., 3]], -1)
    v = nib.reshape(*codes.shape[:-1], -1, GROUP).float() - 8
    return (v * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _pack(v):
    """Values in 32 bits [..., D] -> int4 codes [..., D / 2], E4M3 scales [..., D / 16]."""
    v = v.reshape(*v.shape[:-1], -1, GROUP)
    scales = _over(v.abs().amax(-1), 7.0).clamp(max=448).to(torch.float8_e4m3fn)
    s = scales.float()[..., None]
    c = torch.where(s > 0, (v / s).round().clamp(-7, 7) + 8, 8.0).to(torch.uint8)
    w = c.reshape(*c.shape[:-2], -1, 8)
    lo, hi = w[..., [0, 4, 1, 5]], w[..., [2, 6, 3, 7]]
    return (lo | hi << 4).flatten(-2), scales.view(torch.uint8)


def _slots(s, entry):
    """Rows of the flattened pages that hold entries [B, n] of each sequence."""
    page = s["case"]["page"]
    return torch.gather(s["table"].long(), 1, entry // page) * page + entry % page


def _rows(s, slots):
    """Values in 32 bits of the cache rows `slots`."""
    flat = s["pages"].flatten(0, 1)[slots]
    return flat.float() if s["scales"] is None else _unpack(flat, s["scales"].flatten(0, 1)[slots])


def _norm(s):
    c, x = s["case"], s["x"]
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    f = h.float()
    y = f / torch.sqrt((f * f).mean(-1, keepdim=True) + 1e-6) * s["weight"]
    if c["fp8"]:
        v = y.reshape(c["rows"], -1, c["group"] or c["D"])
        a = v.abs().amax(-1)
        scale = torch.where(a > 0, _over(a, 448.0), 1.0)
        out = (v / scale[..., None]).to(torch.float8_e4m3fn).reshape(y.shape), scale
    else:
        out = (y.to(x.dtype),)
    return out if s["residual"] is None else (*out, h)


def _entries(s):
    c = s["case"]
    i = torch.arange(c["n"], device=s["table"].device)
    live = (i < s["n_new"][:, None]) if c["ragged"] else (i >= 0).expand(c["B"], -1)
    return i, live, _slots(s, s["entry0"].long()[:, None] + i)


def _append(s):
    c, v = s["case"], s["kv"]
    i, live, slots = _entries(s)
    R = c["rope"]
    if R:
        p = (s["pos0"][:, None] + i * c["stride"]).double()
        f = 160000.0 ** (-torch.arange(0, R, 2, device=v.device, dtype=torch.float64) / R)
        cs, sn = torch.cos(p[..., None] * f), torch.sin(p[..., None] * f)
        x = v[..., c["D"] - R:].double().unflatten(-1, (-1, 2))
        y = torch.stack([x[..., 0] * cs - x[..., 1] * sn, x[..., 0] * sn + x[..., 1] * cs], -1)
        v = torch.cat([v[..., :c["D"] - R], y.flatten(-2).to(v.dtype)], -1)
    pages = s["pages"].flatten(0, 1)
    if s["scales"] is None:
        pages[slots[live]] = v[live]
        return s["pages"]
    codes, scales = _pack(v[live].float())
    pages[slots[live]] = codes
    s["scales"].flatten(0, 1)[slots[live]] = scales
    return _read(s)


def _read(s):
    _, live, slots = _entries(s)
    return torch.where(live[..., None], _rows(s, slots).to(s["out"].dtype), s["out"])


def _attend(s):
    c, q = s["case"], s["q"]
    Q, B, W, per = c["Q"], c["B"], c["W"], c["Q"] // c["B"]
    dev = q.device
    if c["op"] == "hca":
        entry = torch.arange(c["N"], device=dev).expand(B, -1)
        rows = _rows(s, _slots(s, entry))[:, None]                                 # [B, 1, N, D]
        live = (entry[:1] < s["n_cmp"][:, None]).reshape(B, per, 1, -1)
    else:
        j = s["idx"].long().reshape(B, -1)
        rows = _rows(s, _slots(s, j.clamp(min=0))).reshape(B, per, c["k"], -1)     # [B, per, k, D]
        live = (j >= 0).reshape(B, per, 1, -1)
    qf = q.float().reshape(B, per, c["H"], -1)
    x = torch.where(live, qf @ rows.transpose(-1, -2) * c["D"] ** -0.5, -math.inf)
    if W:
        t = torch.arange(s["kv_win"].shape[1], device=dev)
        e = s["win_end"].long()[:, None]
        seen = ((t <= e) & (t > e - W)).reshape(B, per, 1, -1)
        win = s["kv_win"].float()[:, None]
        x = torch.cat([x, torch.where(seen, qf @ win.transpose(-1, -2) * c["D"] ** -0.5, -math.inf)], -1)
    sink = s["sink"][:, None]
    m = torch.maximum(x.amax(-1, keepdim=True), sink)
    p = torch.exp(x - m)
    p = p / (p.sum(-1, keepdim=True) + torch.exp(sink - m))
    n = rows.shape[-2]
    out = p[..., :n] @ rows
    if W:
        out = out + p[..., n:] @ win
    return out.reshape(q.shape).to(q.dtype)


# ------------------------------------------------------------------ one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _norm, "append": _append, "read": _read, "hca": _attend, "sparse": _attend}[c["op"]](s)
    from compressed_sparse_attention_15_b200 import ops
    if c["op"] == "norm":
        out = ops.add_rmsnorm(s["x"], s["weight"], residual=s["residual"], fp8=c["fp8"], group=c["group"])
        # the codes as the values they stand for
        return (out[0].view(torch.float8_e4m3fn), *out[1:]) if c["fp8"] else out
    ws = s["ws"] if "ws" in s else s.setdefault("ws", ops.Workspace("cuda"))
    if c["op"] == "append":
        rope = (c["rope"], 160000.0, s["pos0"], c["stride"]) if c["rope"] else None
        ops.paged_append(s["kv"], s["pages"], s["scales"], s["table"], s["entry0"], n_new=s["n_new"], rope=rope, ws=ws)
        if s["scales"] is None:
            return s["pages"]
    if c["op"] in ("append", "read"):
        return ops.paged_read(s["pages"], s["scales"], s["table"], s["entry0"], c["n"], n_new=s["n_new"], out=s["out"], ws=ws)
    scale = c["D"] ** -0.5
    if c["op"] == "hca":
        return ops.paged_hca_mqa(s["q"], s["pages"], s["scales"], s["table"], s["n_cmp"], s["kv_win"], s["win_end"], s["sink"],
                                 scale, c["W"], ws=ws)
    return ops.paged_sparse_mqa(s["q"], s["pages"], s["scales"], s["table"], s["idx"], s["kv_win"], s["win_end"], s["sink"],
                                scale, c["W"], ws=ws)


# ------------------------------------------------------------------ what a pass cannot do without

def _row_bytes(c):
    return c["D"] // 2 + c["D"] // GROUP if c["fmt"] == "int4" else c["D"] * (2 if c["fmt"] == "bf16" else 4)


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "norm":
        n = c["rows"] * c["D"]
        out = n + 4 * (n // (c["group"] or c["D"])) if c["fp8"] else n * e
        return dict(bytes=n * e * (3 if c["residual"] else 1) + out + 4 * c["D"], flops=6 * n)
    part = 0.5 if c["ragged"] else 1.0  # a ragged batch's counts are uniform
    if c["op"] in ("append", "read"):
        n = c["B"] * c["n"] * part
        # an append into 4 bits is read back, as the values that it left
        passes = 2 if c["op"] == "append" and c["fmt"] == "int4" else 1
        return dict(bytes=passes * n * (c["D"] * e + _row_bytes(c)), flops=passes * 4 * n * c["D"])
    Q, B, H, D, W = c["Q"], c["B"], c["H"], c["D"], c["W"]
    rows = Q * (c["k"] if c["op"] == "sparse" else c["N"]) * part
    # a sequence's rows are read once, however many of its queries (or slots) take them
    once = min(rows, B * c["N"]) if c["op"] == "sparse" else rows * B / Q
    win = min(Q * W, B * (W + 37))
    return dict(bytes=once * _row_bytes(c) + win * D * e + 2 * Q * H * D * e, flops=4 * H * D * (rows + Q * W))


# ------------------------------------------------------------------ in 64 bits, from the definition

def _grid_e4m3(v):
    """The E4M3 value nearest to v (ties to the even one), at most 448."""
    e = torch.frexp(v)[1].clamp(min=-5) - 1  # v = m 2^e, m in [1, 2); subnormals share 2^-6
    step = torch.ldexp(torch.ones_like(v), e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _values64(s, page, row):
    """Entries held at (page, row), in 64 bits."""
    if s["scales"] is None:
        return s["pages"][page, row].double()
    words = s["pages"][page, row].contiguous().view(torch.int32).long() & 0xFFFFFFFF
    order = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=words.device)  # bit of dim 0..7's nibble
    v = (((words[..., None] >> order) & 15) - 8).double().flatten(-2)
    u = s["scales"][page, row].long()
    e, m = u >> 3, (u & 7).double()
    scale = torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7).double(), m * 2.0 ** -9)
    return v * scale.repeat_interleave(GROUP, -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        h = s["x"].double()
        total = None
        if s["residual"] is not None:
            total = h + s["residual"].double()
            h = total.to(s["x"].dtype).double()
        y = h * torch.rsqrt(torch.linalg.vector_norm(h, dim=-1, keepdim=True) ** 2 / c["D"] + 1e-6) * s["weight"].double()
        tail = () if total is None else (total,)
        if not c["fp8"]:
            return (y, *tail)
        blocks = y.unflatten(-1, (-1, c["group"] or c["D"]))
        peak = blocks.abs().max(-1).values
        scale = torch.where(peak > 0, peak / 448, torch.ones_like(peak))
        return (_grid_e4m3(blocks / scale[..., None]).flatten(-2), scale, *tail)
    page = c["page"]
    if c["op"] in ("append", "read"):
        e0 = s["entry0"].tolist()
        counts = s["n_new"].tolist() if c["ragged"] else [c["n"]] * c["B"]
        result = s["out"].double()
        held = s["pages"].double() if c["op"] == "append" and s["scales"] is None else None
        for b in range(c["B"]):
            n = counts[b]
            e = torch.arange(e0[b], e0[b] + n, device=s["table"].device)
            at = s["table"][b].long()[e // page], e % page
            if c["op"] == "read":
                result[b, :n] = _values64(s, *at)
                continue
            v = s["kv"][b, :n].double()
            if c["rope"]:
                R, p = c["rope"], s["pos0"][b].double() + c["stride"] * torch.arange(n, device=v.device).double()
                turn = torch.polar(torch.ones((), dtype=torch.float64, device=v.device),
                                   torch.outer(p, torch.pow(160000.0, -torch.arange(R // 2, device=v.device).double() * 2 / R)))
                z = torch.view_as_complex(v[:, c["D"] - R:].reshape(n, R // 2, 2).contiguous()) * turn
                v[:, c["D"] - R:] = torch.view_as_real(z).reshape(n, R)
            if held is not None:
                held[at] = v
                continue
            v = v.to(s["kv"].dtype).double().unflatten(-1, (-1, GROUP))
            sc = _grid_e4m3(v.abs().max(-1, keepdim=True).values / 7)
            result[b, :n] = torch.where(sc > 0, torch.round(v / sc).clamp(-7, 7) * sc, 0.0).flatten(-2)
        return result if held is None else held
    Q, per, W = c["Q"], c["Q"] // c["B"], c["W"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    sink = s["sink"].double()
    if c["op"] == "hca":
        n_cmp = s["n_cmp"].tolist()
    ends = s["win_end"].tolist() if W else None
    for i in range(Q):
        b = i // per
        j = torch.arange(n_cmp[i], device=sink.device) if c["op"] == "hca" else s["idx"][i][s["idx"][i] >= 0].long()
        rows = _values64(s, s["table"][b].long()[j // page], j % page)
        if W:
            rows = torch.cat([rows, s["kv_win"][b, max(0, ends[i] - W + 1):ends[i] + 1].double()])
        logits = torch.cat([s["q"][i].double() @ rows.T / math.sqrt(c["D"]), sink[:, None]], -1)
        out[i] = torch.softmax(logits, -1)[:, :-1] @ rows
    return out
