"""csa_paged_append / csa_paged_read: rows into and out of a paged cache.

A rotated value is formed in double precision and rounded once: bf16 2^-8,
fp32 2^-24 of it, plus, of the pair's length, 2^-40 for the recurrence's 32
steps and 2^-50 times the position for the frequency's and the angle's rounding
(both sides'). A 4-bit value (c - 8) s is within s / 2 of what it stands for,
(1 + 2^-22) for the fp32 division, or at 7 s where that is larger than 7.5 s."""
import ctypes

import pytest
import torch

import paged_reference as R
from compressed_sparse_attention_15_b200 import _lib, ops
from compressed_sparse_attention_15_b200.build import build

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _append(dev, kv, pages, scales, table, entry0, n_new, rope, ws=None):
    d = lambda t: None if t is None else t.to(dev)  # noqa: E731
    pages, scales = d(pages), d(scales)
    if rope:
        rope = (*rope[:2], d(rope[2]), rope[3])
    out = ops.paged_append(d(kv), pages, scales, d(table), d(entry0), n_new=d(n_new), rope=rope, ws=ws)
    assert out.data_ptr() == pages.data_ptr()
    return pages, scales


def _check_rows(kv, before, after, scales, table, entry0, counts, rope, dtype):
    B, n, D = kv.shape
    pos0 = torch.zeros(B, dtype=torch.int64) if not rope or rope[2] is None else rope[2]
    want = R.rotated(kv, rope, pos0) if rope else kv.double()
    u = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    tol = torch.zeros_like(want)
    if rope:
        r = rope[0]
        pair = kv[..., D - r:].double().unflatten(-1, (-1, 2)).norm(dim=-1).repeat_interleave(2, -1)
        far = float(pos0.max() + n * rope[3])
        tol[..., D - r:] = u * want[..., D - r:].abs() + (2.0 ** -40 + 2.0 ** -50 * far) * pair
    got, old = R.values(after, scales), R.values(*before)
    touched = torch.zeros(old.shape[:2], dtype=torch.bool)
    sc = None if scales is None else R.e4m3(scales.cpu().view(torch.uint8)).repeat_interleave(16, -1)
    page = old.shape[1]
    for b in range(B):
        e = torch.arange(int(entry0[b]), int(entry0[b]) + counts[b])
        at = table[b].long()[e // page], e % page
        touched[at] = True
        err = (got[at] - want[b, :counts[b]]).abs()
        t = tol[b, :counts[b]]
        if sc is not None:
            s, w = sc[at], want[b, :counts[b]].abs()
            t = t + torch.maximum(s / 2, w - 7 * s) * (1 + 2.0 ** -20)
        assert torch.all(err <= t), (b, float((err - t).max()))
    same = ~touched
    assert torch.equal(got[same], old[same]), "a row outside the append changed"


CASES = [
    # B, n, D, page, rope dims, pos0, stride, ragged
    (3, 1, 512, 64, 64, 65535, 4, False),
    (1, 333, 512, 64, 64, 1 << 20, 4, False),
    (4, 37, 128, 17, 8, 5, 1, True),
    (2, 70, 320, 16, 64, 0, 128, True),
    (2, 9, 16, 1, 16, 3, 1, True),
    (1, 5, 1024, 256, 1024, 77, 4, False),
    (3, 129, 576, 48, 0, 0, 0, True),
    (1, 1200, 64, 64, 24, 1 << 31, 1, False),
    (1, 20000, 64, 128, 64, 12345, 4, False),
]


@gpu
@pytest.mark.parametrize("fmt,dtype", [("int4", BF16), ("int4", F32), ("rows", BF16), ("rows", F32)])
@pytest.mark.parametrize("B,n,D,page,rope_dims,pos0,stride,ragged", CASES)
def test_append_and_read(cuda_device, B, n, D, page, rope_dims, pos0, stride, ragged, fmt, dtype):
    g = torch.Generator().manual_seed(B * n + D)
    kv = (torch.randn(B, n, D, generator=g) * 3).to(dtype)
    kv[0, 0, :16] = 0  # a group of zeros
    pages, scales, table = R.make_cache(n, B, n + 7, page, D, fmt, dtype)
    entry0 = torch.randint(0, 7, (B,), generator=g, dtype=torch.int32)
    counts = [[n, 0, 1, n // 2][b % 4] if ragged else n for b in range(B)]
    n_new = torch.tensor(counts, dtype=torch.int32) if ragged else None
    rope = (rope_dims, 160000.0, pos0 + 1000 * torch.arange(B), stride) if rope_dims else None
    ws = ops.Workspace(cuda_device)
    a_pages, a_scales = _append(cuda_device, kv, pages, scales, table, entry0, n_new, rope, ws)
    assert ws.status() == 0
    _check_rows(kv, (pages, scales), a_pages.cpu(), None if a_scales is None else a_scales.cpu(), table, entry0, counts,
                rope, dtype)
    # read back: the values exactly, rows past the count untouched
    out = torch.full((B, n + 3, D), 9.0, dtype=dtype, device=cuda_device)[:, :n]
    got = ops.paged_read(a_pages, a_scales, table.to(cuda_device), entry0.to(cuda_device), n,
                         n_new=None if n_new is None else n_new.to(cuda_device), out=out, ws=ws)
    assert ws.status() == 0 and got.data_ptr() == out.data_ptr()
    vals = R.values(a_pages, a_scales)
    for b in range(B):
        e = torch.arange(int(entry0[b]), int(entry0[b]) + counts[b])
        assert torch.equal(got[b, :counts[b]].cpu().double(), R.entries(vals, table, b, e))
        assert torch.all(got[b, counts[b]:] == 9)


@gpu
def test_codes_of_bf16_rows_are_the_formula_s(cuda_device):
    # quotients of bf16 values by E4M3 scales are ties or far from them: the codes have to be equal
    g = torch.Generator().manual_seed(1)
    kv = (torch.randn(1, 400, 64, generator=g) * torch.logspace(-4, 5, 400)[:, None]).to(BF16)
    pages, scales, table = R.make_cache(1, 1, 400, 64, 64, "int4", BF16)
    p, s = _append(cuda_device, kv, pages, scales, table, torch.zeros(1, dtype=torch.int32), None, None)
    v = kv[0].float().reshape(400, 4, 16)
    want_s = (v.abs().amax(-1) / torch.full((), 7.0)).clamp(max=448).to(torch.float8_e4m3fn)
    sv = want_s.double()[..., None]
    want = torch.where(sv > 0, (v.double() / sv).round().clamp(-7, 7) * sv, 0.0).reshape(400, 64)
    e = torch.arange(400)
    at = table[0].long()[e // 64], e % 64
    assert torch.equal(s.cpu().view(torch.uint8)[at], want_s.view(torch.uint8))
    assert torch.equal(R.values(p, s)[at], want)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nan_and_infinity(cuda_device, dtype):
    kv = torch.ones(1, 2, 48, dtype=dtype)
    kv[0, 0, 3] = float("nan")
    kv[0, 0, 20] = float("-inf")
    pages, scales, table = R.make_cache(2, 1, 2, 2, 48, "int4", dtype)
    p, s = _append(cuda_device, kv, pages, scales, table, torch.zeros(1, dtype=torch.int32), None, None)
    got = ops.paged_read(p, s, table.to(cuda_device), torch.zeros(1, dtype=torch.int32, device=cuda_device), 2, dtype=F32)
    got = got.cpu()[0]
    assert torch.isnan(got[0, :16]).all()
    assert got[0, 20] == -7 * 448 and torch.all(got[0, 16:20] == 0)
    assert torch.all((got[0, 32:] - 1).abs() <= 1 / 14 + 1e-6) and torch.all((got[1] - 1).abs() <= 1 / 14 + 1e-6)


@gpu
@pytest.mark.parametrize("fmt", ["int4", "rows"])
def test_strided_and_unaligned_rows(cuda_device, fmt):
    g = torch.Generator().manual_seed(4)
    wide = torch.randn(2, 30, 3, 81, generator=g).to(BF16)
    kv = wide[:, :, 1, 1:65]  # an odd base and odd strides
    pages, scales, table = R.make_cache(3, 2, 40, 16, 64, fmt, BF16)
    entry0 = torch.tensor([0, 9], dtype=torch.int32)
    p, s = pages.to(cuda_device), None if scales is None else scales.to(cuda_device)
    ops.paged_append(wide.to(cuda_device)[:, :, 1, 1:65], p, s, table.to(cuda_device), entry0.to(cuda_device),
                     rope=(16, 10000.0, None, 2))
    _check_rows(kv, (pages, scales), p.cpu(), None if s is None else s.cpu(), table, entry0, [30, 30],
                (16, 10000.0, None, 2), BF16)
    base = torch.full((2 * 30 * 64 + 1,), 9.0, dtype=BF16, device=cuda_device)
    out = base[1:].view(2, 30, 64)
    ops.paged_read(p, s, table.to(cuda_device), entry0.to(cuda_device), 30, out=out)
    assert base[0] == 9
    vals = R.values(p, s)
    for b in range(2):
        assert torch.equal(out[b].cpu().double(), R.entries(vals, table, b, torch.arange(30) + int(entry0[b])))


@gpu
@pytest.mark.parametrize("fmt", ["int4", "rows"])
def test_bad_pages_entries_and_counts_are_skipped_and_reported(cuda_device, fmt):
    pages, scales, table = R.make_cache(5, 3, 8, 4, 32, fmt, BF16)
    table[1, 1] = pages.shape[0]  # outside the pool
    kv = torch.full((3, 6, 32), 2.0, dtype=BF16)
    entry0 = torch.tensor([5, 0, -2], dtype=torch.int32)
    n_new = torch.tensor([6, 6, 6], dtype=torch.int32)
    ws = ops.Workspace(cuda_device)
    p, s = _append(cuda_device, kv, pages, scales, table, entry0, n_new, None, ws)
    assert ws.status() == 2 | 16  # entries 8.. of sequence 0, -2, -1 of sequence 2; page 1 of sequence 1
    vals, old = R.values(p, s), R.values(pages, scales)
    wrote = {(0, e) for e in (5, 6, 7)} | {(1, e) for e in range(4)} | {(2, e) for e in range(4)}
    touched = torch.zeros(old.shape[:2], dtype=torch.bool)
    for b, e in wrote:
        at = int(table[b, e // 4]), e % 4
        touched[at] = True
        assert torch.all((vals[at] - 2).abs() <= 2 / 14 + 1e-6)
    assert torch.equal(vals[~touched], old[~touched])
    dev = cuda_device
    out = torch.full((3, 6, 32), 9.0, dtype=BF16, device=dev)
    ops.paged_read(p, s, table.to(dev), entry0.to(dev), 6, n_new=torch.tensor([7, -1, 6], dtype=torch.int32, device=dev),
                   out=out, ws=ws)
    assert ws.status() == 1 | 2
    assert torch.all(out[0, 3:] == 9) and torch.all(out[1] == 9) and torch.all(out[2, :2] == 9)
    assert torch.all(out[2, 2:] != 9)


@gpu
def test_captured_append_follows_its_inputs(cuda_device):
    dev = cuda_device
    pages, scales, table = R.make_cache(6, 2, 64, 16, 512, "int4", BF16)
    kv = torch.zeros(2, 1, 512, dtype=BF16, device=dev)
    p, s, t = pages.to(dev), scales.to(dev), table.to(dev)
    e0 = torch.zeros(2, dtype=torch.int32, device=dev)
    pos = torch.zeros(2, dtype=torch.int64, device=dev)
    out = torch.zeros(2, 1, 512, dtype=BF16, device=dev)
    ws = ops.Workspace(dev)

    def step():
        ops.paged_append(kv, p, s, t, e0, rope=(64, 160000.0, pos, 4), ws=ws)
        ops.paged_read(p, s, t, e0, 1, out=out, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.Generator().manual_seed(8)
    for i in range(5):
        new = torch.randn(2, 1, 512, generator=g).to(BF16)
        kv.copy_(new)
        e0.fill_(13 * i)
        pos.fill_(1000 * i)
        graph.replay()
        vals = R.values(p, s)
        for b in range(2):
            row = R.entries(vals, table, b, [13 * i])
            assert torch.equal(out[b].cpu().double(), row)
            want = R.rotated(new[b:b + 1], (64, 160000.0, None, 4), torch.tensor([1000 * i]))[0]
            sc = want.abs().reshape(1, 32, 16).amax(-1).repeat_interleave(16, -1) / 7 * (1 + 1 / 16)
            assert torch.all((row - want).abs() <= sc * 0.5 * (1 + 2.0 ** -6) + 2.0 ** -8 * want.abs())


@gpu
def test_offsets_beyond_32_bits(cuda_device):
    # a pool of more than 2^32 bytes of rows: the last page, and one in the middle
    D, page = 1024, 64
    num = (1 << 32) // (2 * D * page) + 40
    pages = torch.empty(num, page, D, dtype=BF16, device=cuda_device)
    table = torch.tensor([[num - 1, num // 2 + 1]], dtype=torch.int32, device=cuda_device)
    kv = torch.randn(1, 100, D, dtype=BF16, device=cuda_device)
    e0 = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    ops.paged_append(kv, pages, None, table, e0)
    assert torch.equal(pages[num - 1], kv[0, :64]) and torch.equal(pages[num // 2 + 1, :36], kv[0, 64:])
    assert torch.equal(ops.paged_read(pages, None, table, e0, 100), kv)


@gpu
def test_empty_calls(cuda_device):
    pages, scales, table = (t.to(cuda_device) for t in R.make_cache(7, 2, 8, 4, 32, "int4", BF16))
    e0 = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    before = pages.clone()
    ops.paged_append(torch.zeros(2, 0, 32, dtype=BF16, device=cuda_device), pages, scales, table, e0)
    assert ops.paged_read(pages, scales, table, e0, 0).shape == (2, 0, 32)
    assert ops.paged_read(pages, scales, table[:0], e0[:0], 5).shape == (0, 5, 32)
    assert torch.equal(pages, before)


def test_entry_points_refuse_bad_arguments():
    build()
    L = _lib.lib()
    N, P = ctypes.c_void_p(0), ctypes.c_void_p(4096)  # P is never dereferenced
    odd = ctypes.c_void_p(4097)

    def append(kv=P, rs=0, ss=0, pages=P, sc=P, table=P, e0=P, nn=N, B=2, n=3, D=64, np_=5, page=16, per=2, rope=0,
               theta=1e4, pos0=N, ps=1, dt=1, cd=3, ws=P, wb=256):
        return L.csa_paged_append(kv, rs, ss, pages, sc, table, e0, nn, B, n, D, np_, page, per, rope, theta, pos0, ps, dt,
                                  cd, ws, wb, N)

    bad = [dict(kv=N), dict(pages=N), dict(sc=N), dict(table=N), dict(e0=N), dict(B=-1), dict(n=-1), dict(D=0), dict(D=8),
           dict(D=24), dict(D=4112), dict(np_=0), dict(page=0), dict(per=0), dict(per=1 << 20, page=1 << 12), dict(dt=2),
           dict(dt=3), dict(cd=1), dict(cd=1, sc=N, dt=0), dict(cd=2, sc=N), dict(rs=63), dict(ss=-1), dict(rope=-8),
           dict(rope=12), dict(rope=72), dict(rope=8, theta=1.0), dict(rope=8, ps=-1), dict(rope=8, D=65, cd=1, sc=N),
           dict(pos0=ctypes.c_void_p(4100)), dict(kv=odd), dict(pages=ctypes.c_void_p(4100)), dict(table=odd), dict(e0=odd),
           dict(nn=odd), dict(cd=1, sc=N, pages=odd)]
    for kw in bad:
        assert append(**kw) == 1, kw
    assert append(ws=N) == 3 and append(wb=255) == 3 and append(ws=ctypes.c_void_p(4100)) == 3
    assert append(B=0) == 0 and append(n=0, kv=N) == 0

    def read(out=P, ss=0, sc=P, cd=3, n=3, B=2, D=64):
        return L.csa_paged_read(P, sc, P, P, N, out, ss, B, n, D, 5, 16, 2, 1, cd, P, 256, N)

    for kw in (dict(out=N), dict(out=odd), dict(ss=191), dict(sc=N), dict(cd=0, sc=N), dict(n=-1), dict(D=40)):
        assert read(**kw) == 1, kw
    assert read(n=0, out=N) == 0


def test_wrappers_refuse_host_tensors():
    pages, scales, table = R.make_cache(9, 2, 8, 4, 32, "int4", BF16)
    e0 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.paged_append(torch.zeros(2, 3, 32, dtype=BF16), pages, scales, table, e0)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ops.paged_read(pages, scales, table, e0, 3)


@gpu
def test_wrappers_refuse_bad_shapes(cuda_device):
    pages, scales, table = (t.to(cuda_device) for t in R.make_cache(9, 2, 8, 4, 32, "int4", BF16))
    z = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype, device=cuda_device)  # noqa: E731
    e0 = z(2, dtype=torch.int32)
    good = dict(kv=z(2, 3, 32), pages=pages, scales=scales, page_table=table, entry0=e0)
    ops.paged_append(**good)
    for kw in (dict(kv=z(1, 3, 32)), dict(kv=z(2, 3, 64)), dict(kv=z(2, 32, 3).transpose(1, 2)),
               dict(kv=z(1, 3, 32).expand(2, 3, 32)), dict(scales=None), dict(scales=scales[:, :, :1]),
               dict(scales=scales[1:]), dict(pages=pages[0]), dict(pages=z(*pages.shape)), dict(page_table=table[0]),
               dict(page_table=table.long()), dict(entry0=z(3, dtype=torch.int32)), dict(entry0=None),
               dict(n_new=z(2, dtype=torch.int64)), dict(rope=(8, 1e4, z(3, dtype=torch.int64), 1)),
               dict(kv=z(2, 3, 32, dtype=torch.float16)), dict(pages=pages[:, ::2], scales=scales[:, ::2])):
        with pytest.raises((ValueError, TypeError)):
            ops.paged_append(**{**good, **kw})
    with pytest.raises((ValueError, TypeError)):
        ops.paged_read(pages, scales, table, e0, 3, out=z(2, 4, 32))
    with pytest.raises((ValueError, TypeError)):
        ops.paged_read(pages, scales, table, e0, 3, out=z(2, 3, 64)[:, :, :32])


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_infinity_in_front_of_a_rotation_inside_its_group(cuda_device, dtype):
    # dims 32 .. 39 are not rotated and share their scale with 40 .. 47, which are
    kv = torch.ones(1, 2, 64, dtype=dtype)
    kv[0, 0, 33], kv[0, 1, 38] = float("inf"), float("-inf")
    pages, scales, table = R.make_cache(11, 1, 2, 2, 64, "int4", dtype)
    e0 = torch.zeros(1, dtype=torch.int32)
    p, s = _append(cuda_device, kv, pages, scales, table, e0, None, (24, 10000.0, None, 3))
    got = ops.paged_read(p, s, table.to(cuda_device), e0.to(cuda_device), 2, dtype=F32).cpu()[0]
    want = torch.zeros(2, 16)
    want[0, 1], want[1, 6] = 7 * 448, -7 * 448
    assert torch.equal(got[:, 32:48], want)
    assert torch.isfinite(got).all()


def test_append_refuses_an_infinite_base():
    build()
    N, P = ctypes.c_void_p(0), ctypes.c_void_p(4096)  # P is never dereferenced
    for theta in (float("inf"), float("nan")):
        assert _lib.lib().csa_paged_append(P, 0, 0, P, P, P, P, N, 2, 3, 64, 5, 16, 2, 8, theta, N, 1, 1, 3, P, 256, N) == 1


@gpu
@pytest.mark.parametrize("fmt", ["int4", "rows"])
@pytest.mark.parametrize("rope", [None, (24, 10000.0, None, 1)])
def test_rows_of_one_append_at_the_same_place(cuda_device, fmt, rope):
    # Sequences 0 and 1 share their first page, and write to it with scales 1,000 apart: what is left there is a
    # mixture of the two; their other pages hold their own rows.
    D, page, n = 64, 8, 16
    g = torch.Generator().manual_seed(12)
    kv = torch.randn(2, n, D, generator=g)
    kv[1] *= 1000
    kv = kv.to(BF16)
    pages, scales, table = R.make_cache(12, 2, n, page, D, fmt, BF16)
    apart = _append(cuda_device, kv, pages, scales, table, torch.zeros(2, dtype=torch.int32), None, rope)
    shared = table.clone()
    shared[1, 0] = shared[0, 0]
    got = _append(cuda_device, kv, pages, scales, shared, torch.zeros(2, dtype=torch.int32), None, rope)
    rows = [[None if t is None else t.cpu().view(torch.uint8 if fmt == "int4" else torch.int16)[table[b, 0].long()] for t in apart]
            for b in range(2)]
    there = [None if t is None else t.cpu().view(torch.uint8 if fmt == "int4" else torch.int16)[table[0, 0].long()] for t in got]
    if fmt == "int4":  # 8 bytes of codes at a time
        one, two, left = (t[0].view(torch.int64) for t in (*rows, there))
        assert torch.all((there[1] == rows[0][1]) | (there[1] == rows[1][1]))
    else:
        one, two, left = (t[0] for t in (*rows, there))
    assert torch.all((left == one) | (left == two))
    for a, b, before in zip(apart, got, (pages, scales)):
        if a is not None:
            a, b, before = (t.cpu().view(torch.uint8) for t in (a, b, before))
            for i in (0, 1):
                assert torch.equal(a[table[i, 1]], b[table[i, 1]])
            untouched = [p for p in range(len(a)) if p not in table[:, 1].tolist() + [int(table[0, 0])]]
            assert torch.equal(b[untouched], before[untouched])


def _nearest_e4m3(q):
    """The E4M3 value nearest to q (64 bits), ties to the even one, at most 448."""
    step = torch.ldexp(torch.ones_like(q), torch.frexp(q)[1].clamp(min=-5) - 4)
    return (torch.round(q / step) * step).clamp(max=448)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("unaligned", [False, True])
@pytest.mark.parametrize("D,rope_dims", [(64, 0), (64, 24), (512, 64), (320, 8), (1024, 1024), (4096, 264)])
def test_scales_are_those_of_the_stored_values(cuda_device, D, rope_dims, dtype, unaligned):
    # Every group has a size of its own (1,000 between the largest and the smallest), so that a maximum over another
    # group, or over values before they are rotated, is far off. The rotated values' rounding and recurrence move a
    # group's maximum by a factor within 1 +- u, the fp32 division by 1 +- 2^-24, and E4M3 keeps order: the stored
    # scale lies between the E4M3 values nearest to the two ends, and is the one nearest where nothing is rotated.
    B, n, page = 2, 40, 16
    g = torch.Generator().manual_seed(D + rope_dims)
    size = torch.exp(torch.rand(B, n, D // 16, 1, generator=g) * 6.9 - 3.45)
    kv = (torch.randn(B, n, D // 16, 16, generator=g) * size).reshape(B, n, D).to(dtype)
    pages, scales, table = R.make_cache(13, B, n, page, D, "int4", dtype)
    rope = (rope_dims, 160000.0, torch.tensor([17, 70000]), 4) if rope_dims else None
    moved = torch.cat([torch.zeros(1, dtype=dtype), kv.flatten()]).to(cuda_device)[1:].view(B, n, D)
    given = moved if unaligned else kv.to(cuda_device)
    assert bool(given.data_ptr() % 16) == unaligned
    on = [t.to(cuda_device) for t in (pages, scales, table, torch.zeros(B, dtype=torch.int32))]
    ops.paged_append(given, *on, rope=rope and (*rope[:2], rope[2].to(cuda_device), rope[3]))
    want = R.rotated(kv, rope, rope[2]) if rope else kv.double()
    got = R.e4m3(on[1].cpu().view(torch.uint8))
    u = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    for b in range(B):
        e = torch.arange(n)
        s = got[table[b].long()[e // page], e % page]
        amax = want[b].reshape(n, D // 16, 16).abs().amax(-1)
        turned = torch.arange(D // 16) >= (D - rope_dims) // 16
        # the rotation's own error, of the pair's length (at most 1.5 times the larger of its two): see the top
        off = torch.where(turned, u * (1 + 2.0 ** -20) + 2.0 ** -30, 0.0) + 2.0 ** -24
        lo, hi = _nearest_e4m3(amax / 7 * (1 - off)), _nearest_e4m3(amax / 7 * (1 + off))
        assert torch.all((lo <= s) & (s <= hi))
        if dtype == BF16:
            assert torch.equal(s[:, ~turned], _nearest_e4m3(amax / 7)[:, ~turned])
