"""The paged cache and its attention from their definitions, in 64 bits on the CPU."""
import math

import torch

ORDER = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28])  # bit at which a word holds the nibble of dim 0..7


def e4m3(bits):
    """Values of E4M3 bytes."""
    u = bits.long()
    e, m = (u >> 3) & 15, (u & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.pow(2.0, (e - 7).double()), m * 2.0 ** -9)
    v = torch.where((u & 127) == 127, math.nan, v)
    return torch.where(u > 127, -v, v)


def values(pages, scales):
    """Every cache row [num_pages, page_size, D] as values."""
    pages = pages.cpu()
    if scales is None:
        return pages.double()
    words = pages.contiguous().view(torch.int32).long() & 0xFFFFFFFF
    v = (((words[..., None] >> ORDER) & 15) - 8).double().flatten(-2)
    return v * e4m3(scales.cpu().view(torch.uint8)).repeat_interleave(16, -1)


def rotated(kv, rope, pos0):
    """kv [B, n, D] in 64 bits, rotated (not rounded)."""
    v = kv.cpu().double()
    R, theta, _, stride = rope
    B, n, D = v.shape
    p = pos0.double()[:, None] + torch.arange(n).double() * stride
    ang = p[..., None] * torch.pow(torch.tensor(float(theta), dtype=torch.float64), -torch.arange(R // 2).double() * 2 / R)
    z = torch.view_as_complex(v[..., D - R:].reshape(B, n, R // 2, 2).contiguous())
    z = z * torch.polar(torch.ones_like(ang), ang)
    return torch.cat([v[..., :D - R], torch.view_as_real(z).flatten(-2)], -1)


def attend(q, rows, sink, scale):
    """(out, softmax-weighted mean of |rows|, sum |q| |row| scale) of one query
    [H, D] over rows [R, D] and the sinks [H], all in 64 bits."""
    q = q.double()
    H, D = q.shape
    if rows.shape[0] == 0:
        return torch.zeros(H, D, dtype=torch.float64), torch.zeros(H, D, dtype=torch.float64), 0.0
    x = torch.cat([q @ rows.T * scale, sink.double()[:, None]], -1)
    p = torch.softmax(x, -1)[:, :-1]
    return p @ rows, p @ rows.abs(), float((q.abs() @ rows.abs().T).max() * abs(scale))


def check_attention(out, refs, dtype, n_rows):
    """out [Q, H, D] against attend()'s triples, one a query.

    With u half a step of dtype (bf16 2^-8, fp32 2^-24), a logit's error d is at
    most D 2^-23 sum|q||row| scale (fp32 accumulation, truncated at worst) plus
    4 2^-23 of its size for scale, log2 and exponential; every weight is then off
    by a factor within 1 +- (2 d + u), the same in the sum as in the product, so
    the output by (2 d + u) (A + |out|) with A the weighted mean of |rows|; the
    sums over R rows add (R + 64) 2^-23 A; the output's rounding u |out|."""
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    out = out.cpu().double()
    assert torch.isfinite(out).all()
    for i, (ref, A, s) in enumerate(refs):
        D = ref.shape[-1]
        d = (D + 4) * 2.0 ** -23 * s + 4 * 2.0 ** -23
        tol = (2 * d + u) * (A + ref.abs()) + (n_rows + 64) * 2.0 ** -23 * A + u * ref.abs() + 1e-30
        err = (out[i] - ref).abs()
        assert torch.all(err <= tol), f"query {i}: error {err.max():.3e}, {float((err / tol).max()):.2f} of the tolerance"


def make_cache(seed, B, n_entries, page, D, fmt, dtype, spare=2):
    """A filled cache on the CPU with a shuffled page table: (pages, scales, table)."""
    g = torch.Generator().manual_seed(seed)
    per = -(-n_entries // page)
    total = B * per + spare
    table = torch.randperm(total, generator=g)[:B * per].reshape(B, per).to(torch.int32)
    if fmt != "int4":
        return torch.randn(total, page, D, generator=g).to(dtype), None, table
    codes = torch.randint(0, 256, (total, page, D // 2), generator=g, dtype=torch.uint8)
    s = (torch.rand(total, page, D // 16, generator=g) * 0.25 + 0.2).to(torch.float8_e4m3fn)
    return codes, s, table


def entries(vals, table, b, idx):
    """Rows of the entries idx of sequence b."""
    page = vals.shape[1]
    idx = torch.as_tensor(idx).long()
    return vals[table[b].long()[idx // page], idx % page]
