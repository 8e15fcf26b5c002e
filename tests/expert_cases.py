"""Inputs and 64-bit references the router, expert and few-token tests share."""
import torch

BLOCK = 128
U = 2.0 ** -24


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def quantised(v, rows):
    """(codes, scales) of v [e, r, c] in blocks of rows x 128, the recipe of the dispatch."""
    e, r, c = v.shape
    rp, cp = -(-r // rows) * rows, -(-c // BLOCK) * BLOCK
    p = torch.nn.functional.pad(v, (0, cp - c, 0, rp - r)).view(e, rp // rows, rows, cp // BLOCK, BLOCK)
    top = p.abs().amax(dim=(2, 4))
    s = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    q = (p / s[:, :, None, :, None]).reshape(e, rp, cp)[:, :r, :c]
    return q.to(torch.float8_e4m3fn).view(torch.uint8).contiguous(), s.contiguous()


def rows_fp8(seed, N, K):
    x = torch.randn((N, K), generator=gen(seed), device="cuda")
    q, s = quantised(x[None], 1)
    return q[0], s[0]


def weights_fp8(seed, E, rows, cols, fan):
    return quantised(torch.randn((E, rows, cols), generator=gen(seed), device="cuda") * fan ** -0.5,
                     BLOCK)


def wide(q, s, rows=BLOCK):
    """float64 values of codes [..., r, c] with scales of rows x 128 blocks."""
    f = q.view(torch.float8_e4m3fn).double()
    s = s.double().repeat_interleave(rows, -2)[..., :q.shape[-2], :]
    return f * s.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def offsets_of(counts):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32, device="cuda")
    o[1:] = torch.tensor(counts, dtype=torch.int64, device="cuda").cumsum(0)
    return o


def product(a, b, counts, transpose):
    """(exact product, product of the magnitudes) in float64, expert by expert."""
    parts, mags, at = [], [], 0
    for e, n in enumerate(counts):
        w = b[e] if transpose else b[e].t()
        parts.append(a[at:at + n] @ w)
        mags.append(a[at:at + n].abs() @ w.abs())
        at += n
    return torch.cat(parts), torch.cat(mags)


def product_bound(mag, K):
    """What fp32 sums may be off by: a block's 128 products within 2^-23 of their magnitudes
    each (a tensor core may truncate instead of rounding), one rounded scale, one fused
    multiply-add for each of the K/128 blocks."""
    return (2 * 128 + K / 128 + 2) * U * mag


def silu(g):
    return g * torch.sigmoid(g)
