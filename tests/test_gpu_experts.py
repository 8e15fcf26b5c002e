"""The experts' products and gradients against 64-bit references.  The bounds
are those of fp32 sums of exact products (expert_cases.product_bound), then one
rounding to the output's type."""
import pytest
import torch

from expert_cases import (BLOCK, U, gen, offsets_of, product, product_bound, quantised, rows_fp8,
                          silu, weights_fp8, wide)

pytestmark = pytest.mark.gpu

# segments: one row, none, ends inside and at tile borders, one long
SEGMENTS = [
    [1], [5], [128], [129, 0, 127], [0, 0, 3, 0], [1, 2, 3, 64, 65, 0, 256, 31], [700], [300, 17, 513],
    [0] * 40 + [2] + [0] * 200 + [33],
]


def m():
    import combine_layout_moe_gb300 as pkg
    return pkg


def check_gemm(counts, K, M, transpose, dtype, seed=0):
    N, E = sum(counts), len(counts)
    a, sa = rows_fp8(seed, N, K)
    b, sb = weights_fp8(seed + 1, E, K, M, K) if transpose else weights_fp8(seed + 1, E, M, K, K)
    err = m().new_error_word()
    out = torch.full((N, M), float("nan"), dtype=dtype, device="cuda")
    m().moe_expert_gemm(a, sa, offsets_of(counts), b, sb, transpose_w=transpose, out_dtype=dtype,
                        out=out, err_word=err)
    assert m().moe_read_error(err) == 0
    ref, mag = product(wide(a, sa, 1), wide(b, sb), counts, transpose)
    bound = product_bound(mag, K) + (ref.abs() * 2.0 ** -8 if dtype == torch.bfloat16 else 0)
    diff = (out.double() - ref).abs()
    assert torch.all(diff <= bound), float((diff - bound).max())


@pytest.mark.parametrize("counts", SEGMENTS)
@pytest.mark.parametrize("transpose", [False, True])
def test_gemm_segments(counts, transpose):
    check_gemm(counts, 384, 272, transpose, torch.bfloat16)


@pytest.mark.parametrize("K,M", [(128, 16), (128, 128), (256, 144), (640, 256), (2048, 400), (1152, 1040),
                                 (7168, 32)])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm_sizes(K, M, transpose, dtype):
    check_gemm([40, 0, 131, 3], K, M, transpose, dtype, seed=3)


def test_gemm_many_tiles():
    """More tiles than the GPU has SMs: every CTA takes several."""
    check_gemm([700, 129, 1024, 1, 640, 0, 333, 257], 256, 4096, False, torch.bfloat16, seed=5)
    check_gemm([700, 129, 1024, 1, 640, 0, 333, 257], 256, 4096, True, torch.bfloat16, seed=6)


def test_gemm_rows_outside_and_bad_offsets():
    K, M = 256, 128
    a, sa = rows_fp8(1, 50, K)
    b, sb = weights_fp8(2, 3, M, K, K)
    out = torch.full((50, M), 7.0, dtype=torch.float32, device="cuda")
    err = m().new_error_word()
    off = torch.tensor([4, 20, 20, 45], dtype=torch.int32, device="cuda")
    m().moe_expert_gemm(a, sa, off, b, sb, out_dtype=torch.float32, out=out, err_word=err)
    assert m().moe_read_error(err) == 0
    assert torch.all(out[:4] == 7.0) and torch.all(out[45:] == 7.0)
    ref, mag = product(wide(a, sa, 1)[4:45], wide(b, sb), [16, 0, 25], False)
    assert torch.all((out[4:45].double() - ref).abs() <= product_bound(mag, K))
    for bad in ([0, 20, 10, 50], [0, 20, 30, 51], [-1, 20, 30, 50]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        m().moe_expert_gemm(a, sa, off, b, sb, err_word=err)
        assert m().moe_read_error(err) == m().MOE_ERRBIT_BAD_INDEX, bad


def test_gemm_wild_rows_stay_in_their_row():
    """NaN codes and infinite scales of one row, and of a row no segment holds,
    reach nothing else; blocks of very different scales add up."""
    K, M = 512, 160
    a, sa = rows_fp8(3, 140, K)
    b, sb = weights_fp8(4, 2, M, K, K)
    sa *= torch.exp2(torch.randint(-40, 41, sa.shape, generator=gen(5), device="cuda").float())
    a[130] = 0x7f
    sa[131] = float("inf")
    off = offsets_of([129, 3])
    a[139] = 0x7f
    out = m().moe_expert_gemm(a, sa, off, b, sb, out_dtype=torch.float32)
    ref, mag = product(wide(a, sa, 1)[:130], wide(b, sb), [129, 1], False)
    assert torch.all((out[:130].double() - ref).abs() <= product_bound(mag, K))
    assert torch.all(torch.isnan(out[130])) and not torch.any(torch.isfinite(out[131]))


def test_gemm_no_rows():
    a, sa = rows_fp8(1, 0, 128)
    b, sb = weights_fp8(2, 2, 32, 128, 128)
    assert m().moe_expert_gemm(a, sa, offsets_of([0, 0]), b, sb).shape == (0, 32)


def half_step(v):
    """Half an E4M3 step around v (largest magnitude 448)."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))).clamp(max=8)
    return torch.exp2(e - 4)


@pytest.mark.parametrize("counts,K,inner", [
    ([1], 128, 128), ([5, 0, 130], 256, 384), ([129, 64, 1, 0, 31], 1024, 256), ([2, 1, 0, 1], 7168, 128),
    ([260, 513], 384, 1152),
])
def test_swiglu(counts, K, inner):
    N, E = sum(counts), len(counts)
    a, sa = rows_fp8(11, N, K)
    b, sb = weights_fp8(12, E, 2 * inner, K, K)
    err = m().new_error_word()
    q, s = m().moe_expert_swiglu(a, sa, offsets_of(counts), b, sb, err_word=err)
    assert m().moe_read_error(err) == 0
    y, mag = product(wide(a, sa, 1), wide(b, sb), counts, False)
    off = product_bound(mag, K)
    g, u, eg, eu = y[:, :inner], y[:, inner:], off[:, :inner], off[:, inner:]
    h = silu(g) * u
    # |silu'| <= 1.1; exp, quotient and product are within eight roundings
    eh = (1.1 * eg + 8 * U * silu(g).abs()) * (u.abs() + eu) + silu(g).abs() * eu
    blocks = h.view(N, -1, BLOCK)
    top = blocks.abs().amax(2)
    etop = eh.view(N, -1, BLOCK).amax(2)
    assert torch.all((s.double() - top / 448).abs() <= etop / 448 + 2 * U * top)
    scale = s.double().repeat_interleave(BLOCK, 1)
    v = h / scale
    code = q.view(torch.float8_e4m3fn).double()
    slack = eh / scale + 4 * U * v.abs()
    assert torch.all((code - v).abs() <= half_step(v.abs() + slack) + slack)
    assert torch.all(code.view(N, -1, BLOCK).abs().amax(2) == 448)


def test_swiglu_zero_rows():
    K, inner = 256, 256
    a, sa = rows_fp8(1, 6, K)
    a[2] = 0
    b, sb = weights_fp8(2, 1, 2 * inner, K, K)
    q, s = m().moe_expert_swiglu(a, sa, offsets_of([6]), b, sb)
    assert torch.all(s[2] == 1) and torch.all(q[2] & 0x7f == 0)


@pytest.mark.parametrize("counts,M,K", [
    ([1], 8, 8), ([5, 0, 64], 136, 72), ([129, 63, 1, 0, 300], 264, 520), ([2000], 128, 384), ([16, 17], 1040, 256),
    ([4097, 3], 256, 256),
])
def test_wgrad(counts, M, K):
    N = sum(counts)
    dy = torch.randn((N, M), generator=gen(21), device="cuda").bfloat16()
    x = torch.randn((N, K), generator=gen(22), device="cuda").bfloat16()
    out = torch.full((len(counts), M, K), float("nan"), device="cuda")
    err = m().new_error_word()
    m().moe_expert_wgrad(dy, x, offsets_of(counts), dw=out, err_word=err)
    assert m().moe_read_error(err) == 0
    at = 0
    for e, n in enumerate(counts):
        p, r = dy[at:at + n].double().t(), x[at:at + n].double()
        assert torch.all((out[e].double() - p @ r).abs() <= 2 * max(n, 1) * U * (p.abs() @ r.abs()))
        at += n


def test_wgrad_rows_outside_and_bad_offsets():
    dy = torch.randn((90, 32), generator=gen(23), device="cuda").bfloat16()
    x = torch.randn((90, 40), generator=gen(24), device="cuda").bfloat16()
    dy[:3] = float("nan")   # rows of no segment, and of another's, reach nothing
    x[70:] = float("inf")
    off = torch.tensor([3, 40, 70, 90], dtype=torch.int32, device="cuda")
    out = m().moe_expert_wgrad(dy, x, off)
    for e, (lo, hi) in enumerate([(3, 40), (40, 70)]):
        p, r = dy[lo:hi].double().t(), x[lo:hi].double()
        assert torch.all((out[e].double() - p @ r).abs() <= 2 * 64 * U * (p.abs() @ r.abs()))
    assert not torch.any(torch.isfinite(out[2]))
    err = m().new_error_word()
    out = m().moe_expert_wgrad(dy, x, torch.tensor([3, 40, 91, 90], dtype=torch.int32, device="cuda"),
                               err_word=err)
    assert m().moe_read_error(err) == m().MOE_ERRBIT_BAD_INDEX
    assert torch.all(out[1] == 0) and torch.all(out[2] == 0)


def test_gradients_against_differences():
    """A linear product's directional differences, in 64 bits, along a random
    direction of its rows and of its weights, against the kernels' gradients."""
    counts, K, M = [9, 0, 30], 256, 128
    N, E = sum(counts), len(counts)
    x = torch.randn((N, K), generator=gen(31), device="cuda").bfloat16()
    dy = torch.randn((N, M), generator=gen(32), device="cuda").bfloat16()
    w, sw = weights_fp8(33, E, M, K, K)
    off = offsets_of(counts)
    dq, ds = quantised(dy.float()[None], 1)
    dx = m().moe_expert_gemm(dq[0], ds[0], off, w, sw, transpose_w=True, out_dtype=torch.float32)
    dw = m().moe_expert_wgrad(dy, x, off)
    w64, x64 = wide(w, sw), x.double()
    dir_x = torch.randn((N, K), generator=gen(34), device="cuda", dtype=torch.float64)
    dir_w = torch.randn((E, M, K), generator=gen(35), device="cuda", dtype=torch.float64)
    dyq = wide(dq[0], ds[0], 1)

    def loss(xx, ww, grad):
        return (product(xx, ww, counts, False)[0] * grad).sum()
    h = 2.0 ** -10
    got = (dx.double() * dir_x).sum()
    want = (loss(x64 + h * dir_x, w64, dyq) - loss(x64 - h * dir_x, w64, dyq)) / (2 * h)
    _, mag = product(dyq, w64, counts, True)
    assert abs(got - want) <= (product_bound(mag, M) * dir_x.abs()).sum() + 1e-9
    got = (dw.double() * dir_w).sum()
    want = (loss(x64, w64 + h * dir_w, dy.double()) - loss(x64, w64 - h * dir_w, dy.double())) / (2 * h)
    mags = torch.stack([dy[lo:hi].double().abs().t() @ x64[lo:hi].abs()
                        for lo, hi in ((0, 9), (9, 9), (9, 39))])
    assert abs(got - want) <= (2 * 30 * U * mags * dir_w.abs()).sum() + 1e-9


def test_products_between_dispatch_and_combine():
    """Router, layout, dispatch, product, combine, and the way back, as a
    training step runs them."""
    T, H, M, E, k = 300, 256, 256, 8, 2
    p = m()
    x = torch.randn((T, H), generator=gen(41), device="cuda").bfloat16()
    logits = torch.randn((T, E), generator=gen(42), device="cuda")
    w, sw = weights_fp8(43, E, M, H, H)
    err = p.new_error_word()
    idx, tw = p.moe_route(logits, k)
    lay, q, s = p.moe_layout_dispatch_quant(x, idx, E, 1, err_word=err)
    y = p.moe_expert_gemm(q, s, lay.expert_offsets, w, sw, err_word=err)
    out = p.moe_combine(y, lay.slot_of, tw, err_word=err)
    counts = lay.expert_counts.tolist()
    ref, mag = product(wide(q, s, 1), wide(w, sw), counts, False)
    assert torch.all((y.double() - ref).abs() <= product_bound(mag, H) + ref.abs() * 2.0 ** -8)
    dout = torch.randn((T, M), generator=gen(44), device="cuda").bfloat16()
    dy, dtw = p.moe_combine_backward(dout, y, lay.slot_of, tw, err_word=err)
    every = torch.arange(T * k, dtype=torch.int32, device="cuda")[:, None]
    dq, ds = p.moe_dispatch_quant(dy, every, err_word=err)
    drecv = p.moe_expert_gemm(dq, ds, lay.expert_offsets, w, sw, transpose_w=True, err_word=err)
    dx = p.moe_dispatch_backward(drecv, lay.slot_of, err_word=err)
    recv = p.moe_dispatch(x, lay.slot_of, err_word=err)
    dw = p.moe_expert_wgrad(dy, recv, lay.expert_offsets, err_word=err)
    dlogits = p.moe_route_backward(idx, tw, dtw, E, err_word=err)
    assert p.moe_read_error(err) == 0
    # the gradients are near those of the unquantised chain: E4M3 is within 2^-4 a value
    xe = x.double()[torch.arange(T, device="cuda").repeat_interleave(k)]
    we = wide(w, sw)[idx.long().flatten()]
    de = (tw.double()[:, :, None] * dout.double()[:, None, :]).view(T * k, M)
    rdx = torch.einsum("nm,nmk->nk", de, we).view(T, k, H).sum(1)
    assert (dx.double() - rdx).norm() / rdx.norm() < 0.05
    rdw = torch.zeros((E, M, H), dtype=torch.float64, device="cuda")
    rdw.index_add_(0, idx.long().flatten(), de[:, :, None] * xe[:, None, :])
    assert (dw.double() - rdw).norm() / rdw.norm() < 0.01
    ye = torch.einsum("nk,nmk->nm", xe, we).view(T, k, M)
    g = (ye * dout.double()[:, None, :]).sum(2)
    wt = tw.double()
    rdl = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(
        1, idx.long(), wt * (g - (wt * g).sum(1, keepdim=True)))
    assert (dlogits.double() - rdl).norm() / rdl.norm() < 0.1
    rout = (ye * wt[:, :, None]).sum(1)
    assert (out.double() - rout).norm() / rout.norm() < 0.05
