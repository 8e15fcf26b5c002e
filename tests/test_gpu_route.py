"""The router and its gradient against a 64-bit implementation.

Weights: exp's argument is one rounded difference (|d| * 2^-24 relative), expf
is within 2 ulp, the sum of k terms adds at most k roundings and the quotient
one: (|d| + k + 6) * 2^-24 relative."""
import math

import pytest
import torch

from expert_cases import U, gen

pytestmark = pytest.mark.gpu


def m():
    import combine_layout_moe_gb300 as pkg
    return pkg


def reference(logits, k, groups, keep):
    x = logits.double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    T, E = x.shape
    if groups > 1:
        per = x.view(T, groups, E // groups)
        two = per.sort(2, descending=True).values[:, :, :2].sum(2).float()
        two = torch.where(torch.isnan(two), -math.inf, two)
        order = torch.sort(two, dim=1, descending=True, stable=True).indices[:, :keep]
        ok = torch.zeros((T, groups), dtype=torch.bool, device=x.device).scatter_(1, order, True)
        x = torch.where(ok[:, :, None], per, -math.inf).reshape(T, E)
    idx = torch.sort(x + 0.0, dim=1, descending=True, stable=True).indices[:, :k]
    top = x.gather(1, idx)
    d = torch.where(top == top[:, :1], 0.0, top - top[:, :1])
    e = torch.where(top == -math.inf, 0.0, torch.exp(d))
    total = e.sum(1, keepdim=True)
    return idx.int(), torch.where(total > 0, e / total.clamp_min(1e-300), 0.0), d


def check(logits, k, groups=1, keep=1):
    idx, w = m().moe_route(logits, k, groups=groups, topk_groups=keep)
    ridx, rw, d = reference(logits, k, groups, keep)
    assert torch.equal(idx, ridx)
    d = torch.where(torch.isfinite(d), d.abs(), 0.0)
    assert torch.all((w.double() - rw).abs() <= (d + k + 6) * U * rw + 1e-44)
    return idx, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,groups,keep", [
    (1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (3, 7, 7, 1, 1), (129, 33, 5, 1, 1), (1024, 256, 8, 1, 1),
    (77, 1024, 32, 1, 1), (50, 1021, 9, 1, 1), (515, 128, 8, 8, 4), (64, 256, 8, 8, 4),
    (33, 60, 6, 6, 2), (19, 24, 3, 24, 5), (40, 96, 4, 32, 32), (4097, 8, 2, 1, 1),
])
def test_route_matches(T, E, k, groups, keep, dtype):
    logits = torch.randn((T, E), generator=gen(E + k), device="cuda").to(dtype)
    check(logits, k, groups, keep)


@pytest.mark.parametrize("groups,keep", [(1, 1), (4, 2)])
def test_route_masks_ties_and_specials(groups, keep):
    inf = math.inf
    base = torch.randint(-3, 4, (64, 48), generator=gen(1), device="cuda").float()  # many ties
    base[0] = -inf                              # nothing left
    base[1] = torch.finfo(torch.float32).min    # the type's lowest value is a value
    base[2] = -inf
    base[2, 41] = 1.0                           # fewer left than k
    base[3, 5] = inf
    base[3, 17] = inf                           # infinite logits share the weight
    base[4, ::2] = math.nan
    base[5] = 0.0
    base[5, 7::3] = -0.0                        # -0 and +0 tie
    base[6] = math.nan
    base[7:20][torch.rand((13, 48), generator=gen(2), device="cuda") < 0.8] = -inf
    idx, w = check(base, 6, groups, keep)
    assert torch.all(w[0] == 0) and torch.all(w[6] == 0)
    # the one expert left takes all of the weight; by groups its group scores
    # 1 - infinity, ties with the empty ones and loses to the lower ids
    assert torch.all(w[2, 1:] == 0) and w[2, 0] == (1 if groups == 1 else 0)


def test_route_strided_and_unaligned_rows():
    big = torch.randn((65, 203), generator=gen(3), device="cuda")
    for off in (0, 1, 4):
        check(big[:, off:off + 160], 6)
    half = big.bfloat16()
    for off in (0, 1, 2):
        check(half[:, off:off + 64], 4, 4, 2)
    idx, w = m().moe_route(big[:0], 3)
    assert idx.shape == (0, 3) and w.shape == (0, 3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 9, 3), (300, 256, 8), (4097, 8, 2), (70, 1021, 32)])
def test_backward_matches_formula(T, E, k, dtype):
    logits = torch.randn((T, E), generator=gen(T), device="cuda")
    idx, w = m().moe_route(logits, k)
    dw = torch.randn((T, k), generator=gen(T + 1), device="cuda")
    err = m().new_error_word()
    got = m().moe_route_backward(idx, w, dw, E, out_dtype=dtype, err_word=err)
    assert m().moe_read_error(err) == 0
    w64, d64 = w.double(), dw.double()
    s = (w64 * d64).sum(1, keepdim=True)
    ref = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, idx.long(), w64 * (d64 - s))
    # k products and sums, one difference, one product
    mag = torch.zeros_like(ref).scatter_(1, idx.long(), w64 * (d64.abs() + (w64 * d64).abs().sum(1, keepdim=True)))
    bound = (k + 4) * U * mag + (ref.abs() * 2.0 ** -8 if dtype == torch.bfloat16 else 0)
    assert torch.all((got.double() - ref).abs() <= bound + 1e-40)


def test_backward_matches_differences():
    T, E, k, h = 40, 24, 5, 1e-6
    logits = torch.randn((T, E), generator=gen(9), device="cuda")
    dw = torch.randn((T, k), generator=gen(10), device="cuda")
    idx, w = m().moe_route(logits, k)
    got = m().moe_route_backward(idx, w, dw, E).double()
    x = logits.double()
    for e in range(E):
        def loss(step):
            y = x.clone()
            y[:, e] += step
            return (torch.softmax(y.gather(1, idx.long()), 1) * dw.double()).sum(1)
        diff = (loss(h) - loss(-h)) / (2 * h)
        # central difference: h^2 / 6 of the third derivative, and 2^-53 / h of rounding
        assert torch.all((diff - got[:, e]).abs() <= 1e-6)


def test_backward_masked_rows_and_bad_ids():
    logits = torch.full((3, 16), -math.inf, device="cuda")
    logits[1, 4] = 2.0
    idx, w = m().moe_route(logits, 4)
    dw = torch.randn((3, 4), generator=gen(4), device="cuda")
    assert torch.all(m().moe_route_backward(idx, w, dw, 16) == 0)  # one weight of 1 or none
    bad = idx.clone()
    bad[0, 1], bad[2, 3] = 16, -1
    err = m().new_error_word()
    m().moe_route_backward(bad, w, dw, 16, err_word=err)
    assert m().moe_read_error(err) == m().MOE_ERRBIT_BAD_INDEX


def test_route_on_another_stream():
    s = torch.cuda.Stream()
    logits = torch.randn((512, 64), generator=gen(6), device="cuda")
    torch.cuda.synchronize()
    idx, w = m().moe_route(logits, 4, stream=s)
    s.synchronize()
    ridx, rw, _ = reference(logits, 4, 1, 1)
    assert torch.equal(idx, ridx)
