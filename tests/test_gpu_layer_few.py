"""The few-token layer against a 64-bit reference, its agreement with the
long-batch path, and `MoELayer`, which chooses between them.

Bound: a product of n terms in fp32 (tensor cores may truncate) is within 2 n
2^-24 of its magnitudes' sum, scales add two roundings a term; between the
products h is held in two bf16 terms (2^-17); the output rounds once."""
import pytest
import torch

from expert_cases import U, gen, silu, weights_fp8, wide

pytestmark = pytest.mark.gpu


def m():
    import combine_layout_moe_gb300 as pkg
    return pkg


def make(T, k, H, inner, E, fp8, seed=0, repeat=False):
    g = gen(seed)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    if repeat:
        idx = torch.randint(0, E, (T, k), generator=g, device="cuda").int()
    else:
        idx = torch.rand((T, E), generator=g, device="cuda").topk(k, 1).indices.int()
    w = torch.rand((T, k), generator=g, device="cuda")
    if fp8:
        w13, s13 = weights_fp8(seed + 1, E, 2 * inner, H, H)
        w2, s2 = weights_fp8(seed + 2, E, H, inner, inner)
    else:
        w13 = (torch.randn((E, 2 * inner, H), generator=g, device="cuda") * H ** -0.5).bfloat16()
        w2 = (torch.randn((E, H, inner), generator=g, device="cuda") * inner ** -0.5).bfloat16()
        s13 = s2 = None
    return x, idx, w, w13, s13, w2, s2


def reference(x, idx, w, w13, s13, w2, s2):
    T, H = x.shape
    inner = w2.shape[2]
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    off = torch.zeros_like(out)
    E = w13.shape[0]
    for e in idx.unique().tolist():
        if not 0 <= e < E:
            continue
        t, j = (idx == e).nonzero(as_tuple=True)
        a = wide(w13[e], s13[e]) if s13 is not None else w13[e].double()
        b = wide(w2[e], s2[e]) if s2 is not None else w2[e].double()
        xt, wt = x[t].double(), w[t, j].double()[:, None]
        y, ey = xt @ a.t(), 2 * (H + 2) * U * (xt.abs() @ a.abs().t())
        g, u, eg, eu = y[:, :inner], y[:, inner:], ey[:, :inner], ey[:, inner:]
        h = silu(g) * u
        eh = (1.1 * eg + 8 * U * silu(g).abs()) * (u.abs() + eu) + silu(g).abs() * eu + 2.0 ** -17 * h.abs()
        out.index_add_(0, t, wt * (h @ b.t()))
        off.index_add_(0, t, wt.abs() * (eh @ b.abs().t() + 2 * (inner + 2) * U * ((h.abs() + eh) @ b.abs().t())))
    return out, off + 2 * idx.shape[1] * U * out.abs() + 64 * U * off


def check(args, dtype=torch.bfloat16):
    x, idx, w, w13, s13, w2, s2 = args
    err = m().new_error_word()
    out = m().moe_layer_few(x, idx, w, w13, w2, w13_scales=s13, w2_scales=s2, out_dtype=dtype, err_word=err)
    assert m().moe_read_error(err) == 0
    ref, bound = reference(*args)
    bound = bound * (1 + idx.shape[1]) + (ref.abs() * 2.0 ** -8 if dtype == torch.bfloat16 else 0)
    diff = (out.double() - ref).abs()
    assert torch.all(diff <= bound), float((diff / bound).max())
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,H,inner,E", [
    (1, 1, 128, 128, 1), (1, 8, 1024, 256, 32), (2, 2, 256, 384, 8), (7, 3, 640, 128, 5), (8, 2, 512, 256, 2),
    (17, 8, 256, 640, 64), (33, 2, 384, 512, 4), (64, 8, 256, 256, 256), (64, 1, 128, 256, 1), (61, 8, 1152, 128, 16),
    (16, 32, 256, 128, 40),
])
def test_fp8_weights(T, k, H, inner, E, dtype):
    check(make(T, k, H, inner, E, True, seed=T + k), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,H,inner,E", [
    (1, 1, 8, 8, 1), (1, 2, 1000, 248, 8), (3, 2, 72, 136, 4), (9, 4, 264, 40, 6), (64, 2, 512, 200, 8),
    (64, 8, 136, 128, 8), (40, 1, 1024, 1016, 2),
])
def test_bf16_weights(T, k, H, inner, E, dtype):
    check(make(T, k, H, inner, E, False, seed=T + k), dtype)


@pytest.mark.parametrize("fp8", [True, False])
def test_repeated_experts_and_one_hot_expert(fp8):
    check(make(20, 6, 256, 128, 3, fp8, seed=5, repeat=True))
    args = list(make(64, 8, 256, 128, 9, fp8, seed=6))
    args[1] = torch.full_like(args[1], 4)        # every pair on one expert
    check(args)


@pytest.mark.parametrize("fp8", [True, False])
def test_bad_ids_add_nothing(fp8):
    args = list(make(5, 3, 256, 128, 4, fp8, seed=7))
    args[1][1, 0], args[1][3, 2], args[1][4] = 4, -1, 99
    x, idx, w, w13, s13, w2, s2 = args
    err = m().new_error_word()
    out = m().moe_layer_few(x, idx, w, w13, w2, w13_scales=s13, w2_scales=s2, err_word=err)
    assert m().moe_read_error(err) == m().MOE_ERRBIT_BAD_INDEX
    ref, bound = reference(*args)
    assert torch.all((out.double() - ref).abs() <= 4 * bound + ref.abs() * 2.0 ** -8)
    assert torch.all(out[4] == 0)


def test_zero_weights_and_empty_batch():
    args = list(make(4, 2, 256, 128, 8, True, seed=8))
    args[2][1] = 0
    out = check(args)
    assert torch.all(out[1] == 0)
    x, idx, w, w13, s13, w2, s2 = args
    assert m().moe_layer_few(x[:0], idx[:0], w[:0], w13, w2, w13_scales=s13, w2_scales=s2).shape == (0, 256)


def test_wild_values_stay_with_their_token():
    args = list(make(6, 2, 256, 128, 3, True, seed=9))
    args[0][2, 17] = float("nan")
    args[0][4, 3] = float("inf")
    x, idx, w, w13, s13, w2, s2 = args
    out = m().moe_layer_few(x, idx, w, w13, w2, w13_scales=s13, w2_scales=s2)
    ref, bound = reference(*args)
    ok = [0, 1, 3, 5]
    assert torch.all((out[ok].double() - ref[ok]).abs() <= 4 * bound[ok] + ref[ok].abs() * 2.0 ** -8)
    assert torch.all(torch.isnan(out[2])) and not torch.any(torch.isfinite(out[4]))


def test_same_bits_every_call():
    x, idx, w, w13, s13, w2, s2 = make(30, 8, 512, 256, 32, True, seed=10)
    first = m().moe_layer_few(x, idx, w, w13, w2, w13_scales=s13, w2_scales=s2)
    for _ in range(5):
        again = m().moe_layer_few(x, idx, w, w13, w2, w13_scales=s13, w2_scales=s2)
        assert torch.equal(first.view(torch.int16), again.view(torch.int16))


def test_graph_replay_and_other_stream():
    x, idx, w, w13, s13, w2, s2 = make(4, 2, 256, 256, 8, True, seed=11)
    p = m()
    ws = torch.empty(p.moe_layer_few_workspace_bytes(4, 2, 256, 256), dtype=torch.uint8, device="cuda")
    out = torch.empty((4, 256), dtype=torch.bfloat16, device="cuda")

    def call():
        p.moe_layer_few(x, idx, w, w13, w2, w13_scales=s13, w2_scales=s2, out=out, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
    x.copy_(torch.randn((4, 256), generator=gen(12), device="cuda"))
    idx.copy_(torch.rand((4, 8), generator=gen(13), device="cuda").topk(2, 1).indices)
    g.replay()
    torch.cuda.synchronize()
    ref, bound = reference(x, idx, w, w13, s13, w2, s2)
    assert torch.all((out.double() - ref).abs() <= 3 * bound + ref.abs() * 2.0 ** -8)


def test_layer_takes_both_forms():
    T, k, H, inner, E = 100, 4, 256, 256, 16
    p = m()
    x, _, _, w13, s13, w2, s2 = make(T, k, H, inner, E, True, seed=14)
    logits = torch.randn((T, E), generator=gen(15), device="cuda")
    layer = p.MoELayer(w13, s13, w2, s2, k)
    assert layer.few(64) and not layer.few(65)
    long = layer(x, logits)
    short = torch.cat([layer(x[i:i + 50], logits[i:i + 50]) for i in (0, 50)])
    assert p.moe_read_error(layer.err_word) == 0
    idx, w = p.moe_route(logits, k)
    ref, _ = reference(x, idx, w, w13, s13, w2, s2)
    assert (short.double() - ref).norm() / ref.norm() < 0.003   # bf16 output
    assert (long.double() - ref).norm() / ref.norm() < 0.06     # E4M3 rows before each product


@pytest.mark.parametrize("T,few", [(16, True), (16, False), (100, False)])
def test_on_another_stream(T, few):
    """Memory of the calling stream, given out again while another stream has the call's
    work still before it, is not part of that work."""
    H, inner, E, k = 512, 256, 16, 4
    p = m()
    x, idx, w, w13, s13, w2, s2 = make(T, k, H, inner, E, True, seed=21)
    logits = torch.randn((T, E), generator=gen(22), device="cuda")
    layer = p.MoELayer(w13, s13, w2, s2, k)

    def call(stream=None):
        if few:
            return p.moe_layer_few(x, idx, w, w13, w2, w13_scales=s13, w2_scales=s2,
                                   stream=stream)
        return layer(x, logits, stream=stream)

    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = call(side)
    sizes = [1 << i for i in range(9, 24)]
    over = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in (0, 1)]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    assert len(over) == 2 * len(sizes)
    assert torch.equal(got, want)
    assert p.moe_read_error(layer.err_word) == 0
