"""The router, expert and few-token calls reject bad arguments on the host,
before anything is launched (addresses here are never dereferenced)."""
import pytest

FAKE = 1 << 20


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__._cuda_build_module().build()
    import combine_layout_moe_gb300 as pkg
    return pkg


def test_route_refusals(m):
    def call(T=4, E=8, k=2, groups=1, keep=1, logits=FAKE, stride=8, dtype=1, idx=FAKE, w=FAKE):
        return m._lib.moe_route(T, E, k, groups, keep, logits, stride, dtype, idx, w, None)
    bad = m.MOE_ERR_INVALID_ARG
    assert call(T=-1) == bad
    assert call(k=0) == bad
    assert call(k=9) == bad                            # more than the experts
    assert call(E=0) == bad
    assert call(E=9, stride=9, groups=2, keep=1) == bad  # E % groups
    assert call(groups=4, keep=5) == bad
    assert call(groups=4, keep=0) == bad
    assert call(groups=4, keep=1, k=3) == bad          # a group holds two experts
    assert call(stride=7) == bad
    assert call(dtype=2) == bad
    assert call(logits=None) == bad and call(idx=None) == bad and call(w=None) == bad
    assert call(logits=FAKE + 2) == bad                # fp32 rows off a 4-byte boundary
    assert call(w=FAKE + 1) == bad
    assert call(E=2048, stride=2048) == m.MOE_ERR_UNSUPPORTED
    assert call(E=64, stride=64, k=33) == m.MOE_ERR_UNSUPPORTED
    assert call(E=64, stride=64, groups=64, keep=2) == m.MOE_ERR_UNSUPPORTED
    assert call(T=0, logits=None, idx=None, w=None) == m.MOE_OK


def test_route_backward_refusals(m):
    def call(T=4, E=8, k=2, idx=FAKE, w=FAKE, dw=FAKE, out=FAKE, dtype=1, err=None):
        return m._lib.moe_route_backward(T, E, k, idx, w, dw, out, dtype, err, None)
    bad = m.MOE_ERR_INVALID_ARG
    assert call(T=-1) == bad and call(k=0) == bad and call(k=9) == bad and call(dtype=7) == bad
    assert call(idx=None) == bad and call(dw=None) == bad and call(out=None) == bad
    assert call(out=FAKE + 2) == bad and call(err=FAKE + 1) == bad
    assert call(E=64, k=40) == m.MOE_ERR_UNSUPPORTED
    assert call(T=0, idx=None, w=None, dw=None, out=None) == m.MOE_OK


def test_expert_gemm_refusals(m):
    def call(N=4, K=256, M=64, E=2, a=FAKE, sa=FAKE, off=FAKE, w=FAKE, sw=FAKE, tr=0, out=FAKE,
             dtype=0, err=None):
        return m._lib.moe_expert_gemm(N, K, M, E, a, sa, off, w, sw, tr, out, dtype, err, None)
    bad = m.MOE_ERR_INVALID_ARG
    assert call(N=-1) == bad and call(K=64) == bad and call(K=192) == bad
    assert call(M=8) == bad and call(M=24) == bad and call(E=0) == bad
    assert call(tr=2) == bad and call(dtype=2) == bad
    for name in ("a", "sa", "w", "sw", "out"):
        assert call(**{name: None}) == bad, name
        assert call(**{name: FAKE + 8}) == bad, name
    assert call(off=None) == bad and call(off=FAKE + 2) == bad and call(err=FAKE + 2) == bad
    assert call(E=2000) == m.MOE_ERR_UNSUPPORTED
    assert call(N=0, a=None, sa=None, off=None, w=None, sw=None, out=None) == m.MOE_OK


def test_expert_swiglu_refusals(m):
    def call(N=4, K=256, inner=128, E=2, a=FAKE, sa=FAKE, off=FAKE, w=FAKE, sw=FAKE, h=FAKE,
             hs=FAKE, err=None):
        return m._lib.moe_expert_swiglu(N, K, inner, E, a, sa, off, w, sw, h, hs, err, None)
    bad = m.MOE_ERR_INVALID_ARG
    assert call(N=-1) == bad and call(K=130) == bad and call(inner=64) == bad
    assert call(inner=192) == bad and call(E=0) == bad
    for name in ("a", "sa", "w", "sw", "h", "hs"):
        assert call(**{name: None}) == bad, name
        assert call(**{name: FAKE + 4}) == bad, name
    assert call(off=None) == bad
    assert call(E=1025) == m.MOE_ERR_UNSUPPORTED
    assert call(N=0, a=None, sa=None, off=None, w=None, sw=None, h=None, hs=None) == m.MOE_OK


def test_expert_wgrad_refusals(m):
    def call(N=4, M=16, K=16, E=2, dy=FAKE, x=FAKE, off=FAKE, dw=FAKE, err=None):
        return m._lib.moe_expert_wgrad(N, M, K, E, dy, x, off, dw, err, None)
    bad = m.MOE_ERR_INVALID_ARG
    assert call(N=-1) == bad and call(M=12) == bad and call(K=4) == bad and call(E=0) == bad
    for name in ("dy", "x", "dw"):
        assert call(**{name: None}) == bad, name
        assert call(**{name: FAKE + 8}) == bad, name
    assert call(off=None) == bad and call(off=FAKE + 1) == bad
    assert call(E=1025) == m.MOE_ERR_UNSUPPORTED


def test_layer_few_refusals(m):
    need = m.moe_layer_few_workspace_bytes(4, 2, 256, 128)
    assert need > 0
    assert m.moe_layer_few_workspace_bytes(65, 2, 256, 128) == 0
    assert m.moe_layer_few_workspace_bytes(64, 9, 256, 128) == 0
    assert m.moe_layer_few_workspace_bytes(4, 2, 252, 128) == 0

    def call(T=4, k=2, H=256, inner=128, E=8, x=FAKE, idx=FAKE, w=FAKE, w13=FAKE, s13=FAKE,
             w2=FAKE, s2=FAKE, kind=1, out=FAKE, dtype=0, ws=FAKE, nbytes=need, err=None):
        return m._lib.moe_layer_few(T, k, H, inner, E, x, idx, w, w13, s13, w2, s2, kind, out,
                                    dtype, ws, nbytes, err, None)
    bad = m.MOE_ERR_INVALID_ARG
    assert call(T=-1) == bad and call(k=0) == bad and call(E=0) == bad
    assert call(H=192) == bad and call(inner=64) == bad       # E4M3 takes whole blocks
    assert call(kind=0, H=252) == bad and call(kind=2) == bad and call(dtype=3) == bad
    for name in ("x", "idx", "w", "w13", "s13", "w2", "s2", "out", "ws"):
        assert call(**{name: None}) == bad, name
    for name in ("x", "w13", "s13", "w2", "s2", "out", "ws"):
        assert call(**{name: FAKE + 8}) == bad, name
    assert call(nbytes=need - 1) == bad
    assert call(T=65) == m.MOE_ERR_UNSUPPORTED
    assert call(T=64, k=9, nbytes=1 << 30) == m.MOE_ERR_UNSUPPORTED
    assert call(E=1025) == m.MOE_ERR_UNSUPPORTED


def test_bindings_reject_host_tensors(m):
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 8))
    with pytest.raises(ValueError):
        m.moe_route(x, 2)
    with pytest.raises(ValueError):
        m.moe_expert_wgrad(x.bfloat16(), x.bfloat16(), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        m.MoELayer(x, x, x, x, 2)
