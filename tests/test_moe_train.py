"""CPU checks of the mixture-of-experts training operators: the reference's
gradients against differences of the reference's forward forms, and the host
side's refusals (no device work is issued; the pointers are placeholders that
are never dereferenced)."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from fp8_math_b200 import workloads as W


@pytest.fixture(scope="module")
def L():
    import os

    from fp8_math_b200 import bsq
    if not os.path.exists(bsq.LIB_PATH):
        from fp8_math_b200 import build
        build.build()
    return bsq


def _differences(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(5, 4, 2), (7, 9, 9), (3, 6, 1)])
def test_route_gradient_formula_matches_differences(T, E, k, renorm):
    rng = np.random.default_rng(T + E + k)
    z = rng.standard_normal((T, E))
    mask = np.ones(T)
    mask[1] = 0
    r = ref.route(z, k, mask, renorm, 0.3)
    a = rng.standard_normal((T, k))
    dloss = 0.7

    def total(x):
        q = ref.route(x, k, mask, renorm, 0.3)
        # the choice and the counts are constants of the gradient
        assert np.array_equal(q["expert_ids"], r["expert_ids"])
        return (a * q["weights"]).sum() + dloss * q["loss"]

    d = rng.standard_normal((T, E))
    dz, _ = ref.route_bwd(z, r["expert_ids"], r["weights"], a, r["counts"], dloss, 0.3, renorm)
    # the difference's own error is h^2 times a third derivative: these functions' derivatives are of order 1
    assert abs((dz * d).sum() - _differences(total, z, d)) <= 1e-6 * (1 + abs(dz * d).sum())
    assert (dz[1] == 0).all()


def test_combine_and_swiglu_gradient_formulas_match_differences():
    rng = np.random.default_rng(1)
    T, k, R, H = 4, 3, 12, 16
    rows = rng.permutation(R).reshape(T, k)
    rows[2, 1] = -1
    y, w, g = rng.standard_normal((R, H)), rng.random((T, k)), rng.standard_normal((T, H))
    dy = np.zeros((R, H))
    dw, _ = ref.combine_bwd(g, y, rows, w, dy)
    vy, vw = rng.standard_normal((R, H)), rng.standard_normal((T, k))
    f = lambda x: (g * ref.combine(y + x * vy, rows, w + x * vw)[0]).sum()  # noqa: E731
    assert abs((dy * vy).sum() + (dw * vw).sum() - _differences(f, 0.0, 1.0)) <= 1e-6 * (1 + abs(dy * vy).sum())
    u, dh, v = rng.standard_normal((5, 64)) * 3, rng.standard_normal((5, 32)), rng.standard_normal((5, 64))
    du, _ = ref.swiglu_bwd(dh, u)
    assert abs((du * v).sum() - _differences(lambda x: (dh * ref.swiglu(x)).sum(), u, v)) <= 1e-6 * (
        1 + abs(du * v).sum())


@pytest.mark.parametrize("T,E,k", [(40, 8, 3), (300, 5, 2)])
def test_route_reference_matches_the_workloads_row_order(T, E, k):
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(T))
    ri, off, sfo = W.route_topk(z, k)
    r = ref.route(z.numpy(), k)
    assert np.array_equal(r["row_index"], ri)
    assert np.array_equal(r["row_offsets"], off) and np.array_equal(r["sf_row_offsets"], sfo)


def test_route_workspace_and_refusals(L):
    lib = L.lib()
    assert L.bsq_moe_route_workspace(0, 8) > 0 and L.bsq_moe_route_workspace(1 << 20, 1024) > 0
    for T, E in [(-1, 8), (8, 0), (8, 1025), (1 << 31, 8)]:
        assert L.bsq_moe_route_workspace(T, E) == 0
    p, ws = 256, L.bsq_moe_route_workspace(16, 8)

    def call(logits=p, kind=0, T=16, E=8, ldl=8, mask=None, k=2, ids=p, w=p, rows=p, ri=p, ro=p, so=p, counts=p,
             ps=None, loss=None, work=p, nbytes=ws):
        return lib.bsq_moe_route(logits, kind, T, E, ldl, mask, k, 1, ids, w, rows, ri, ro, so, counts, ps, 0.0, loss,
                                 work, nbytes, None)

    for bad in [dict(logits=None), dict(kind=2), dict(T=-1), dict(E=0), dict(ldl=7), dict(k=0), dict(k=9),
                dict(ids=None), dict(w=None), dict(rows=None), dict(ri=None), dict(ro=None), dict(so=None),
                dict(counts=None), dict(work=None), dict(nbytes=ws - 1)]:
        assert call(**bad) == L.BSQ_ERR_INVALID, bad
    for bad in [dict(E=1025, ldl=1025), dict(E=64, ldl=64, k=33), dict(T=1 << 31), dict(T=1 << 30, k=2)]:
        assert call(**bad) == L.BSQ_ERR_UNSUPPORTED, bad
    for bad in [dict(logits=258), dict(logits=257, kind=1), dict(ids=258), dict(w=258), dict(rows=258), dict(ri=258),
                dict(ro=258), dict(so=258), dict(counts=258), dict(ps=258), dict(loss=258), dict(work=272)]:
        assert call(**bad) == L.BSQ_ERR_ALIGN, bad


def test_route_bwd_refusals(L):
    lib, p = L.lib(), 256

    def call(logits=p, kind=0, T=16, E=8, ldl=8, k=2, ids=p, w=p, dw=p, counts=p, dloss=p, out=p, ldd=8):
        return lib.bsq_moe_route_bwd(logits, kind, T, E, ldl, k, 1, ids, w, dw, counts, 0.0, dloss, out, ldd, None)

    for bad in [dict(logits=None), dict(kind=-1), dict(T=-1), dict(ldl=7), dict(ldd=7), dict(k=9), dict(ids=None),
                dict(w=None), dict(counts=None), dict(out=None)]:
        assert call(**bad) == L.BSQ_ERR_INVALID, bad
    assert call(E=1025, ldl=1025, ldd=1025) == L.BSQ_ERR_UNSUPPORTED
    for bad in [dict(logits=258), dict(out=258), dict(ids=257), dict(w=257), dict(dw=257), dict(counts=257),
                dict(dloss=257)]:
        assert call(**bad) == L.BSQ_ERR_ALIGN, bad


def test_combine_refusals(L):
    lib, p = L.lib(), 256

    def fwd(y=p, R=8, H=64, ldy=64, rows=p, w=p, T=4, k=2, out=p, ldo=64):
        return lib.bsq_moe_combine(y, R, H, ldy, rows, w, T, k, out, ldo, None)

    for bad in [dict(y=None), dict(R=-1), dict(H=60, ldy=64), dict(ldy=56), dict(rows=None), dict(T=-1), dict(k=0),
                dict(out=None), dict(ldo=56)]:
        assert fwd(**bad) == L.BSQ_ERR_INVALID, bad
    for bad in [dict(y=264), dict(out=264), dict(ldy=68), dict(ldo=68), dict(rows=258), dict(w=258)]:
        assert fwd(**bad) == L.BSQ_ERR_ALIGN, bad
    assert fwd(k=33) == L.BSQ_ERR_UNSUPPORTED and fwd(T=1 << 31) == L.BSQ_ERR_UNSUPPORTED

    def bwd(dout=p, ldo=64, y=p, ldy=64, c=None, s=None, R=8, H=64, rows=p, w=p, T=4, k=2, dy=p, lddy=64, dw=p):
        return lib.bsq_moe_combine_bwd(dout, ldo, y, ldy, c, s, R, H, rows, w, T, k, dy, lddy, dw, None)

    for bad in [dict(dout=None), dict(y=None), dict(y=p, c=p, s=p), dict(y=None, c=p), dict(y=None, s=p),
                dict(y=None, c=p, s=p, H=40), dict(ldy=56), dict(ldo=56), dict(lddy=56), dict(rows=None),
                dict(w=None), dict(dy=None), dict(dw=None), dict(k=0), dict(H=60)]:
        assert bwd(**bad) == L.BSQ_ERR_INVALID, bad
    for bad in [dict(dout=264), dict(y=264), dict(y=None, c=264, s=p), dict(y=None, c=p, s=264), dict(dy=264),
                dict(ldo=68), dict(ldy=68), dict(lddy=68), dict(rows=258), dict(w=258), dict(dw=258)]:
        assert bwd(**bad) == L.BSQ_ERR_ALIGN, bad
    assert bwd(k=33) == L.BSQ_ERR_UNSUPPORTED and bwd(T=1 << 30, k=2) == L.BSQ_ERR_UNSUPPORTED
    assert bwd(H=1 << 26, ldo=1 << 26, ldy=1 << 26, lddy=1 << 26) == L.BSQ_ERR_UNSUPPORTED


def test_swiglu_refusals(L):
    lib, p = L.lib(), 256

    def fwd(u=p, M=4, F=32, ldu=64, n=None, h=p, ldh=32, c=p, s=p, amax=None):
        return lib.bsq_swiglu_ckpt(u, M, F, ldu, n, h, ldh, c, s, amax, None)

    for bad in [dict(u=None), dict(M=-1), dict(F=24), dict(ldu=56), dict(h=None), dict(ldh=24), dict(c=None),
                dict(s=None)]:
        assert fwd(**bad) == L.BSQ_ERR_INVALID, bad
    for bad in [dict(u=264), dict(h=264), dict(c=264), dict(s=264), dict(ldu=68), dict(ldh=36), dict(n=258),
                dict(amax=258)]:
        assert fwd(**bad) == L.BSQ_ERR_ALIGN, bad

    assert fwd(M=1 << 30, F=32) == L.BSQ_ERR_UNSUPPORTED and fwd(M=1 << 31) == L.BSQ_ERR_UNSUPPORTED

    def bwd(dh=p, lddh=32, c=p, s=p, M=4, F=32, n=None, du=p, lddu=64, h=None, ldh=0):
        return lib.bsq_swiglu_ckpt_bwd(dh, lddh, c, s, M, F, n, du, lddu, h, ldh, None)

    for bad in [dict(dh=None), dict(c=None), dict(s=None), dict(du=None), dict(F=24), dict(lddh=24), dict(lddu=56),
                dict(h=p, ldh=24), dict(M=-1)]:
        assert bwd(**bad) == L.BSQ_ERR_INVALID, bad
    for bad in [dict(dh=264), dict(c=264), dict(s=264), dict(du=264), dict(h=264, ldh=32), dict(h=p, ldh=36),
                dict(lddh=36), dict(lddu=68), dict(n=258)]:
        assert bwd(**bad) == L.BSQ_ERR_ALIGN, bad


def test_route_sizes_are_told_before_the_workspace_is_asked_for(L):
    """For sizes that are not supported the workspace has 0 bytes, and so a caller's pointer may be null."""
    lib, p = L.lib(), 256

    def call(T=16, E=8, k=2, ldl=2048):
        n = L.bsq_moe_route_workspace(T, E)
        return lib.bsq_moe_route(p, 0, T, E, ldl, None, k, 1, p, p, p, p, p, p, p, None, 0.0, None, p if n else None, n,
                                 None)

    assert call(E=1025) == L.BSQ_ERR_UNSUPPORTED
    assert call(T=1 << 31) == L.BSQ_ERR_UNSUPPORTED
    assert call(T=(1 << 31) - 1024, E=1024) == L.BSQ_ERR_UNSUPPORTED
    assert call(E=0) == L.BSQ_ERR_INVALID and call(T=-1) == L.BSQ_ERR_INVALID
