"""The mixture-of-experts training operators where their kernels change form:
sizes at the limit of shared memory, more slots than lanes, tokens of a second
round, several chunks per CTA, sigmoids below the normal numbers, exponents far
below the largest; and refusals with their exact status.  Tolerances count fp32
roundings as in test_gpu_moe.py."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import moe_ref as ref
from fp8_math_b200 import api, bsq
from gpu_util import dev
from moe_ref import B, U, within
from test_gpu_moe import check_route_bwd, decode8, ints, logits_of, n64

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))

# (T, E, k) whose first launch asks for 48 KB of dynamic shared memory, or up to 15 bytes less: one CTA of a cluster,
# 16 warps, 8 warps
AT_48K = [(65, 440, 31), (65, 463, 26), (65, 472, 24), (65, 495, 19), (65, 504, 17), (65, 527, 12), (65, 536, 10),
          (65, 559, 5), (65, 568, 3), (1000, 519, 30), (1000, 535, 27), (1000, 551, 24), (1000, 567, 21),
          (1000, 583, 18), (1000, 599, 15), (1000, 615, 12), (1000, 631, 9), (1000, 647, 6), (1000, 663, 3),
          (20000, 915, 32), (20000, 934, 30), (20000, 963, 27), (20000, 982, 25), (20000, 1011, 22)]


def route_at_48k():
    """Run in a process of its own: a call of a larger size would raise the limit for the kernel it takes."""
    for T, E, k in AT_48K:
        for dtype in (torch.float32, torch.bfloat16):
            z = torch.randn(T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(E)).to(dtype)
            r = api.moe_route(z, k, balance_coef=0.5)
            best = torch.sort(z.double(), dim=1, descending=True, stable=True)
            assert torch.equal(r.expert_ids.long(), best.indices[:, :k]), (T, E, k)
            w = torch.softmax(best.values[:, :k], 1)
            assert (r.weights.double() - w).abs().max() < 1e-5, (T, E, k)
            assert (r.prob_sums.double() - torch.softmax(z.double(), 1).sum(0)).abs().max() < 1e-5 * T, (T, E, k)
    assert bsq.bsq_check() == bsq.BSQ_OK
    print("route_at_48k ok")


def test_route_at_the_default_limit_of_shared_memory():
    code = f"import sys; sys.path[:0] = [{os.path.dirname(HERE)!r}, {HERE!r}]; import test_gpu_moe_edges as m; " \
           "m.route_at_48k()"
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "route_at_48k ok" in p.stdout, p.stderr[-2000:]


# ------------------------------------------------------------------ refusals
def status_of(call):
    with pytest.raises(bsq.BsqError) as e:
        call()
    return e.value.status


def test_route_says_unsupported_for_sizes_it_does_not_take():
    assert status_of(lambda: api.moe_route(torch.zeros(4, 1025, device="cuda"), 2)) == bsq.BSQ_ERR_UNSUPPORTED
    assert status_of(lambda: api.moe_route(torch.zeros(4, 64, device="cuda"), 33)) == bsq.BSQ_ERR_UNSUPPORTED
    assert status_of(lambda: api.moe_route(torch.zeros(4, 8, device="cuda"), 9)) == bsq.BSQ_ERR_INVALID


def test_route_bwd_refuses_a_loss_gradient_without_its_coefficient():
    z = dev(logits_of(20, 8, 1))
    r = api.moe_route(z, 2, balance_coef=0.5)
    one = torch.ones(1, device="cuda")
    assert status_of(lambda: api.moe_route_bwd(z, r.expert_ids, r.weights, counts=r.counts, dloss=one)) == \
        bsq.BSQ_ERR_INVALID
    with_loss = api.moe_route_bwd(z, r.expert_ids, r.weights, counts=r.counts, dloss=one, balance_coef=0.5)
    assert (with_loss != 0).any()
    assert (api.moe_route_bwd(z, r.expert_ids, r.weights, counts=r.counts, dloss=one, balance_coef=0.0) == 0).all()


def test_route_refuses_a_coefficient_without_a_place_for_the_loss():
    z = dev(logits_of(20, 8, 1))
    r = api.moe_route(z, 2, balance_coef=0.5)
    for out in [(*r[:7], r.prob_sums, None), (*r[:7], None, None)]:
        assert status_of(lambda: api.moe_route(z, 2, balance_coef=0.5, out=out)) == bsq.BSQ_ERR_INVALID
    assert api.moe_route(z, 2, out=(*r[:7], None, None)).loss is None


def test_wrappers_refuse_with_the_librarys_error():
    """Each of these is a BsqError of status invalid, never an error of another kind from inside the wrapper."""
    z = torch.zeros(4, 8, device="cuda")
    i = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    y = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(8, 64, dtype=torch.uint8, device="cuda")
    d = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(api.sf_bytes(8, 2), dtype=torch.uint8, device="cuda")
    for bad in [lambda: api.moe_route(z, 0), lambda: api.moe_route(z, -1), lambda: api.moe_route_bwd(z, i, None),
                lambda: api.moe_combine_bwd(d, y, i, None), lambda: api.moe_combine_bwd(None, y, i, w),
                lambda: api.moe_combine_bwd(d, (c, None), i, w), lambda: api.swiglu_ckpt_bwd(y[:, :32], None, s),
                lambda: api.swiglu_ckpt_bwd(y[:, :32], c, None),
                lambda: api.moe_combine(y, i, out=[1.0]), lambda: api.moe_combine(y, i, [1.0] * 8),
                lambda: api.swiglu_ckpt(y, n_rows=8)]:
        assert status_of(bad) == bsq.BSQ_ERR_INVALID


@pytest.mark.parametrize("n", [0, 3, 40])
def test_swiglu_rows_that_do_not_exist_are_zeros_without_out(n):
    """A buffer that the wrapper makes has no row left unwritten: whole-tensor calls read it next."""
    M, F = 40, 64
    u = torch.randn(M, 2 * F, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    count = torch.tensor([n], dtype=torch.int32, device="cuda")
    for _ in range(2):
        for size in (M * F * 2, M * F, M * F * 4):  # what the allocator hands out next holds NaN and large codes
            junk = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
            del junk
        h, codes, sf, _ = api.swiglu_ckpt(u, n_rows=count)
        assert (h[n:].view(torch.int16) == 0).all() and (codes[n:] == 0).all()
        for size in (M * F * 2, M * F * 4):
            junk = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
            del junk
        du, again = api.swiglu_ckpt_bwd(h, codes, sf, n_rows=count, recompute_h=True)
        assert (du[n:].view(torch.int16) == 0).all() and (again[n:].view(torch.int16) == 0).all()


# ------------------------------------------------------------------ router
def check_route_large(z, k, mask, renorm, coef):
    """As check_route of test_gpu_moe.py, with a reference that is vectorised over the tokens."""
    T, E = z.shape
    r = api.moe_route(dev(z), k, token_mask=None if mask is None else dev(mask), renorm=renorm, balance_coef=coef)
    live = np.ones(T, bool) if mask is None else mask.numpy() != 0
    zz = np.where(live[:, None], n64(z), -np.inf)
    ids = np.argsort(-zz, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(zz, ids, 1)
    ids[~live] = -1
    assert np.array_equal(ints(r.expert_ids), ids)
    flat = np.where(ids < 0, E, ids).ravel()
    order = np.argsort(flat, kind="stable")
    n = int((ids >= 0).sum())
    rows = np.full(T * k, -1)
    rows[order[:n]] = np.arange(n)
    assert np.array_equal(ints(r.rows).ravel(), rows)
    index = np.full(T * k, order[0] // k)
    index[:n] = order[:n] // k
    assert np.array_equal(ints(r.row_index), index)
    count = np.bincount(flat, minlength=E + 1)[:E]
    assert np.array_equal(ints(r.counts), np.append(count, live.sum()))
    assert np.array_equal(ints(r.row_offsets), np.append(0, np.cumsum(count)))
    p = ref.softmax(zz, live)
    w = ref.softmax(top, live) if renorm else np.where(live[:, None], np.take_along_axis(p, np.maximum(ids, 0), 1), 0)
    rel = (3 * ref.spread(n64(z), live) + 4 + -(-E // 32) + 5 + 3) * U
    within(n64(r.weights), w, rel * w + ref.TINY, "weights")
    # the tokens of a warp, its warps, the chunks of a CTA, the CTAs, a tree
    rel += (8 + 8 + 16 + T / 4096 + 16) * U
    within(n64(r.prob_sums), p.sum(0), rel * p.sum(0) + T * ref.TINY, "prob_sums")
    loss = coef * E * (count * p.sum(0)).sum() / k / live.sum() ** 2
    within(n64(r.loss), [loss], (rel + (E / 32 + 20) * U) * loss, "loss")


@pytest.mark.parametrize("T,E,k", [(25000, 160, 8), (25000, 256, 8), (21000, 140, 11), (20001, 600, 3),
                                   (16384, 128, 8), (16000, 200, 2)])
@pytest.mark.parametrize("bf16", [False, True])
def test_route_with_several_chunks_per_cta(T, E, k, bf16):
    """More chunks than CTAs (or than fit at once): masks are cleared and sums go on from chunk to chunk."""
    mask = torch.ones(T, dtype=torch.uint8)
    mask[5000:5400] = 0
    mask[T - 70:T - 3] = 0
    check_route_large(logits_of(T, E, T + E, bf16), k, mask, not bf16, 0.5)


@pytest.mark.parametrize("T,E,k", [(60, 64, 10), (40, 20, 20), (30, 400, 20), (33, 300, 17), (50, 250, 32),
                                   (70, 37, 9)])
@pytest.mark.parametrize("bf16,renorm", [(False, True), (True, False), (True, True), (False, False)])
def test_route_bwd_with_more_slots_than_lanes(T, E, k, bf16, renorm):
    z = dev(logits_of(T, E, T * E, bf16, "shut" if E > 100 else "normal"))
    r = api.moe_route(z, k, renorm=renorm)
    a = torch.randn(T, k, generator=torch.Generator().manual_seed(k))
    check_route_bwd(z, r, a, 1.5, 0.1, renorm)
    check_route_bwd(z, r, a, None, 0.1, renorm)


@pytest.mark.parametrize("T,E,k", [(30000, 32, 4), (30000, 31, 4), (30000, 24, 11), (25000, 160, 6), (25000, 158, 12),
                                   (8000, 1000, 12), (8000, 999, 32)])
@pytest.mark.parametrize("bf16,renorm", [(False, True), (True, False)])
def test_route_bwd_of_more_tokens_than_fit_at_once(T, E, k, bf16, renorm):
    """A group of lanes takes a second token: the row of shared memory between them is zero again."""
    z = dev(logits_of(T, E, T + E, bf16))
    mask = torch.ones(T, dtype=torch.uint8)
    mask[100:400] = 0
    mask[T - 500:T - 200] = 0
    r = api.moe_route(z, k, token_mask=dev(mask), renorm=renorm)
    a = torch.randn(T, k, generator=torch.Generator().manual_seed(k))
    check_route_bwd(z, r, a, 1.5, 0.1, renorm)
    check_route_bwd(z, r, a, None, 0.1, renorm)


def exact_differences(T, E, seed):
    """fp32 logits whose differences from the largest are exact (multiples of 1/64 below 64 in magnitude), far apart:
    the weights' exponentials then have no rounding that grows with the distance."""
    z = torch.randint(-84 * 64, 1, (T, E), generator=torch.Generator().manual_seed(seed)).float() / 64
    z[:, 0] = 0
    return z


@pytest.mark.parametrize("E,k", [(8, 8), (12, 12), (5, 4), (200, 8)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_exponentials_far_below_the_largest(E, k, renorm):
    """e^d for an exact d: 0.05 |d| U from the constant that splits d, ex2 4 U, its correction 1 U; then the sum over E
    (a lane's quads, 5 exchanges), the reciprocal 2 U and two products."""
    T = 2000
    z = exact_differences(T, E, E)
    r = api.moe_route(dev(z), k, renorm=renorm, balance_coef=1.0)
    ids = np.argsort(-n64(z), axis=1, kind="stable")[:, :k]
    assert np.array_equal(ints(r.expert_ids), ids)
    x = np.exp(n64(z))
    chosen = np.take_along_axis(x, ids, 1)
    w = chosen / (chosen if renorm else x).sum(1, keepdims=True)
    rel = 2 * (0.05 * 84 + 5) + -(-E // 32) + 5 + 2 + 2
    within(n64(r.weights), w, rel * U * w, "weights")
    # gradient of the loss alone: p, the bias's sum, their difference and product
    one = torch.ones(1, device="cuda")
    d = api.moe_route_bwd(dev(z), r.expert_ids, r.weights, counts=r.counts, dloss=one, balance_coef=1.0, renorm=renorm)
    want, mag = ref.route_bwd(n64(z), ids, n64(r.weights), None, ints(r.counts), 1.0, 1.0, renorm)
    within(n64(d), want, (2 * rel + 10) * U * mag + 1e-37, "dlogits")


# ------------------------------------------------------------------ gated SiLU
def far_gates(M, F, seed):
    """Gates between -150 and -80 with v up to 1e32, so that h is an ordinary number though the sigmoid is not."""
    g = torch.Generator().manual_seed(seed)
    u = torch.empty(M, 2 * F)
    u[:, :F] = -80 - 70 * torch.rand(M, F, generator=g) ** 2
    u[:, F:] = 10.0 ** (32 * torch.rand(M, F, generator=g)) * torch.randn(M, F, generator=g)
    return u.to(torch.bfloat16)


def test_swiglu_keeps_sigmoids_below_the_normal_numbers():
    """The sigmoid: 2 |g| for the square of a half exponent, 2 x 4 for ex2, four products and sums, the reciprocal 2;
    one more product with v; bf16's rounding.  g s and s are held in fp32 with its subnormal numbers: half a step of
    those (2^-150) times v; bf16's own half step there is 2^-134."""
    M, F = 64, 512
    u = far_gates(M, F, 1)
    h, codes, sf, _ = api.swiglu_ckpt(dev(u))
    g, v = n64(u)[:, :F], n64(u)[:, F:]
    want = ref.swiglu(n64(u))
    assert (abs(want) > 1e-30).mean() > 0.1
    tol = (2 * abs(g) + 8 + 4 + 2 + 1) * U
    within(n64(h), want, (B + tol) * abs(want) + 2.0 ** -149 * abs(v) + 2.0 ** -134, "h")
    # the gradient, on the decoded values
    dh = torch.randn(M, F, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    du, again = api.swiglu_ckpt_bwd(dev(dh), codes, sf, recompute_h=True)
    x = decode8(codes, sf)
    g, v = x[:, :F], x[:, F:]
    want = ref.swiglu(x)
    tol = (2 * abs(g) + 15) * U
    within(n64(again), want, (B + tol) * abs(want) + 2.0 ** -149 * abs(v) + 2.0 ** -134, "h again")
    want, mag = ref.swiglu_bwd(n64(dh), x)
    d = abs(n64(dh))
    assert (abs(want[:, :F]) > 1e-30).mean() > 0.1
    sub = 2.0 ** -148 * np.concatenate([d * abs(v), d], 1)  # s and g s, each half a step
    t = np.concatenate([tol, tol], 1) + 6 * U
    within(n64(du), want, t * mag + sub + B * (abs(want) + sub) + 2.0 ** -134, "du")
