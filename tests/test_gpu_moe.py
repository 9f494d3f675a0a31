"""The mixture-of-experts training operators on the GPU against their binary64
forms (moe_ref.py): the router, its balance loss and gradient, the combine and
its gradients, the gated SiLU with its MXFP8 checkpoint, and a layer's forward
and backward pass that runs them together with the quantizers and grouped
GEMMs.

Tolerances count fp32 roundings (U = 2^-24 relative each) along the longest
chain of operations, and one rounding of the output type (bf16: 2^-8).  An
exponential e^d of d = x - max is formed as 2^(d log2 e): the roundings of the
difference, of the product and of the constant are each |d| U in d, so 3 |d| U
in e^d; ex2.approx adds 4 U (2^-22), rcp.approx 2 U, a product or sum 1 U per
step.  In the sigmoid d = -g is exact, which leaves 2 |g| U; one below 2^-126 is
0 there (its exponential overflows), which adds 2^-126 times what it multiplies."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from fp8_math_b200 import api, bsq
from gpu_util import assert_codes_equal, bits, dev
from moe_ref import B, TINY, U, within

pytestmark = pytest.mark.gpu


def n64(t):
    return t.detach().double().cpu().numpy()


def ints(t):
    return t.cpu().numpy().astype(np.int64)


def logits_of(T, E, seed, bf16=False, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) * 2
    if kind == "ties":          # few distinct values, both zeros among them
        z = torch.randint(-1, 2, (T, E), generator=g).float()
        z[::2] *= -1.0          # turns 0 into -0
    elif kind == "shut":        # experts shut to some tokens; some tokens have none left
        z[torch.rand(T, E, generator=g) < 0.6] = -np.inf
        z[::5] = -np.inf
    elif kind == "lowest":      # masks written as the type's lowest value
        low = torch.finfo(torch.bfloat16 if bf16 else torch.float32).min
        z[torch.rand(T, E, generator=g) < 0.7] = low
        z[::4] = low
    elif kind == "near":        # fp32 values that differ in their last bits only
        z = 1.0 + torch.randint(0, 300, (T, E), generator=g).float() * 2.0 ** -23
        z[1::2] *= -1.0
        z[::3, ::2] = torch.randn(z[::3, ::2].shape, generator=g)
    elif kind == "wide":        # far apart: small probabilities underflow
        z *= 60
    return z.to(torch.bfloat16) if bf16 else z


def check_route(r, z, k, mask, renorm, coef):
    """Every output of api.moe_route against the reference."""
    want = ref.route(n64(z), k, None if mask is None else ints(mask), renorm, coef or 0.0)
    for name in ("expert_ids", "rows", "row_index", "row_offsets", "sf_row_offsets", "counts"):
        assert np.array_equal(ints(getattr(r, name)), want[name]), name
    T, E = z.shape
    # the exponential, the sum over E (32 lanes), the reciprocal and its product
    rel = (3 * ref.spread(n64(z), want["live"]) + 4 + -(-E // 32) + 5 + 3) * U
    within(n64(r.weights), want["weights"], rel * want["weights"] + TINY, "weights")
    if coef is not None:
        # the tokens of a warp, the warps, the chunks, a tree, then the loss's own steps
        rel += (8 + 8 + 16 + T / 4096 + 16) * U
        within(n64(r.prob_sums), want["prob_sums"], rel * want["prob_sums"] + T * TINY, "prob_sums")
        within(n64(r.loss), [want["loss"]], (rel + (E / 256 + 20) * U) * want["loss"] + TINY, "loss")
    return want


ROUTES = [(1, 1, 1), (1, 64, 8), (63, 7, 7), (64, 33, 4), (65, 160, 6), (200, 256, 8), (130, 257, 3), (77, 1024, 32),
          (1000, 60, 5), (700, 512, 10), (5, 1000, 1)]


@pytest.mark.parametrize("T,E,k", ROUTES)
@pytest.mark.parametrize("bf16,renorm", [(False, True), (True, False)])
def test_route(T, E, k, bf16, renorm):
    z = dev(logits_of(T, E, T + E, bf16))
    check_route(api.moe_route(z, k, renorm=renorm, balance_coef=0.02), z, k, None, renorm, 0.02)
    check_route(api.moe_route(z, k, renorm=renorm), z, k, None, renorm, None)


@pytest.mark.parametrize("kind", ["ties", "shut", "lowest", "near", "wide"])
@pytest.mark.parametrize("bf16,renorm,T,E,k", [(False, True, 150, 40, 6), (True, False, 300, 130, 8),
                                               (True, True, 64, 256, 4), (False, False, 67, 3, 3),
                                               (False, True, 70, 512, 8), (False, True, 90, 64, 12),
                                               (True, True, 33, 700, 16), (False, True, 65, 1000, 2),
                                               (False, False, 40, 160, 8), (False, True, 30, 256, 1)])
def test_route_difficult_logits(kind, bf16, renorm, T, E, k):
    z = dev(logits_of(T, E, T + k, bf16, kind))
    mask = dev((torch.rand(T, generator=torch.Generator().manual_seed(4)) < 0.8).to(torch.uint8))
    for m in (None, mask):
        check_route(api.moe_route(z, k, token_mask=m, renorm=renorm, balance_coef=1.0), z, k, m, renorm, 1.0)


@pytest.mark.parametrize("T,E,k,masked", [(9000, 257, 2, False), (33000, 12, 3, True), (40000, 100, 1, True),
                                          (4096 * 3, 300, 9, True)])
def test_route_of_many_tokens(T, E, k, masked):
    """More chunks than one launch adds up, blocks of chunks that hold no row of an expert (or none at all), a ragged
    last chunk.  The reference is vectorised here: sort by (expert, token)."""
    z = logits_of(T, E, T, False)
    z[:5000, 0] = -np.inf                      # expert 0 starts late
    mask = torch.ones(T, dtype=torch.uint8)
    if masked:
        mask[:4200] = 0                        # the first block of chunks is padding
        mask[T // 2:T // 2 + 77] = 0
    r = api.moe_route(dev(z), k, token_mask=dev(mask) if masked else None, balance_coef=0.5)
    live = mask.numpy() != 0
    zz = np.where(live[:, None], z.numpy().astype(np.float64), -np.inf)
    ids = np.argsort(-zz, axis=1, kind="stable")[:, :k]
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
    assert np.array_equal(ints(r.sf_row_offsets), np.append(0, np.cumsum((count + 127) // 128 * 128)))
    p = ref.softmax(zz, live).sum(0)
    rel = (3 * ref.spread(z.numpy(), live) + 4 + -(-E // 32) + 5 + 3 + 8 + 8 + 8 + 8 + T / 4096 + 16) * U
    within(n64(r.prob_sums), p, rel * p + T * TINY, "prob_sums")
    loss = 0.5 * E * (count * p).sum() / k / live.sum() ** 2
    within(n64(r.loss), [loss], (rel + (E / 32 + 20) * U) * loss, "loss")


@pytest.mark.parametrize("T", [64, 65, 128, 129, 256, 257, 448, 512, 513])
@pytest.mark.parametrize("masked", [False, True])
def test_route_around_the_cluster_sizes(T, masked):
    """One, two, four and eight CTAs of 64 tokens that finish the call together, with CTAs that have no tokens, and
    one token more than they take; the first CTA's tokens may all be padding."""
    z = dev(logits_of(T, 72, T, False, "shut"))
    mask = torch.ones(T, dtype=torch.uint8)
    if masked:
        mask[:min(T - 1, 70)] = 0
    check_route(api.moe_route(z, 5, token_mask=dev(mask), balance_coef=0.3), z, 5, dev(mask), True, 0.3)


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (130, 24, 3)])
def test_route_of_masked_tokens_reads_nothing_of_them(T, E, k):
    """Padding may hold NaN; with every token masked nothing is routed."""
    z = logits_of(T, E, 9)
    mask = (torch.arange(T) % 3 == 1).to(torch.uint8)
    z[mask == 0] = float("nan")
    zd, md = dev(z), dev(mask)
    clean = dev(torch.where(mask[:, None] == 0, 0.0, z))
    for kind in (md, md.bool()):
        r = api.moe_route(zd, k, token_mask=kind, balance_coef=0.5)
        check_route(r, clean, k, md, True, 0.5)
    d = api.moe_route_bwd(zd, r.expert_ids, r.weights, dweights=torch.full_like(r.weights, float("nan")),
                          counts=r.counts, dloss=torch.ones(1, device="cuda"), balance_coef=0.5)
    assert (n64(d)[mask.numpy() == 0] == 0).all()
    r = api.moe_route(zd, k, token_mask=torch.zeros_like(md), balance_coef=0.5)
    assert (ints(r.expert_ids) == -1).all() and (ints(r.row_index) == 0).all() and (ints(r.counts) == 0).all()
    assert r.loss.item() == 0 and (n64(r.weights) == 0).all() and (n64(r.prob_sums) == 0).all()


def test_route_without_tokens_writes_its_offsets():
    r = api.moe_route(torch.empty(0, 8, device="cuda"), 2, balance_coef=0.1,
                      out=[torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda"),
                           torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                           torch.empty(0, dtype=torch.int32, device="cuda")] +
                          [torch.full((9,), 7, dtype=torch.int32, device="cuda") for _ in range(3)] +
                          [torch.full((8,), 7.0, device="cuda"), torch.full((1,), 7.0, device="cuda")])
    for t in r[4:]:
        assert (n64(t) == 0).all()
    assert api.moe_route_bwd(torch.empty(0, 8, device="cuda"), r.expert_ids, r.weights).shape == (0, 8)


@pytest.mark.parametrize("bf16", [False, True])
def test_route_takes_any_leading_dimension_and_offset(bf16):
    T, E, k = 90, 37, 5
    z = logits_of(T, E, 3, bf16)
    big = torch.full((T, E + 14), float("nan"), dtype=z.dtype)
    big[:, 3:3 + E] = z
    view = dev(big)[:, 3:3 + E]
    r = api.moe_route(view, k, balance_coef=0.1)
    check_route(r, dev(z), k, None, True, 0.1)
    out = torch.full((T, E + 5), 9.0, dtype=z.dtype, device="cuda")
    a = torch.randn(T, k, generator=torch.Generator().manual_seed(1))
    api.moe_route_bwd(view, r.expert_ids, r.weights, dweights=dev(a), out=out[:, 2:2 + E])
    assert (out[:, :2] == 9).all() and (out[:, 2 + E:] == 9).all()
    same = api.moe_route_bwd(dev(z), r.expert_ids, r.weights, dweights=dev(a))
    assert torch.equal(out[:, 2:2 + E].contiguous(), same)


def check_route_bwd(z, r, a, dloss, coef, renorm):
    d = api.moe_route_bwd(z, r.expert_ids, r.weights, dweights=None if a is None else dev(a), counts=r.counts,
                          dloss=None if dloss is None else torch.full((1,), dloss, device="cuda"), balance_coef=coef,
                          renorm=renorm)
    a64 = None if a is None else n64(a)
    want, mag = ref.route_bwd(n64(z), ints(r.expert_ids), n64(r.weights), a64, ints(r.counts), dloss, coef, renorm)
    live = ints(r.expert_ids)[:, 0] >= 0
    # p's own error, the sums over E and over k, and the products and differences
    tol = (3 * ref.spread(n64(z), live) + 7 + 2 * (-(-z.shape[1] // 32) + 5) + 10) * U * mag + TINY
    if z.dtype == torch.bfloat16:
        tol = tol + B * (abs(want) + tol)
    within(n64(d), want, tol, "dlogits")


@pytest.mark.parametrize("T,E,k", ROUTES)
@pytest.mark.parametrize("bf16,renorm", [(False, True), (True, False), (True, True), (False, False)])
def test_route_bwd(T, E, k, bf16, renorm):
    z = dev(logits_of(T, E, T * E, bf16))
    r = api.moe_route(z, k, renorm=renorm)
    a = torch.randn(T, k, generator=torch.Generator().manual_seed(k))
    check_route_bwd(z, r, a, 1.5, 0.1, renorm)
    check_route_bwd(z, r, a, None, 0.1, renorm)
    check_route_bwd(z, r, None, 0.5, 0.1, renorm)
    check_route_bwd(z, r, None, None, 0.1, renorm)


@pytest.mark.parametrize("kind", ["ties", "shut", "lowest", "wide"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_bwd_difficult_logits(kind, renorm):
    T, E, k = 111, 48, 6
    z = dev(logits_of(T, E, 6, False, kind))
    r = api.moe_route(z, k, renorm=renorm)
    check_route_bwd(z, r, torch.randn(T, k, generator=torch.Generator().manual_seed(0)), 2.0, 0.3, renorm)


@pytest.mark.parametrize("T,E", [(40, 24), (300, 24), (5000, 24), (40000, 24), (3000, 300)])
def test_route_loss_and_sums_each_alone(T, E):
    """Every launch shape with the sums but no loss, and with the loss but no sums."""
    z = dev(logits_of(T, E, T))
    both = api.moe_route(z, 2, balance_coef=0.25)
    sums = torch.full((E,), -1.0, device="cuda")
    bufs = [torch.empty_like(t) for t in both[:7]]
    r = api.moe_route(z, 2, out=(*bufs, sums, None))
    assert torch.equal(sums, both.prob_sums) and r.loss is None
    loss = torch.full((1,), -1.0, device="cuda")
    r = api.moe_route(z, 2, balance_coef=0.25, out=(*bufs, None, loss))
    assert torch.equal(loss, both.loss) and all(torch.equal(a, b) for a, b in zip(r[:7], both[:7]))


def test_route_bwd_with_counts_of_all_ranks():
    """Counts summed over ranks: each rank's gradient is its rows of the gradient of the loss over all tokens."""
    T, E, k = 90, 20, 3
    z = [dev(logits_of(T, E, s)) for s in (1, 2)]
    whole = api.moe_route(torch.cat(z), k)
    one = torch.ones(1, device="cuda")
    want = api.moe_route_bwd(torch.cat(z), whole.expert_ids, whole.weights, counts=whole.counts, dloss=one,
                             balance_coef=0.7)
    parts = [api.moe_route(x, k) for x in z]
    counts = parts[0].counts + parts[1].counts
    assert torch.equal(counts, whole.counts)
    for i, (x, r) in enumerate(zip(z, parts)):
        d = api.moe_route_bwd(x, r.expert_ids, r.weights, counts=counts, dloss=one, balance_coef=0.7)
        assert torch.equal(d, want[i * T:(i + 1) * T])


def test_route_bwd_of_an_empty_slot_ignores_its_gradient():
    z = dev(logits_of(50, 8, 2, False, "shut"))
    r = api.moe_route(z, 6)
    a = torch.randn(50, 6, generator=torch.Generator().manual_seed(0))
    clean = api.moe_route_bwd(z, r.expert_ids, r.weights, dweights=dev(a))
    dirty = torch.where(r.expert_ids < 0, float("nan"), dev(a))
    assert torch.equal(api.moe_route_bwd(z, r.expert_ids, r.weights, dweights=dirty), clean)
    assert torch.isfinite(clean).all()


# ------------------------------------------------------------------ combine
def rows_of(T, k, R, seed, empty=0.2):
    g = np.random.default_rng(seed)
    rows = g.permutation(max(R, T * k))[:T * k].reshape(T, k)
    rows[g.random((T, k)) < empty] = -1
    if T > 1:
        rows[T // 2] = -1  # a token without slots
    return np.where(rows < R, rows, -1).astype(np.int32)


COMBINES = [(1, 1, 8), (3, 2, 64), (64, 8, 4096), (37, 6, 1000), (20, 32, 264), (11, 3, 10240), (129, 5, 2080)]


@pytest.mark.parametrize("T,k,H", COMBINES)
def test_combine(T, k, H):
    g = torch.Generator().manual_seed(T)
    R = T * k + 3
    rows = rows_of(T, k, R, H)
    y = torch.randn(R, H, generator=g).to(torch.bfloat16)
    y[np.setdiff1d(np.arange(R), rows)] = float("nan")  # rows of no slot are not looked at
    w = torch.rand(T, k, generator=g)
    wide = dev(torch.cat([y, torch.full((R, 8), float("nan"), dtype=y.dtype)], 1))[:, :H]  # ldy = H + 8
    for weights in (w, None):
        out = api.moe_combine(wide, dev(torch.from_numpy(rows)), None if weights is None else dev(weights))
        want, mag = ref.combine(n64(y), rows, None if weights is None else n64(weights))
        tol = (k + 1) * U * mag
        within(n64(out), want, tol + B * (abs(want) + tol), "combine")
        assert (n64(out)[(rows < 0).all(1)] == 0).all()


@pytest.mark.parametrize("T,k,H", COMBINES)
@pytest.mark.parametrize("y8", [False, True])
def test_combine_bwd(T, k, H, y8):
    g = torch.Generator().manual_seed(T + 1)
    R = T * k + 3
    if y8:
        H = -(-H // 32) * 32
    rows = rows_of(T, k, R, H)
    y = torch.randn(R, H, generator=g).to(torch.bfloat16)
    y[0, :32] = 0
    dout = (torch.randn(T, H, generator=g) * 1e-3).to(torch.bfloat16)
    w = torch.rand(T, k, generator=g)
    if y8:
        kept = api.quant_mxfp8(dev(y))
        y = decode8(*kept)
    else:
        kept = dev(y)
        y = n64(y)
    big = torch.full((R + 2, H + 16), 9.0, dtype=torch.bfloat16, device="cuda")
    dy = big[1:R + 1, 8:H + 8]
    _, dw = api.moe_combine_bwd(dev(dout), kept, dev(torch.from_numpy(rows)), dev(w),
                                out=(dy, torch.full((T, k), 7.0, device="cuda")))
    want_dy = np.full((R, H), 9.0)
    want_dw, mag = ref.combine_bwd(n64(dout), y, rows, n64(w), want_dy)
    within(n64(dy), want_dy, (U + B + U * B) * abs(want_dy), "dy")
    around = n64(big)
    around[1:R + 1, 8:H + 8] = 9
    assert (around == 9).all(), "written outside dy"
    # products, a thread's sum, the trees over lanes and warps
    within(n64(dw), want_dw, (H / 256 + 8 + 5 + 8 + 2) * U * mag, "dweights")
    assert (n64(dw)[rows < 0] == 0).all()


def test_combine_rows_out_of_range_add_nothing():
    y = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([[0, 4], [-7, 2 ** 31 - 1], [3, -2 ** 31]], dtype=torch.int32, device="cuda")
    w = torch.full((3, 2), 2.0, device="cuda")
    assert n64(api.moe_combine(y, rows, w))[:, 0].tolist() == [2, 0, 2]
    dy, dw = api.moe_combine_bwd(torch.ones(3, 64, dtype=torch.bfloat16, device="cuda"), y, rows, w)
    assert n64(dy)[:, 0].tolist() == [2, 0, 0, 2] and n64(dw).tolist() == [[64, 0], [0, 0], [64, 0]]


def test_combine_may_list_a_row_more_than_once():
    y = torch.arange(1, 5, device="cuda").to(torch.bfloat16)[:, None].expand(4, 64).contiguous()
    rows = torch.tensor([[3, 3, 3], [0, 3, 0]], dtype=torch.int32, device="cuda")
    assert n64(api.moe_combine(y, rows))[:, 7].tolist() == [12, 6]


def test_combine_without_tokens_or_rows():
    rows = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    y = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    assert api.moe_combine(y, rows).shape == (0, 64)
    none = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    y0 = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert (n64(api.moe_combine(y0, none)) == 0).all()
    dy, dw = api.moe_combine_bwd(torch.ones(3, 64, dtype=torch.bfloat16, device="cuda"), y0, none,
                                 torch.ones(3, 2, device="cuda"))
    assert dy.shape == (0, 64) and (n64(dw) == 0).all()
    dy, dw = api.moe_combine_bwd(torch.ones(3, 40, dtype=torch.bfloat16, device="cuda"), y0[:, :40].contiguous(), none,
                                 torch.ones(3, 2, device="cuda"))
    assert dy.shape == (0, 40) and (n64(dw) == 0).all()


# ------------------------------------------------------------------ gated SiLU
def decode8(codes, sf):
    """MXFP8 (codes [M, K], swizzled sf) in binary64, by the code's bits."""
    c = codes.cpu().numpy().astype(np.int64)
    M, K = c.shape
    e, m = (c >> 3) & 15, c & 7
    mag = np.where(e > 0, np.ldexp(1 + m / 8, e - 7), np.ldexp(m / 8, -6))
    r, b = np.arange(M)[:, None], np.arange(K // 32)[None, :]
    at = (r // 128 * (-(-(K // 32) // 4)) + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4
    scale = np.ldexp(1.0, sf.cpu().numpy().astype(np.int64)[at] - 127)
    return np.where(c >= 128, -mag, mag) * np.repeat(scale, 32, 1)


def gate_input(M, F, seed):
    u = torch.randn(M, 2 * F, generator=torch.Generator().manual_seed(seed)) * 3
    u[0, :32] = 0.0
    u[0, F:F + 16] = -0.0
    if M > 4:
        u[1, :F] = torch.linspace(-120, 120, F)     # sigmoid's ends
        u[2] *= 1e-38                               # subnormal products
        u[3] = u[3].sign() * 1e4                    # saturated gates
        u[4, :8] = torch.tensor([-1.2784645, 0.0, -0.0, 88.8, -88.8, 3.0e38, -3.0e38, 1.0])
        u[4, F:F + 8] = 1e-3                        # (products stay finite)
    return u.to(torch.bfloat16)


def swiglu_tol(u, want):
    """The sigmoid (2 |g| + 4 for the exponential, 1 + e, the reciprocal 2) and two products, all U; bf16's rounding,
    whose subnormal half step is 2^-134; a sigmoid of 0."""
    F = u.shape[1] // 2
    g, v = np.minimum(abs(u[:, :F]), 104), abs(u[:, F:])
    return (B + (2 * g + 10) * U) * abs(want) + 1e-40 + 2.0 ** -126 * g * v


def swiglu_bwd_tol(dh, u, mag, want):
    """The same sigmoid, 1 - s (its error is that of s), and five products and sums, relative to mag."""
    F = u.shape[1] // 2
    g, v = np.minimum(abs(u[:, :F]), 104), abs(u[:, F:])
    t = (2 * (2 * np.concatenate([g, g], 1) + 7) + 6) * U * mag
    t = t + 2.0 ** -126 * np.concatenate([abs(dh) * v * (1 + g), abs(dh) * g], 1)
    return t + B * (abs(want) + t) + 1e-40


SWIGLUS = [(1, 32), (5, 96), (130, 64), (64, 768), (37, 1376), (300, 256), (9, 4128)]


@pytest.mark.parametrize("M,F", SWIGLUS)
def test_swiglu_ckpt(ora, M, F):
    u = gate_input(M, F, M + F)
    wide = dev(torch.cat([u, torch.full((M, 8), float("nan"), dtype=u.dtype)], 1))[:, :2 * F]
    h, codes, sf, amax = api.swiglu_ckpt(wide)
    want = ref.swiglu(n64(u))
    within(n64(h), want, swiglu_tol(n64(u), want), "h")
    assert amax.item() == h.float().abs().max().item()
    qc, qs = api.quant_mxfp8(dev(u))
    assert torch.equal(codes, qc) and torch.equal(sf, qs)
    oc, os_ = ora.quant_mxfp8(bits(u))
    assert_codes_equal(codes.cpu().numpy(), oc, "checkpoint codes")
    assert_codes_equal(ora.sf_unswizzle(sf.cpu().numpy(), M, 2 * F // 32), os_, "checkpoint scales")


@pytest.mark.parametrize("M,F", SWIGLUS)
@pytest.mark.parametrize("again", [False, True])
def test_swiglu_ckpt_bwd(M, F, again):
    u = gate_input(M, F, M * F)
    codes, sf = api.quant_mxfp8(dev(u))
    v = decode8(codes, sf)
    dh = torch.randn(M, F, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16)
    wide = dev(torch.cat([dh, torch.full((M, 8), float("nan"), dtype=dh.dtype)], 1))[:, :F]
    out = (torch.zeros(M, 2 * F + 8, dtype=torch.bfloat16, device="cuda")[:, :2 * F],
           torch.zeros(M, F + 8, dtype=torch.bfloat16, device="cuda")[:, :F] if again else None)
    du, h = api.swiglu_ckpt_bwd(wide, codes, sf, out=out)
    with np.errstate(over="ignore"):
        want, mag = ref.swiglu_bwd(n64(dh), v)
        tol = swiglu_bwd_tol(n64(dh), v, mag, want)
        fine = np.isfinite(want) & (abs(want) < 1e38)  # 3e38 times dh passes bf16's range
        got = np.where(fine, n64(du), 0)
        want, tol = np.where(fine, want, 0), np.where(fine, tol, 0)
        within(got, want, tol, "du")
        assert again == (h is not None)
        if again:
            want = ref.swiglu(v)
            within(n64(h), want, swiglu_tol(v, want), "h")


@pytest.mark.parametrize("n", [0, 1, 33, 127, 200])
def test_swiglu_of_a_padded_buffer_leaves_the_rest(n):
    """Rows behind the count are neither read (they hold NaN) nor written."""
    M, F = 150, 96
    u = gate_input(M, F, 5)
    want = [t.clone() for t in api.swiglu_ckpt(dev(u[:max(min(n, M), 1)]))]
    u[n:] = float("nan")
    count = torch.tensor([n], dtype=torch.int32, device="cuda")
    nb = api.sf_bytes(M, F // 16)
    out = (torch.full((M, F), 9.0, dtype=torch.bfloat16, device="cuda"),
           torch.full((M, 2 * F), 9, dtype=torch.uint8, device="cuda"),
           torch.full((nb,), 9, dtype=torch.uint8, device="cuda"), torch.full((1,), 9.0, device="cuda"))
    h, codes, sf, amax = api.swiglu_ckpt(dev(u), n_rows=count, out=out)
    m = min(n, M)
    assert torch.equal(h[:m], want[0][:m]) and (h[m:] == 9).all()
    assert torch.equal(codes[:m], want[1][:m]) and (codes[m:] == 9).all()
    assert amax.item() == (want[3].item() if n else 0.0)
    r, b = np.arange(M)[:, None], np.arange(2 * F // 32)[None, :]
    at = (r // 128 * (-(-(2 * F // 32) // 4)) + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4
    got = sf.cpu().numpy()
    assert (got[at[m:]] == 9).all() and (np.delete(got, at.ravel()) == 9).all()
    dh = torch.full((M, F), float("nan"))
    dh[:m] = 0.5
    out = (torch.full((M, 2 * F), 9.0, dtype=torch.bfloat16, device="cuda"),
           torch.full((M, F), 9.0, dtype=torch.bfloat16, device="cuda"))
    du, again = api.swiglu_ckpt_bwd(dev(dh.to(torch.bfloat16)), codes, sf, n_rows=count, out=out)
    assert (du[m:] == 9).all() and (again[m:] == 9).all()
    assert torch.isfinite(du[:m]).all() and (m == 0 or not (du[:m] == 9).all())
    negative = torch.tensor([-5], dtype=torch.int32, device="cuda")
    h[:] = 9
    api.swiglu_ckpt(dev(u), n_rows=negative, out=(h, codes, sf, amax))
    assert (h == 9).all() and amax.item() == 0


def test_swiglu_without_rows():
    h, codes, sf, amax = api.swiglu_ckpt(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert h.shape == (0, 32) and amax.item() == 0
    du, _ = api.swiglu_ckpt_bwd(h, codes, sf)
    assert du.shape == (0, 64)


# ------------------------------------------------------------------ as a user calls them
def test_wrappers_refuse_what_the_library_cannot_see():
    z = torch.zeros(4, 8, device="cuda")
    i = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    y = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    d = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    u = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    n = torch.zeros(1, dtype=torch.int64, device="cuda")
    s = torch.zeros(api.sf_bytes(8, 2), dtype=torch.uint8, device="cuda")
    for bad in [lambda: api.moe_route(z.double(), 2), lambda: api.moe_route(z.cpu(), 2), lambda: api.moe_route(z, 9),
                lambda: api.moe_route(z.t(), 2), lambda: api.moe_route(z, 2, token_mask=torch.ones(4, device="cuda")),
                lambda: api.moe_route(z, 2, token_mask=torch.ones(5, dtype=torch.uint8, device="cuda")),
                lambda: api.moe_route(z, 2, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
                lambda: api.moe_route_bwd(z, i.long(), w), lambda: api.moe_route_bwd(z, i, w[:3]),
                lambda: api.moe_route_bwd(z, i, w, dloss=torch.ones(1, device="cuda")),
                lambda: api.moe_combine(y.float(), i), lambda: api.moe_combine(y, i.long()),
                lambda: api.moe_combine(y[:, :60], i), lambda: api.moe_combine(y, i, w.t()),
                lambda: api.moe_combine_bwd(d.float(), y, i, w), lambda: api.moe_combine_bwd(d[:3], y, i, w),
                lambda: api.moe_combine_bwd(d, (y, s), i, w), lambda: api.moe_combine_bwd(d, y, i, None),
                lambda: api.swiglu_ckpt(u.float()), lambda: api.swiglu_ckpt(u[:, :48]),
                lambda: api.swiglu_ckpt(u, n_rows=n), lambda: api.swiglu_ckpt(u[:, ::2]),
                lambda: api.swiglu_ckpt_bwd(u[:, :32], y.view(torch.uint8)[:, :64], s[:8]),
                lambda: api.swiglu_ckpt_bwd(u[:, :32], u, s)]:
        with pytest.raises((bsq.BsqError, AttributeError)):
            bad()


def test_same_bits_every_time_on_two_streams_at_once():
    T, E, k, H = 3000, 96, 6, 512
    z = dev(logits_of(T, E, 1, False, "ties"))
    first = api.moe_route(z, k, balance_coef=0.1)
    y = torch.randn(T * k, H, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    dout = torch.randn(T, H, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    want = api.moe_combine_bwd(dout, y, first.rows, first.weights)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                r = api.moe_route(z, k, balance_coef=0.1)
                got.append((r, api.moe_combine_bwd(dout, y, r.rows, r.weights)))
    torch.cuda.synchronize()
    for r, c in got:
        assert all(torch.equal(a, b) for a, b in zip(r, first))
        assert all(torch.equal(a, b) for a, b in zip(c, want))


def test_offsets_past_31_bits():
    """Tensors of more than 2^31 elements: rows at both ends against the same rows alone."""
    T, E = 8_500_000, 256                                                   # 2.2e9 logits
    want = torch.randint(0, E, (T,), device="cuda", dtype=torch.int32)
    z = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    z.scatter_(1, want.long()[:, None], 1.0)
    r = api.moe_route(z, 1, balance_coef=1.0)
    assert torch.equal(r.expert_ids[:, 0], want)
    order = torch.sort(want, stable=True).indices
    assert torch.equal(r.row_index, order.int())
    assert torch.equal(r.rows[:, 0].long()[order], torch.arange(T, device="cuda"))
    assert torch.equal(r.counts[:E], torch.bincount(want, minlength=E).int())
    one = torch.ones(1, device="cuda")
    d = api.moe_route_bwd(z, r.expert_ids, r.weights, counts=r.counts, dloss=one, balance_coef=1e6)
    for at in (slice(0, 9), slice(T - 9, T)):
        alone = api.moe_route_bwd(z[at].clone(), r.expert_ids[at], r.weights[at], counts=r.counts, dloss=one,
                                  balance_coef=1e6)
        assert torch.equal(d[at], alone) and (alone != 0).any()
    del z, d, r, order, want
    R, H = 300_000, 8192                                                    # 2.5e9 values
    y = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")
    y[-4:] = torch.randn(4, H, device="cuda")
    rows = torch.tensor([[R - 1, 0], [R - 3, R - 4]], dtype=torch.int32, device="cuda")
    w = torch.rand(2, 2, device="cuda")
    near = torch.tensor([[3, -1], [1, 0]], dtype=torch.int32, device="cuda")  # in the last four rows
    assert torch.equal(api.moe_combine(y, rows, w), api.moe_combine(y[-4:].clone(), near, w))
    g = torch.randn(2, H, device="cuda").to(torch.bfloat16)
    dy, dw = api.moe_combine_bwd(g, y, rows, w)
    dy4, dw4 = api.moe_combine_bwd(g, y[-4:].clone(), near, w)
    assert torch.equal(dy[-4:], dy4) and torch.equal(dw, dw4)
    codes, sf = api.quant_mxfp8(y)
    _, dw8 = api.moe_combine_bwd(g, (codes, sf), rows, w, out=(dy, dw))
    _, dw84 = api.moe_combine_bwd(g, api.quant_mxfp8(y[-4:].clone()), near, w)
    assert torch.equal(dw8, dw84)
    del dy, codes, sf
    u = y.view(R * 4, 2048)                                                 # gate and v of 1024 columns each
    h, codes, sf, am = api.swiglu_ckpt(u)
    h4, codes4, _, am4 = api.swiglu_ckpt(u[-16:].clone())
    assert torch.equal(h[-16:], h4) and torch.equal(codes[-16:], codes4) and am.item() == am4.item() > 0
    dh = torch.zeros_like(h)
    dh[-16:] = 1
    du, _ = api.swiglu_ckpt_bwd(dh, codes, sf)
    du4, _ = api.swiglu_ckpt_bwd(dh[-16:].clone(), *api.quant_mxfp8(u[-16:].clone()))
    assert torch.equal(du[-16:], du4) and (du4 != 0).any()


class Layer:
    """A mixture-of-experts layer's forward and backward pass in the library's calls."""

    def __init__(self, H, F, E, k, seed):
        g = torch.Generator().manual_seed(seed)
        self.H, self.F, self.E, self.k = H, F, E, k
        up = (torch.randn(E, 2 * F, H, generator=g) * 0.1).to(torch.bfloat16).cuda()
        dn = (torch.randn(E, H, F, generator=g) * 0.1).to(torch.bfloat16).cuda()

        def stack(qs):
            return [torch.stack([q[0] for q in qs]), torch.cat([q[1] for q in qs])] + (
                [torch.cat([q[2] for q in qs])] if len(qs[0]) > 2 else [])

        self.up = stack([api.quant_nvfp4(w, block_2d=True) for w in up])
        self.dn = stack([api.quant_nvfp4(w, block_2d=True) for w in dn])
        self.up_t = stack([api.quant_mxfp8(w.t().contiguous()) for w in up])
        self.dn_t = stack([api.quant_mxfp8(w.t().contiguous()) for w in dn])

    def rows8(self, x, r, R):
        """Rows of x in MXFP8 with their scales in the grouped GEMM's layout."""
        c, s = api.quant_mxfp8(x)
        nb = x.shape[1] // 32
        plain = torch.empty(R, nb, dtype=torch.uint8, device="cuda")
        bsq.bsq_sf_to_rows(s, R, nb, plain)
        out = torch.zeros(api.sf_bytes(R + 127 * self.E, nb), dtype=torch.uint8, device="cuda")
        bsq.bsq_sf_from_rows(plain, R, nb, self.E, r.row_offsets, r.sf_row_offsets, out)
        return c, out

    def step(self, x, z, dout, mask):
        H, F, E, k = self.H, self.F, self.E, self.k
        R = x.shape[0] * k
        r = api.moe_route(z, k, token_mask=mask, balance_coef=0.01)
        n = r.row_offsets[E:]
        groups = (r.row_offsets, r.sf_row_offsets, R + 127 * E)
        c, s, g = api.quant_nvfp4_gather(x, r.row_index, four_over_six=True, groups=groups)
        u = api.grouped_gemm(0, r.row_offsets, r.sf_row_offsets, c, s, self.up[0], self.up[1], R, 2 * F, H, gsA=g,
                             gsB=self.up[2])
        h, uc, us, am = api.swiglu_ckpt(u, n_rows=n)
        c, s, g = api.quant_nvfp4(h, four_over_six=True, groups=groups, amax_in=am)
        y = api.grouped_gemm(0, r.row_offsets, r.sf_row_offsets, c, s, self.dn[0], self.dn[1], R, H, F, gsA=g,
                             gsB=self.dn[2])
        out = api.moe_combine(y, r.rows, r.weights)
        # backward
        dy, dw = api.moe_combine_bwd(dout, y, r.rows, r.weights)
        c, s = self.rows8(dy, r, R)
        dh = api.grouped_gemm(1, r.row_offsets, r.sf_row_offsets, c, s, self.dn_t[0], self.dn_t[1], R, F, H)
        du, again = api.swiglu_ckpt_bwd(dh, uc, us, n_rows=n, recompute_h=True)
        c, s = self.rows8(du, r, R)
        dxr = api.grouped_gemm(1, r.row_offsets, r.sf_row_offsets, c, s, self.up_t[0], self.up_t[1], R, H, 2 * F)
        dx = api.moe_combine(dxr, r.rows)
        dz = api.moe_route_bwd(z, r.expert_ids, r.weights, dweights=dw, counts=r.counts,
                               dloss=torch.ones(1, device="cuda"), balance_coef=0.01)
        return dict(r=r, u=u, h=h, uc=uc, us=us, am=am, y=y, out=out, dy=dy, dw=dw, dh=dh, du=du, again=again, dxr=dxr,
                    dx=dx, dz=dz)


def layer_inputs(T, H, E, seed):
    g = torch.Generator().manual_seed(seed)
    return (dev(torch.randn(T, H, generator=g).to(torch.bfloat16)), dev(torch.randn(T, E, generator=g)),
            dev(torch.randn(T, H, generator=g).to(torch.bfloat16)),
            dev((torch.rand(T, generator=g) < 0.85).to(torch.uint8)))


def test_layer_forward_and_backward():
    """Each operator against its binary64 form on what the call before it gave, in one chain with the
    quantizers and grouped GEMMs on a padded batch."""
    T, H, F, E, k = 300, 256, 128, 6, 2
    x, z, dout, mask = layer_inputs(T, H, E, 11)
    o = Layer(H, F, E, k, 1).step(x, z, dout, mask)
    assert bsq.bsq_check() == bsq.BSQ_OK
    r = o["r"]
    check_route(r, z, k, mask, True, 0.01)
    n = int(r.row_offsets[E])
    assert 0 < n < T * k
    rows, w = ints(r.rows), n64(r.weights)
    want = ref.swiglu(n64(o["u"][:n]))
    within(n64(o["h"][:n]), want, swiglu_tol(n64(o["u"][:n]), want), "h")
    assert o["am"].item() == o["h"][:n].float().abs().max().item()
    want, mag = ref.combine(n64(o["y"][:n]), rows, w)
    within(n64(o["out"]), want, 3 * U * mag + B * (abs(want) + 3 * U * mag), "out")
    want_dy = np.zeros((n, H))
    want, mag = ref.combine_bwd(n64(dout), n64(o["y"][:n]), rows, w, want_dy)
    within(n64(o["dw"]), want, 40 * U * mag, "dw")
    within(n64(o["dy"][:n]), want_dy, (U + B + U * B) * abs(want_dy), "dy")
    assert (n64(o["dy"][n:]) == 0).all()
    v = decode8(o["uc"][:n], o["us"])
    want, mag = ref.swiglu_bwd(n64(o["dh"][:n]), v)
    within(n64(o["du"][:n]), want, swiglu_bwd_tol(n64(o["dh"][:n]), v, mag, want), "du")
    want = ref.swiglu(v)
    within(n64(o["again"][:n]), want, swiglu_tol(v, want), "h again")
    want, mag = ref.combine(n64(o["dxr"][:n]), rows, None)
    within(n64(o["dx"]), want, 3 * U * mag + B * (abs(want) + 3 * U * mag), "dx")
    check_route_bwd(z, r, o["dw"].cpu(), 1.0, 0.01, True)


def test_launch_overlap_changes_no_byte(knobs):
    """Back-to-back steps, each call reading what the one before it wrote, with and without overlapped launches."""
    layer = Layer(128, 128, 4, 2, 3)
    ins = layer_inputs(150, 128, 4, 5)
    got = []
    for overlap in (0, 1):
        knobs(bsq.BSQ_KNOB_LAUNCH_OVERLAP, overlap)
        for _ in range(3):
            o = layer.step(*ins)
        torch.cuda.synchronize()
        got.append(o)
    n = int(got[0]["r"].row_offsets[4])
    for name in ("out", "dw", "dx", "dz", "am"):
        assert torch.equal(got[0][name], got[1][name]), name
    for name in ("h", "du", "again"):
        assert torch.equal(got[0][name][:n], got[1][name][:n]), name
    assert bsq.bsq_check() == bsq.BSQ_OK


def test_layer_replayed_from_a_graph():
    """The whole step captured once and replayed on new inputs gives the eager calls' bytes."""
    T, H, F, E, k = 130, 128, 128, 5, 3
    layer = Layer(H, F, E, k, 2)
    ins = list(layer_inputs(T, H, E, 21))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(*ins)  # every call once outside capture
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = layer.step(*ins)
    for seed in (22, 23):
        for a, b in zip(ins, layer_inputs(T, H, E, seed)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want = layer.step(*ins)
        torch.cuda.synchronize()
        n = int(want["r"].row_offsets[E])
        for name in ("out", "dw", "dx", "dz", "am"):
            assert torch.equal(o[name], want[name]), name
        for name in ("h", "du", "again"):
            assert torch.equal(o[name][:n], want[name][:n]), name
        assert all(torch.equal(a, b) for a, b in zip(o["r"], want["r"]))
    assert bsq.bsq_check() == bsq.BSQ_OK
