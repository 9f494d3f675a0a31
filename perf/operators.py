"""The training operators of a mixture-of-experts layer, as cases that can be timed and compared.

Four operators, each in its plain form (elementary torch operations in 32 bits) and as the framework's
calls (``own``):

* ``route``: router logits -> the top-k experts of each token with their weights, the counts per expert
  and the row order that the grouped quantizer and GEMM take; with ``loss``, the balance loss too;
* ``route_bwd``: the gradient of the logits from the weights' gradient and the balance loss's;
* ``combine`` / ``combine_bwd``: the weighted sum of a token's expert rows, and the gradients of rows and
  weights (the rows kept in bf16, or in 8 bits);
* ``swiglu`` / ``swiglu_bwd``: the gated SiLU whose input is kept in 8 bits (MXFP8) for the backward pass.

Sizes: the mixture-of-experts workload has 16384 tokens, hidden size 4096, 64 experts, top-8 and up
projections of 1536 outputs, here a gate and an up half of 768 each; rollout steps have 64 tokens.
"""
import torch

own = False

NEG = float("-inf")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one step of a rollout: the whole call is latency
        dict(name="route rollout 64x64", op="route", T=64, E=64, k=8, bf16=False, renorm=True, loss=False, mask=0.0),
        # the training workload's router, with its balance loss
        dict(name="route train 16384x64", op="route", T=16384, E=64, k=8, bf16=False, renorm=True, loss=True, mask=0.0),
        # a long batch over many experts, padded, logits in bf16
        dict(name="route long 131072x256", op="route", T=131072, E=256, k=8, bf16=True, renorm=True, loss=True,
             mask=0.1),
        dict(name="route bwd 16384x64", op="route_bwd", T=16384, E=64, k=8, bf16=False, renorm=True, loss=True,
             mask=0.0),
        # odd counts, weights straight from the softmax over all experts
        dict(name="route bwd 100003x160", op="route_bwd", T=100003, E=160, k=6, bf16=True, renorm=False, loss=True,
             mask=0.2),
        dict(name="combine rollout 64x8x4096", op="combine", T=64, k=8, H=4096, mask=0.0),
        dict(name="combine train 16384x8x4096", op="combine", T=16384, k=8, H=4096, mask=0.0),
        dict(name="combine bwd 16384x8x4096", op="combine_bwd", T=16384, k=8, H=4096, mask=0.0, y8=False),
        # a padded, ragged batch whose expert rows were kept in 8 bits
        dict(name="combine bwd 5003x6x2080 y8", op="combine_bwd", T=5003, k=6, H=2080, mask=0.3, y8=True),
        # the up projection's output of the training workload's routed rows
        dict(name="swiglu train 131072x768", op="swiglu", M=131072, F=768, part=1.0),
        # its backward, with h formed again for the down projection's weight gradient
        dict(name="swiglu bwd 131072x768", op="swiglu_bwd", M=131072, F=768, part=1.0, h=True),
        # a rollout's routed rows, a padded buffer
        dict(name="swiglu rollout 515x1376", op="swiglu", M=515, F=1376, part=0.9),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "combine", "combine_bwd", "swiglu", "swiglu_bwd"])
    if op in ("route", "route_bwd"):
        E = rng.choice([_log(rng, 4, 256), 8 * _log(rng, 1, 32)])
        return dict(op=op, T=_log(rng, 16, 131072), E=E, k=rng.randint(1, min(E, 10)), bf16=rng.random() < 0.5,
                    renorm=rng.random() < 0.5, loss=rng.random() < 0.7, mask=rng.choice([0.0, 0.05, 0.5]))
    if op in ("combine", "combine_bwd"):
        c = dict(op=op, T=_log(rng, 16, 16384), k=rng.randint(1, 8), H=8 * _log(rng, 8, 512),
                 mask=rng.choice([0.0, 0.05, 0.5]))
        if op == "combine_bwd":
            c["y8"] = rng.random() < 0.5
            c["H"] = 32 * _log(rng, 2, 128) if c["y8"] else c["H"]  # whole blocks of 32
        return c
    c = dict(op=op, M=_log(rng, 64, 131072), F=32 * _log(rng, 2, 24), part=rng.choice([1.0, 0.9, 0.4]))
    return dict(c, h=rng.random() < 0.5) if op == "swiglu_bwd" else c


def work(case):
    op = case["op"]
    if op in ("route", "route_bwd"):
        T, E, k, b = case["T"], case["E"], case["k"], 2 if case["bf16"] else 4
        m = T if case["mask"] else 0
        if op == "route":
            return {"bytes": T * E * b + m + 16 * T * k + 4 * (4 * E + 4), "flops": 5 * T * E}
        reads = T * E * b if case["loss"] or not case["renorm"] else 0
        return {"bytes": T * E * b + reads + m + 12 * T * k + 4 * E, "flops": 10 * T * E}
    if op in ("combine", "combine_bwd"):
        T, k, H = case["T"], case["k"], case["H"]
        rows = int(round(T * (1 - case["mask"]))) * k  # the rows that some token has
        if op == "combine":
            return {"bytes": 2 * H * (rows + T) + 8 * T * k, "flops": 2 * rows * H}
        y = 1 + 1 / 32 if case["y8"] else 2
        return {"bytes": H * (rows * (y + 2) + 2 * rows // k) + 12 * T * k, "flops": 3 * rows * H}
    M, F = int(case["M"] * case["part"]), case["F"]
    if op == "swiglu":
        return {"bytes": M * F * (4 + 2 + 2 + 1 / 16), "flops": 8 * M * F}
    return {"bytes": M * F * (2 + 2 + 1 / 16 + 4 + (2 if case["h"] else 0)), "flops": 16 * M * F}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _mask(T, share, g):
    """1 for a token, 0 for padding; padding comes at the end of a batch's sequences, so in runs."""
    if not share:
        return None
    run = 64
    n = -(-T // run)
    length = torch.rand(n, generator=g, device="cuda") * 2 * share  # share of each run that is padding
    at = torch.arange(T, device="cuda")
    return ((at % run) < (1 - length[at // run]) * run).to(torch.uint8)


def _routing(T, E, k, mask, g):
    """Expert ids [T, k] of random tokens and the rows they have, ordered by expert, then token."""
    z = torch.randn(T, E, generator=g, device="cuda")
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    gone = torch.zeros(T, dtype=torch.bool, device="cuda") if mask is None else mask == 0
    key = torch.where(gone[:, None], E, ids).reshape(-1)
    order = torch.sort(key, stable=True).indices
    rows = torch.empty_like(order)
    rows[order] = torch.arange(T * k, device="cuda")
    rows = torch.where(gone[:, None], -1, rows.view(T, k))
    return rows.to(torch.int32), (~gone).sum() * k


def _quant8(x):
    """MXFP8 of rows: codes [M, K] and one scale byte for each 32 values, in the layout of the matrix units."""
    M, K = x.shape
    b = x.float().view(M, K // 32, 32)
    top = b.abs().amax(2)
    e = torch.where(top > 0, torch.frexp(top).exponent.float() - 1 - 8, -127.0).clamp(-127, 127)
    q = (b * torch.exp2(-e)[:, :, None]).clamp(-448, 448)
    fine = torch.exp2((torch.frexp(q).exponent.float() - 1).clamp(min=-6) - 3)  # an e4m3 step at q
    q = torch.round(q / fine) * fine
    return q.view(M, K).to(torch.float8_e4m3fn).view(torch.uint8), _swizzle((e + 127).to(torch.uint8))


def _swizzle(s):
    M, n = s.shape
    full = torch.zeros(-(-M // 128) * 128, -(-n // 4) * 4, dtype=torch.uint8, device=s.device)
    full[:M, :n] = s
    return full.view(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _unswizzle(s, M, n):
    bt = -(-n // 4)
    return s.view(-1, bt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, bt * 4)[:M, :n]


def _decode8(codes, sf):
    M, K = codes.shape
    e = _unswizzle(sf, M, K // 32).float() - 127
    return (codes.view(torch.float8_e4m3fn).float().view(M, K // 32, 32) * torch.exp2(e)[:, :, None]).view(M, K)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=dict(case))
    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        # logits as a router's: some experts preferred by all, each token with its own
        z = torch.randn(T, E, generator=g, device="cuda") * 1.5 + torch.randn(E, generator=g, device="cuda") * 0.5
        st["logits"] = z.to(torch.bfloat16) if case["bf16"] else z
        st["mask"] = _mask(T, case["mask"], g)
        i32 = dict(dtype=torch.int32, device="cuda")
        f32 = dict(dtype=torch.float32, device="cuda")
        if op == "route":
            # what a program keeps from step to step: the plan's buffers and the workspace
            st["out"] = (torch.empty(T, k, **i32), torch.empty(T, k, **f32), torch.empty(T, k, **i32),
                         torch.empty(T * k, **i32), torch.empty(E + 1, **i32), torch.empty(E + 1, **i32),
                         torch.empty(E + 1, **i32), torch.empty(E, **f32) if case["loss"] else None,
                         torch.empty(1, **f32) if case["loss"] else None)
            st["workspace"] = None
        else:
            r = _route(st["logits"], st["mask"], k, case["renorm"], 0.0)
            st["ids"], st["weights"], st["counts"] = r["ids"], r["weights"], r["counts"]
            st["dweights"] = torch.randn(T, k, generator=g, device="cuda") * 0.1
            st["dloss"] = torch.full((1,), 1.0, device="cuda") if case["loss"] else None
            st["dlogits"] = torch.empty_like(st["logits"])
    elif op in ("combine", "combine_bwd"):
        T, k, H = case["T"], case["k"], case["H"]
        mask = _mask(T, case["mask"], g)
        st["rows"], st["n"] = _routing(T, max(2 * k, 64), k, mask, g)
        w = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
        st["weights"] = torch.where(st["rows"] < 0, 0.0, w)
        y = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
        for r in range(0, T * k, 16384):
            y[r:r + 16384] = torch.randn(y[r:r + 16384].shape, generator=g, device="cuda") * 0.05
        if op == "combine":
            st["y"] = y
            st["out"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        else:
            st["y"] = _quant8(y) if case["y8"] else y
            st["dout"] = (torch.randn(T, H, generator=g, device="cuda") * 1e-3).to(torch.bfloat16)
            st["dy"] = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
            st["dweights"] = torch.empty(T, k, dtype=torch.float32, device="cuda")
    else:
        M, F = case["M"], case["F"]
        u = (torch.randn(M, 2 * F, generator=g, device="cuda") * 1.3).to(torch.bfloat16)
        n = int(M * case["part"])
        st["n"] = torch.full((1,), n, dtype=torch.int32, device="cuda") if n < M else None
        if op == "swiglu":
            st["u"] = u
            st["out"] = (torch.zeros(M, F, dtype=torch.bfloat16, device="cuda"),
                         torch.zeros(M, 2 * F, dtype=torch.uint8, device="cuda"),
                         torch.zeros(-(-M // 128) * 128 * (-(-F // 64) * 4), dtype=torch.uint8, device="cuda"),
                         torch.empty(1, dtype=torch.float32, device="cuda"))
        else:
            st["codes"], st["sf"] = _quant8(u)
            st["dh"] = (torch.randn(M, F, generator=g, device="cuda") * 1e-3).to(torch.bfloat16)
            st["out"] = (torch.zeros(M, 2 * F, dtype=torch.bfloat16, device="cuda"),
                         torch.zeros(M, F, dtype=torch.bfloat16, device="cuda") if case["h"] else None)
    return st


# ------------------------------------------------------------------ plain forms
def _softmax(z, mask):
    """Softmax rows in 32 bits; a masked row, and one with nothing but -inf, gives zeros."""
    z = z.float()
    if mask is not None:
        z = torch.where(mask[:, None] != 0, z, NEG)
    top = z.amax(1, keepdim=True)
    x = torch.exp(z - torch.where(top == NEG, 0.0, top))
    s = x.sum(1, keepdim=True)
    return z, x / torch.where(s > 0, s, 1.0)


def _route(logits, mask, k, renorm, coef):
    T, E = logits.shape
    z, p = _softmax(logits, mask)
    best = torch.sort(z, dim=1, descending=True, stable=True)
    empty = best.values[:, :k] == NEG
    ids = torch.where(empty, -1, best.indices[:, :k])
    w = torch.where(empty, 0.0, torch.gather(p, 1, ids.clamp(min=0)))
    if renorm:
        top = torch.where(empty, NEG, best.values[:, :k])
        x = torch.where(empty, 0.0, torch.exp(top - torch.where(empty[:, :1], 0.0, top[:, :1])))
        s = x.sum(1, keepdim=True)
        w = x / torch.where(s > 0, s, 1.0)
    flat = torch.where(empty, E, ids).reshape(-1)
    count = torch.zeros(E + 1, dtype=torch.int64, device=z.device).index_add_(0, flat, torch.ones_like(flat))[:E]
    order = torch.sort(flat, stable=True).indices
    at = torch.arange(T * k, device=z.device)
    rows = torch.empty_like(order)
    rows[order] = at
    total = count.sum()
    token = order // k
    row_index = torch.where(at < total, token, torch.where(total > 0, token[0], 0))
    n = (~empty[:, 0]).sum()
    zero = torch.zeros(1, dtype=torch.int64, device=z.device)
    psum = p.sum(0)
    loss = coef * E * (count.float() * psum).sum() / (k * n.float() * n.float()).clamp(min=1)
    i = lambda t: t.to(torch.int32)  # noqa: E731
    return dict(ids=i(ids), weights=w, rows=i(torch.where(empty, -1, rows.view(T, k))), row_index=i(row_index),
                row_offsets=i(torch.cat([zero, count.cumsum(0)])),
                sf_row_offsets=i(torch.cat([zero, ((count + 127) // 128 * 128).cumsum(0)])),
                counts=i(torch.cat([count, n[None]])), prob_sums=psum, loss=loss[None])


def _route_bwd(logits, mask, ids, weights, dweights, counts, renorm, coef, dloss):
    T, E = logits.shape
    k = ids.shape[1]
    _, p = _softmax(logits, mask)
    empty = ids < 0
    at = ids.clamp(min=0).long()
    dw = torch.where(empty, 0.0, dweights)
    d = torch.zeros_like(p)
    if renorm:
        d.scatter_add_(1, at, weights * (dw - (dw * weights).sum(1, keepdim=True)))
    else:
        d.scatter_add_(1, at, dw)
        d = p * (d - (d * p).sum(1, keepdim=True))
    if dloss is not None:
        n = counts[E].float().clamp(min=1)
        f = counts[:E].float() / (k * n)
        d = d + dloss * coef * E / n * p * (f - (p * f).sum(1, keepdim=True))
    return d.to(logits.dtype)


def _swiglu_bwd(dh, codes, sf, n, du, h):
    n = dh.shape[0] if n is None else int(n)
    F = dh.shape[1]
    v = _decode8(codes, sf)[:n]
    g, u, d = v[:, :F], v[:, F:], dh[:n].float()
    s = torch.sigmoid(g)
    du[:n, :F] = (d * u * s * (1 + g * (1 - s))).to(torch.bfloat16)
    du[:n, F:] = (d * g * s).to(torch.bfloat16)
    if h is not None:
        h[:n] = (g * s * u).to(torch.bfloat16)


COEF = 0.01


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        return _run_own(st, case, op)
    if op == "route":
        r = _route(st["logits"], st["mask"], case["k"], case["renorm"], COEF)
        if not case["loss"]:
            del r["prob_sums"], r["loss"]
        return r
    if op == "route_bwd":
        return _route_bwd(st["logits"], st["mask"], st["ids"], st["weights"], st["dweights"], st["counts"],
                          case["renorm"], COEF, st["dloss"])
    if op == "combine":
        rows = st["rows"].long()
        part = torch.where(rows[:, :, None] >= 0, st["y"][rows.clamp(min=0)].float(), 0.0)
        return (part * st["weights"][:, :, None]).sum(1).to(torch.bfloat16)
    if op == "combine_bwd":
        y = _decode8(*st["y"]) if case["y8"] else st["y"]
        rows = st["rows"].long()
        d = st["dout"].float()
        has = rows >= 0
        part = torch.where(has[:, :, None], y[rows.clamp(min=0)].float(), 0.0)
        dw = (part * d[:, None, :]).sum(2)
        del part
        dy = st["dy"]
        t = torch.arange(rows.shape[0], device=rows.device)[:, None].expand_as(rows)[has]
        dy[rows[has]] = (st["weights"][has][:, None] * d[t]).to(torch.bfloat16)
        return dict(dy=dy, dweights=dw)
    if op == "swiglu":
        h, codes, sf, _ = st["out"]
        n = case["M"] if st["n"] is None else int(st["n"])
        F = case["F"]
        g, u = st["u"][:n, :F].float(), st["u"][:n, F:].float()
        h[:n] = (g * torch.sigmoid(g) * u).to(torch.bfloat16)
        c, s = _quant8(st["u"][:n])
        codes[:n] = c
        M = case["M"]
        keep = _unswizzle(sf, M, 2 * F // 32).clone()
        keep[:n] = _unswizzle(s, n, 2 * F // 32)
        return _swiglu_out(h, codes, _swizzle(keep), h[:n].float().abs().max()[None])
    du, h = st["out"]
    _swiglu_bwd(st["dh"], st["codes"], st["sf"], st["n"], du, h)
    return (du, h) if h is not None else (du,)


def _swiglu_out(h, codes, sf, amax):
    # the 8-bit codes as the numbers they are: e4m3 elements and power-of-two scales
    return dict(h=h, codes=codes.view(torch.float8_e4m3fn), scales=sf.view(torch.float8_e8m0fnu), amax=amax)


def _run_own(st, case, op):
    from fp8_math_b200 import api

    if op == "route":
        if st["workspace"] is None:
            st["workspace"] = torch.empty(api.moe_route_workspace(case["T"], case["E"]), dtype=torch.uint8,
                                          device="cuda")
        r = api.moe_route(st["logits"], case["k"], token_mask=st["mask"], renorm=case["renorm"],
                          balance_coef=COEF if case["loss"] else None, out=st["out"], workspace=st["workspace"])
        names = ("ids", "weights", "rows", "row_index", "row_offsets", "sf_row_offsets", "counts", "prob_sums", "loss")
        return {n: t for n, t in zip(names, r) if t is not None}
    if op == "route_bwd":
        return api.moe_route_bwd(st["logits"], st["ids"], st["weights"], dweights=st["dweights"], counts=st["counts"],
                                 dloss=st["dloss"], balance_coef=COEF, renorm=case["renorm"], out=st["dlogits"])
    if op == "combine":
        return api.moe_combine(st["y"], st["rows"], st["weights"], out=st["out"])
    if op == "combine_bwd":
        dy, dw = api.moe_combine_bwd(st["dout"], st["y"], st["rows"], st["weights"], out=(st["dy"], st["dweights"]))
        return dict(dy=dy, dweights=dw)
    if op == "swiglu":
        return _swiglu_out(*api.swiglu_ckpt(st["u"], n_rows=st["n"], out=st["out"]))
    du, h = api.swiglu_ckpt_bwd(st["dh"], st["codes"], st["sf"], n_rows=st["n"], out=st["out"])
    return (du, h) if h is not None else (du,)


# ------------------------------------------------------------------ 64 bits, from the definitions
def _mx_value64(codes, sf):
    """Values of an MXFP8 tensor by its bits: sign, four exponent bits (bias 7), three fraction bits, times 2^(s-127)."""
    M, K = codes.shape
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, torch.ldexp(1 + m / 8, e - 7), torch.ldexp(m / 8, torch.full_like(e, -6)))
    r = torch.arange(M, device=codes.device)[:, None]
    b = torch.arange(K // 32, device=codes.device)[None, :]
    at = (r // 128 * (-(-(K // 32) // 4)) + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4
    scale = sf[at].to(torch.int64) - 127
    return torch.where(c >= 128, -mag, mag) * torch.ldexp(torch.ones(M, K // 32, dtype=torch.float64,
                                                                    device=codes.device), scale).repeat_interleave(32, 1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("route", "route_bwd"):
        z, k, E = st["logits"].double(), case["k"], case["E"]
        live = torch.ones(z.shape[0], dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"].bool()
        p = torch.zeros_like(z)
        p[live] = torch.softmax(z[live], 1)
        if op == "route":
            top = torch.topk(z, k, dim=1).values
            w = torch.softmax(top, 1) if case["renorm"] else torch.exp(top - torch.logsumexp(z, 1, keepdim=True))
            w[~live] = 0
            out = dict(ids=None, weights=w, rows=None, row_index=None, row_offsets=None, sf_row_offsets=None,
                       counts=None)
            if case["loss"]:
                kth = top[:, -1:]
                above, level = z > kth, z == kth
                take = above | (level & (level.cumsum(1) <= k - above.sum(1, keepdim=True)))
                f = (take & live[:, None]).sum(0).double()
                n = max(int(live.sum()), 1)
                out["prob_sums"] = p.sum(0)
                out["loss"] = (COEF * E * (f / (k * n) * (p.sum(0) / n)).sum())[None]
            return out
        ids = st["ids"].long()
        hit = torch.zeros(z.shape[0], E + 1, dtype=torch.float64, device="cuda")
        hit.scatter_(1, torch.where(ids < 0, E, ids), st["dweights"].double())
        hit = hit[:, :E]
        if case["renorm"]:
            q = torch.zeros(z.shape[0], E + 1, dtype=torch.float64, device="cuda")
            q.scatter_(1, torch.where(ids < 0, E, ids), st["weights"].double())
            q = q[:, :E]
        else:
            q = p
        d = q * hit - q * (q * hit).sum(1, keepdim=True)
        if case["loss"]:
            n = max(int(st["counts"][E]), 1)
            f = st["counts"][:E].double() / (k * n)
            d += COEF * E / n * (p * f - p * (p @ f)[:, None])
        return d
    if op in ("combine", "combine_bwd"):
        rows, w = st["rows"].long(), st["weights"].double()
        T, k = rows.shape
        y = _mx_value64(*st["y"]) if case.get("y8") else st["y"]
        if op == "combine":
            out = torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")
            for j in range(k):
                at = (rows[:, j] >= 0).nonzero()[:, 0]
                out[at] += w[at, j, None] * y[rows[at, j]].double()
            return out
        d = st["dout"].double()
        dy = torch.zeros(T * k, case["H"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            at = (rows[:, j] >= 0).nonzero()[:, 0]
            dw[at, j] = torch.einsum("th,th->t", d[at], y[rows[at, j]].double())
            dy[rows[at, j]] = w[at, j, None] * d[at]
        return dict(dy=dy, dweights=dw)
    M, F = case["M"], case["F"]
    n = M if st["n"] is None else int(st["n"])
    if op == "swiglu":
        v = st["u"][:n].double()
        h = torch.zeros(M, F, dtype=torch.float64, device="cuda")
        h[:n] = v[:, :F] / (1 + torch.exp(-v[:, :F])) * v[:, F:]
        # amax is that of h as it is stored
        return dict(h=h, codes=None, scales=None, amax=h.to(torch.bfloat16).double().abs().max()[None])
    v = _mx_value64(st["codes"][:n], st["sf"])
    g, u, d = v[:, :F], v[:, F:], st["dh"][:n].double()
    e = torch.exp(-g)
    du = torch.zeros(M, 2 * F, dtype=torch.float64, device="cuda")
    du[:n, :F] = d * u * (1 + e + g * e) / (1 + e) ** 2
    du[:n, F:] = d * g / (1 + e)
    if not case["h"]:
        return (du,)
    h = torch.zeros(M, F, dtype=torch.float64, device="cuda")
    h[:n] = g / (1 + e) * u
    return (du, h)
