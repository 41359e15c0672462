"""The packed-sequence operators from their definitions, in 64 bits (torch
float64 on the tensors' device), and the error bounds of the kernels' tests.

Bounds count roundings: half a step of a type is finfo(t).eps / 2 of the value.
"""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def norm_rope(x, w, positions, axis_dim, theta, eps):
    """x [T][h][d] -> (z, the norm of each element's pair), both float64."""
    y = x.double()
    if w is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    freq = [theta ** (-2.0 * i / a) for a in axis_dim for i in range(a // 2)]
    axis = [n for n, a in enumerate(axis_dim) for _ in range(a // 2)]
    angle = positions.double()[:, axis] * torch.tensor(freq, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    z = torch.view_as_complex(y.unflatten(-1, (-1, 2)).contiguous()) * turn
    mag = z.abs()
    return torch.view_as_real(z).flatten(-2), torch.stack((mag, mag), -1).flatten(-2)


def norm_rope_grads(x, w, positions, axis_dim, theta, eps, gz):
    """(dx, dw, bound parts): the gradients, and sums of magnitudes for their error bounds."""
    x = x.double().requires_grad_(True)
    wd = w.double().requires_grad_(True) if w is not None else None
    z, _ = norm_rope(x, wd, positions, axis_dim, theta, eps)
    got = torch.autograd.grad(z, (x, wd) if w is not None else (x,), gz.double())
    # |g| through the rotation: the norm of each pair
    gp = torch.view_as_complex(gz.double().unflatten(-1, (-1, 2)).contiguous()).abs()
    gp = torch.stack((gp, gp), -1).flatten(-2)
    xd = x.detach()
    if w is None:
        return got[0], None, gp, None
    r = 1.0 / (xd.square().mean(-1, keepdim=True) + eps).sqrt()
    g, xh = gp * w.double().abs(), (xd * r).abs()
    return got[0], got[1], r * (g + xh * (g * xh).mean(-1, keepdim=True)), (gp * xh).sum((0, 1))


def limits(Lq, Lk, block, device):
    i = torch.arange(Lq, device=device)
    if block == 0:
        return torch.full((Lq,), Lk, device=device)
    return (((i + Lk - Lq).div(block, rounding_mode="floor") + 1) * block).clamp(0, Lk)


def sequences(q_lens, k_lens, q_first=0, k_first=0):
    cq, ck = q_first, k_first
    for a, b in zip(q_lens, k_lens):
        yield slice(cq, cq + a), slice(ck, ck + b)
        cq, ck = cq + a, ck + b


def attention(q, k, v, q_lens, k_lens, block, q_first=0, k_first=0):
    """out [Tq][H][d], lse [H][Tq] and their error bounds; rows outside the sequences are 0."""
    H, Hkv, d = q.shape[1], k.shape[1], q.shape[2]
    z = lambda *s: torch.zeros(s, dtype=torch.float64, device=q.device)  # noqa: E731
    out, lse, b_out, b_lse = z(*q.shape), z(H, q.shape[0]), z(*q.shape), z(H, q.shape[0])
    for rq, rk in sequences(q_lens, k_lens, q_first, k_first):
        Lq, Lk = rq.stop - rq.start, rk.stop - rk.start
        hide = torch.arange(Lk, device=q.device)[None] >= limits(Lq, Lk, block, q.device)[:, None]
        for h in range(H):
            qd, kd, vd = q[rq, h].double(), k[rk, h // (H // Hkv)].double(), v[rk, h // (H // Hkv)].double()
            if Lk == 0:
                lse[h, rq] = -float("inf")
                continue
            s = (qd @ kd.T / d ** 0.5).masked_fill(hide, -float("inf"))
            a = torch.where(hide, torch.zeros_like(s), qd.abs() @ kd.abs().T / d ** 0.5).amax(-1)
            lse[h, rq] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[h, rq][:, None]).masked_fill(hide, 0.0)
            out[rq, h] = p @ vd
            # P rounded to bf16 (half a step of each term); the logits' fp32 sums of 128 products (16 * 2^-23 of
            # the sum of magnitudes is generous) and 2^x (2^-22) move P by 2^-13 more at |s| <= 100; out rounded once
            b_out[rq, h] = HALF[torch.bfloat16] * out[rq, h].abs() + (2.0 ** -8 + 2.0 ** -13) * (p @ vd.abs())
            b_lse[h, rq] = 2.0 ** -19 * (a + 1) + 2.0 ** -20 * lse[h, rq].abs().nan_to_num(posinf=0.0)
    return out, lse, b_out, b_lse


def attention_grads(q, k, v, out, lse, dout, q_lens, k_lens, block, q_first=0, k_first=0):
    """(dq, dk, dv) and their error bounds, from the forward pass's out and lse."""
    H, Hkv, d = q.shape[1], k.shape[1], q.shape[2]
    G, sc = H // Hkv, d ** -0.5
    z = lambda t: torch.zeros(t.shape, dtype=torch.float64, device=q.device)  # noqa: E731
    dq, dk, dv, bq, bk, bv = z(q), z(k), z(k), z(q), z(k), z(k)
    u = HALF[torch.float16] if q.dtype == torch.float16 else HALF[torch.bfloat16]
    tops = [1e-300, 1e-300]  # largest row norms of dout and v: fp16's smallest step is 2^-38 of twice their product
    for rq, rk in sequences(q_lens, k_lens, q_first, k_first):
        if rq.stop > rq.start and rk.stop > rk.start:
            tops[0] = max(tops[0], float(dout[rq].double().norm(dim=-1).max()))
            tops[1] = max(tops[1], float(v[rk].double().norm(dim=-1).max()))
    tiny = 2.0 ** -38 * 2 * tops[0] * tops[1] if q.dtype == torch.float16 else 0.0
    for rq, rk in sequences(q_lens, k_lens, q_first, k_first):
        Lq, Lk = rq.stop - rq.start, rk.stop - rk.start
        if not Lq or not Lk:
            continue
        hide = torch.arange(Lk, device=q.device)[None] >= limits(Lq, Lk, block, q.device)[:, None]
        for h in range(H):
            j = h // G
            qd, kd, vd = q[rq, h].double(), k[rk, j].double(), v[rk, j].double()
            od, gd = out[rq, h].double(), dout[rq, h].double()
            l = lse[h, rq].double()[:, None]
            p = torch.exp(qd @ kd.T * sc - l.clamp(min=-1e300)).masked_fill(hide, 0.0)
            ds = p * (gd @ vd.T - (gd * od).sum(-1, keepdim=True))
            dv[rk, j] += p.T @ gd
            dk[rk, j] += ds.T @ qd * sc
            dq[rq, h] = ds @ kd * sc
            # dS rounded (u of each term, `tiny` at least), P off by 2^-13 as in the forward pass, dP and D summed in
            # fp32 over 128 products (2^-19 of the magnitudes)
            e = (u + 2.0 ** -13) * ds.abs() + p * 2.0 ** -19 * (gd.abs() @ vd.abs().T + (gd * od).abs().sum(-1, keepdim=True))
            e = e + tiny * (~hide)
            bq[rq, h] = e @ kd.abs() * sc
            bk[rk, j] += e.T @ qd.abs() * sc
            bv[rk, j] += (2.0 ** -8 + 2.0 ** -13) * (p.T @ gd.abs())
    half = HALF[torch.bfloat16]  # the rounding of the result itself; 1 + 2^-7 of the bound for what it rounds
    return (dq, dk, dv), tuple(b * (1 + 2.0 ** -7) + half * r.abs() for b, r in ((bq, dq), (bk, dk), (bv, dv)))


def assert_within(got, ref, bound, what=""):
    got = got.double()
    same = (got == ref) | (got.isnan() & ref.isnan())
    err = torch.where(same, torch.zeros_like(ref), (got - ref).abs())
    worst = (err / bound.clamp(min=1e-300)).max() if err.numel() else torch.zeros(())
    assert bool((err <= bound).all()), f"{what}: {float(worst):.3g} of the bound (largest error {float(err.max()):.3g})"
