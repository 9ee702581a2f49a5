"""Plain 64-bit forms of rotary positions and cross attention, with error
bounds of the kernels derived from their arithmetic, shared by the tests.

u = 2^-24 is half a step of fp32, ub = 2^-8 half a step of bf16.  Every bound
is a sum over the terms of the formula, so it holds element by element:

  scores     an fp32 sum of D products is off by at most D 2^-22 sum |q_d k_d|
             (a rounding per product and per addition, doubled because a
             tensor core aligns the terms of a partial sum before it adds
             them and drops bits below the largest), times the scale; the
             probability then is off by that in relative terms (e^x ~ 1 + x),
             plus 2^-20 for the exponential itself.
  bf16       P and dS are rounded to bf16 for the products that they enter;
             outputs are rounded once more.
  Delta      dO . O with O rounded to the stored type: ub sum |dO_d O_d|
             (2^-16 of it with the residual, which is bf16 itself).
"""

import math

import torch

U, UB = 2.0**-24, 2.0**-8


# ------------------------------------------------------- rotary positions
def zorder_xy(rows):
    out = []
    for t in range(rows):
        x = y = 0
        for b in range(16):
            x |= ((t >> (2 * b)) & 1) << b
            y |= ((t >> (2 * b + 1)) & 1) << b
        out.append((x, y))
    return torch.tensor(out, dtype=torch.float64)


def inv_freq(n, base=10000.0, scaling=0, factor=1.0, orig_len=0, fast=32.0, slow=1.0):
    if scaling == 2 and n > 1:
        base = base * factor ** (n / (n - 1))
    f = [base ** (-j / n) for j in range(n)]
    if scaling == 1:
        f = [x / factor for x in f]
    if scaling == 3:
        def at(turns):
            return n * math.log(orig_len / (turns * 2 * math.pi)) / math.log(base)
        lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), n - 1)
        r = [min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0) for j in range(n)]
        f = [x / factor * t + x * (1 - t) for x, t in zip(f, r)]
    return torch.tensor(f, dtype=torch.float64)


def rope_table(pos, rot, axes=1, m=1.0, **scaling):
    """[rows, rot / 2, 2] in 64 bits; pos: [rows, axes] float64 on the CPU."""
    f = inv_freq(rot // 2 // axes, **scaling)
    ang = (pos[:, :, None] * f).reshape(pos.shape[0], rot // 2)
    return torch.stack([ang.cos() * m, ang.sin() * m], -1)


def rotate(x, table, rot, interleaved, adjoint=False):
    """x [B, H, N, D] and table [N or B N, rot / 2, 2] in 64 bits; also the sum
    of the absolute products of each output element."""
    B, _, N, _ = x.shape
    t = table.reshape(-1, N, rot // 2, 2)[:, None]
    c, s = t[..., 0], t[..., 1]
    if adjoint:
        s = -s
    y, mag = x.clone(), torch.zeros_like(x)
    i0 = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    i1 = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    mag[..., i0], mag[..., i1] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return y, mag


def rotate_bound(y, mag, bf16):
    """Two roundings on the way of each product to the sum (its own and the
    sum's), then the stored type's: channels that pass through have mag 0."""
    fp32 = 2 * U * mag * (1 + 2 * U)
    return fp32 + ((y.abs() + fp32) * UB if bf16 else 0.0) * (mag > 0)


# --------------------------------------------------------- cross attention
def seen(B, S, kv_len, mask, device):
    ok = torch.ones(B, S, dtype=torch.bool, device=device)
    if kv_len is not None:
        ok &= torch.arange(S, device=device) < kv_len.long().clamp(0, S)[:, None]
    if mask is not None:
        ok &= mask != 0
    return ok


def cross(q, k, v, kv_len=None, mask=None, scale=None, do=None, bf16=True, residual=False):
    """Cross attention and its gradients in 64 bits, with bounds.  Returns a
    dict name -> (value, bound)."""
    B, H, N, D = q.shape
    Hkv, S = k.shape[1:3]
    G = H // Hkv
    ok = seen(B, S, kv_len, mask, q.device)
    scale = scale or 1.0 / math.sqrt(D)
    q = q.double()
    # what is not seen does not count, whatever it holds
    k, v = (torch.where(ok[:, None, :, None], t.double(), 0.0).repeat_interleave(G, 1) for t in (k, v))
    x = (q @ k.mT * scale).masked_fill(~ok[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True) if S else torch.full_like(q[..., :1], -math.inf)
    m0 = m.masked_fill(m == -math.inf, 0.0)
    e = (x - m0).exp()
    l = e.sum(-1, keepdim=True)
    p = e / l.masked_fill(l == 0, 1.0)
    o = p @ v
    lse = (m + l.log()).squeeze(-1)
    # a score's error, and with it a probability's relative one (its own, and
    # the sum's that it is divided by)
    ds_abs = scale * D * 2.0**-22 * (q.abs() @ k.abs().mT)
    worst = (ds_abs * (p > 0)).amax(-1, keepdim=True) if S else torch.zeros_like(l)
    rel = 2 * worst + 2.0**-19 + S * 2.0**-22
    half = UB if bf16 else U
    store = (lambda t, err: (t.abs() + err) * half + err)
    out = {}
    out["o"] = (o, store(o, (rel + (UB if bf16 else 0.0)) * (p @ v.abs())) + 1e-30)
    out["lse"] = (lse, worst.squeeze(-1) + 2.0**-19 + S * 2.0**-22 + lse.abs().nan_to_num(posinf=0.0) * 4 * U)
    if do is None:
        return out
    do = do.double()
    dp = do @ v.mT
    delta = (do * o).sum(-1, keepdim=True)
    d = p * (dp - delta)
    # the gradient's terms: how far P, dP and Delta each move a dS
    dp_err = D * 2.0**-22 * (do.abs() @ v.abs().mT)
    o_err = out["o"][1] if not residual else (rel + (UB if bf16 else 0.0)) * (p @ v.abs()) + 2 * UB * UB * o.abs()
    delta_err = (do.abs() * o_err).sum(-1, keepdim=True) + D * 2.0**-22 * (do * o).abs().sum(-1, keepdim=True)
    d_err = p * (dp_err + delta_err) + d.abs() * (rel + (UB if bf16 else 0.0)) + p * rel * (dp.abs() + delta.abs())
    group = (lambda t: t.unflatten(1, (Hkv, G)).sum(2))
    acc = N * G * 2.0**-22  # a running fp32 sum over all queries
    dq = d @ k * scale
    dq_err = scale * ((d_err + d.abs() * S * 2.0**-22) @ k.abs())
    dk = group(d.mT @ q) * scale
    dk_err = scale * group((d_err + d.abs() * acc).mT @ q.abs())
    dv = group(p.mT @ do)
    dv_err = group((p * (rel + (UB if bf16 else 0.0) + acc)).mT @ do.abs())
    for name, t, err in (("dq", dq, dq_err), ("dk", dk, dk_err), ("dv", dv, dv_err)):
        out[name] = (t, store(t, err) + 1e-30)
    return out


def within(got, want, bound, what):
    got = got.double()
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf].to(got.dtype)), f"{what}: infinities differ"
    err = (got - want)[~inf].abs()
    bad = ~(err <= bound.expand_as(want)[~inf])
    if bad.any():
        worst = (err / bound.expand_as(want)[~inf]).nan_to_num(nan=math.inf).max()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst {float(worst):.3g}x")
