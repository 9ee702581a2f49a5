"""Gradients of cross attention on the GPU, by the norm of their error.

The element bounds of block_testlib add up every rounding in absolute value and
take Delta from the stored O, so they are wide where many keys or queries share
a sum.  These tests hold the whole of a gradient to the size that its roundings
have when they are independent of one another.

bf16: a rounding to bf16 is off by R of the value, root mean square: half a step
(2^-8 of the power of two below the value) uniformly, sqrt(1/3), over mantissas
that are spread evenly by logarithm, sqrt(3/4 / (2 ln 2)).  With P and dS rounded
for the products and the result rounded once,
    |err dV|^2 = R^2 (sum_ij P_ij^2 |dO_i|^2            + |dV|^2)
    |err dK|^2 = R^2 (scale^2 sum_ij dS_ij^2 |q_i|^2    + |dK|^2)
    |err dQ|^2 = R^2 (scale^2 sum_ij (dS_ij^2 + P_ij^2 f_i^2) |k_j - m_i|^2 + |dQ|^2)
as the first pass rounds P (dP - c), and P for its product with f = c - Delta, and
f makes the rounded weights of the keys add up to zero, so that any m_i may be
taken off them: the mean by P, of a row.  c = dO . O carries O's rounding, those
of the sums of up to four products that a lane keeps in bf16 (1 + 2 + 3 + 4 squares
of products for four) and its own: f_i^2 = R^2 (3.5 sum_d (dO_d O_d)^2 + Delta_i^2).
All three are held to 1.5 of the total, as thousands of roundings add up to their
mean square.

fp32: a sum of n products is off by sqrt(n) u of its terms' absolute sum, u =
2^-24 (roundings of independent signs), which carries through the formula
element by element; the norm of that."""

import math

import pytest
import torch

import block_testlib as bt
from test_gpu_cross_attn import make, run

pytestmark = pytest.mark.gpu

R = 2.0**-8 * math.sqrt(0.75 / (2 * math.log(2)) / 3)


def parts(x, kv_len, mask):
    """P, dP, Delta, and what the bounds take of the inputs, in 64 bits, keys of
    shared heads repeated."""
    q, k, v, do = (x[n].double() for n in ("q", "k", "v", "do"))
    B, H, N, D = q.shape
    G = H // k.shape[1]
    ok = bt.seen(B, k.shape[2], kv_len, mask, q.device)[:, None, :, None]
    k, v = (torch.where(ok, t, 0.0).repeat_interleave(G, 1) for t in (k, v))
    s = (q @ k.mT / math.sqrt(D)).masked_fill(~ok.mT, -math.inf)
    lse = s.logsumexp(-1, keepdim=True)
    p = (s - lse.masked_fill(lse == -math.inf, 0.0)).exp()
    dp = do @ v.mT
    delta = (p * dp).sum(-1, keepdim=True)
    return q, k, v, do, s.masked_fill(s == -math.inf, 0.0), p, dp, delta, G


def expected(x, want, kv_len, mask):
    """Norms of the errors of dq, dk and dv."""
    q, k, v, do, s, p, dp, delta, G = parts(x, kv_len, mask)
    D, S = q.shape[-1], k.shape[-2]
    scale = 1.0 / math.sqrt(D)
    ds = p * (dp - delta)
    if x["q"].dtype == torch.bfloat16:
        sq = (lambda t: (t * t).sum(-1))
        f2 = R**2 * (3.5 * sq(do * (p @ v)) + sq(delta))[..., None]
        w, m = ds * ds + p * p * f2, p @ k  # sum_j w |k - m|^2, written out
        spread = w @ sq(k)[..., None] - 2 * (m * (w @ k)).sum(-1, keepdim=True) + w.sum(-1, keepdim=True) * sq(m)[..., None]
        sums = {"dq": scale**2 * spread.clamp_min(0.0).sum(),
                "dk": scale**2 * ((ds * ds).mT @ sq(q)[..., None]).sum(),
                "dv": ((p * p).mT @ sq(do)[..., None]).sum()}
        return {n: 1.5 * R * float(t + sq(want[n][0]).sum()) ** 0.5 for n, t in sums.items()}
    u, rows = bt.U, q.shape[2] * G
    e_s = u * (math.sqrt(D) * scale * (q.abs() @ k.abs().mT) + 4 * s.abs() + 4)
    rel = e_s + (p * e_s).sum(-1, keepdim=True) + u * (math.sqrt(S) + 4)  # of P: its score, lse
    e_dp = u * math.sqrt(D) * (do.abs() @ v.abs().mT)
    o = p @ v
    e_o = (p * (rel + u * math.sqrt(S))) @ v.abs() + u * o.abs()
    e_delta = (do.abs() * e_o).sum(-1, keepdim=True) + u * math.sqrt(D) * (do * o).abs().sum(-1, keepdim=True)
    e_ds = rel * ds.abs() + p * (e_dp + e_delta + 2 * u * (dp.abs() + delta.abs()))
    group = (lambda t: t.unflatten(1, (-1, G)).sum(2))
    out = {"dq": scale * ((e_ds + u * math.sqrt(S) * ds.abs()) @ k.abs()),
           "dk": scale * group((e_ds + u * math.sqrt(rows) * ds.abs()).mT @ q.abs()),
           "dv": group((p * (rel + u * math.sqrt(rows))).mT @ do.abs())}
    return {n: float((t + u * want[n][0].abs()).norm()) for n, t in out.items()}


def hold(x, kv_len=None, mask=None):
    out = run(x, kv_len, mask)
    want = bt.cross(x["q"], x["k"], x["v"], kv_len, mask, do=x["do"], bf16=x["q"].dtype == torch.bfloat16)
    most = expected(x, want, kv_len, mask)
    far = {n: float((out[n].double() - want[n][0]).norm()) / most[n] for n in most}
    assert max(far.values()) <= 1, far


SHAPES = [
    # B, H, Hkv, N, S, D
    (2, 4, 2, 127, 128, 128),
    (1, 2, 1, 300, 333, 128),
    (2, 2, 2, 200, 256, 64),
    (3, 8, 2, 97, 512, 64),
    (1, 16, 4, 17, 2500, 128),
    (1, 2, 2, 2500, 80, 64),
    (1, 2, 2, 1111, 700, 128),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norms(shape, dtype):
    hold(make(*shape, dtype, seed=51))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norms_masked(shape, dtype):
    B, _, _, _, S, _ = shape
    g = torch.Generator(device="cuda").manual_seed(52)
    lens = torch.tensor([S, S - S // 3, S // 2][:B], dtype=torch.int32, device="cuda")
    hold(make(*shape, dtype, seed=53), lens, (torch.rand(B, S, generator=g, device="cuda") < 0.8).to(torch.uint8))


@pytest.mark.parametrize("front", [0, 7, 16, 40, 64, 130])
@pytest.mark.parametrize("shape", [(2, 4, 2, 300, 333, 64), (1, 2, 2, 200, 300, 128), (1, 4, 1, 9, 3000, 64),
                                   (2, 8, 8, 1300, 200, 64), (2, 6, 6, 1700, 300, 128)], ids=str)
def test_common_part_behind_hidden_keys(shape, front):
    """Keys and values with a large common part, the front of the sequence
    hidden (a caption padded on the left): what the values share must leave dQ
    wherever the first key that is seen lies, with the keys in one piece (the
    last two shapes) and split."""
    B, _, _, _, S, _ = shape
    x = make(*shape, "bf16", seed=54, gain=0.3)
    for n in "kv":
        x[n] = (x[n].float() + 16.0).to(torch.bfloat16)
    mask = torch.ones(B, S, dtype=torch.uint8, device="cuda")
    mask[:, :front] = 0
    if B > 1:
        mask[1, S // 2 :] = 0  # and unlike fronts
        mask[1, : front // 2 + 3] = 0
    hold(x, None, mask)


@pytest.mark.parametrize("gain", [4.0, 16.0])
@pytest.mark.parametrize("shape", [(2, 4, 4, 1000, 333, 64), (1, 4, 2, 1000, 300, 128), (1, 4, 1, 30, 3000, 64)], ids=str)
def test_rows_that_sit_on_few_keys(shape, gain):
    """Sharp rows, whose gradient is what little the probabilities share."""
    hold(make(*shape, "bf16", seed=55, gain=gain))


@pytest.mark.parametrize("shape", [(2, 4, 4, 1000, 60, 64), (1, 4, 2, 1000, 200, 128)], ids=str)
def test_few_keys_of_many(shape):
    """Three keys in unlike tiles are all that is seen."""
    B, _, _, _, S, _ = shape
    mask = torch.zeros(B, S, dtype=torch.uint8, device="cuda")
    mask[:, [S // 9, S // 2, S - 2]] = 1
    hold(make(*shape, "bf16", seed=56), None, mask)
