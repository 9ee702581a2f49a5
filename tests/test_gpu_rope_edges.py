"""The rotary table on the GPU where its frequencies and angles are hardest."""

import math
from decimal import Decimal, getcontext

import pytest
import torch

import block_testlib as bt
import hierarchical_top_sparse_llsa_b200 as llsa

pytestmark = pytest.mark.gpu


def table(rope, rows, half, pos=None):
    t = torch.full((rows, half, 2), float("nan"), device="cuda")
    llsa.llsa_rope_table(rope, rows, None if pos is None else pos.data_ptr(), t.data_ptr(),
                         torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return t.cpu().double()


def yarn(dim, base, factor, orig_len, fast=32.0, slow=1.0):
    """YaRN's frequencies of an axis of `dim` rotated channels, as its authors
    compute them: the ends of the ramp by channels, the upper one within dim - 1."""
    def at(turns):
        return dim * math.log(orig_len / (turns * 2 * math.pi)) / (2 * math.log(base))
    low, high = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), dim - 1)
    out = []
    for i in range(dim // 2):
        f = base ** (-2 * i / dim)
        keep = 1 - min(max((i - low) / max(high - low, 0.001), 0), 1)
        out.append(f / factor * (1 - keep) + f * keep)
    return out


@pytest.mark.parametrize("rot,axes,base,factor,orig_len", [
    (128, 1, 10000.0, 4.0, 131072),   # the ramp ends past the last pair
    (128, 1, 10000.0, 4.0, 8192),     # and before it
    (16, 2, 10000.0, 4.0, 8192),      # four pairs an axis
    (64, 1, 1000.0, 16.0, 1 << 24),   # every pair keeps its frequency
    (2, 1, 10000.0, 2.0, 4096),
])
def test_yarn_frequencies(rot, axes, base, factor, orig_len):
    rope = llsa.make_rope(rot, axes=axes, base=base, scaling=llsa.ROPE_SCALE_YARN, factor=factor, orig_len=orig_len)
    pos = torch.tensor([0, 1, 2, 3, 1000, 100003], dtype=torch.int32)
    f = torch.tensor(yarn(rot // axes, base, factor, orig_len) * axes, dtype=torch.float64)
    got = table(rope, len(pos), rot // 2, pos[:, None].repeat(1, axes).contiguous().cuda())
    ang = pos.double()[:, None] * f
    m = 0.1 * math.log(factor) + 1
    want = torch.stack([ang.cos(), ang.sin()], -1) * m
    # 2^-22 m of the table, and these angles in 64 bits: 4 roundings of up to 1e5
    assert float((got - want).abs().max()) <= m * (2.0**-22 + 4 * 2.0**-53 * 100003)


PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494")


@pytest.mark.parametrize("rot,base,kw", [
    (128, 10000.0, {}),
    (64, 500000.0, {}),
    (64, 10500.0, dict(scaling=llsa.ROPE_SCALE_LINEAR, factor=3.0)),
    (64, 10000.0, dict(scaling=llsa.ROPE_SCALE_NTK, factor=8.0)),
    (2, 10000.0, dict(mscale=1.75)),
])
def test_table_as_far_as_positions_go(rot, base, kw):
    """Each entry is within 2^-22 m of the exact value at any int32 position,
    against angles of 50 digits."""
    getcontext().prec = 50
    n, factor = rot // 2, Decimal(kw.get("factor", 1.0))
    b = Decimal(base)
    if kw.get("scaling") == llsa.ROPE_SCALE_NTK:
        b *= factor ** (Decimal(n) / (n - 1))
    f = [b ** (-Decimal(j) / n) for j in range(n)]
    if kw.get("scaling") == llsa.ROPE_SCALE_LINEAR:
        f = [w / factor for w in f]
    pos = torch.randint(2**31 - 4096, 2**31, (40,), generator=torch.Generator().manual_seed(3), dtype=torch.int64)
    pos = torch.cat([pos, -pos, torch.tensor([-(2**31), 2**31 - 1, 0, 1 << 24, 1 << 28, 123456789])])
    got = table(llsa.make_rope(rot, base=base, **kw), len(pos), n, pos.to(torch.int32).cuda())
    want = torch.empty(len(pos), n, 2, dtype=torch.float64)
    for i, p in enumerate(pos.tolist()):
        for j, w in enumerate(f):
            ang = float((p * w) % (2 * PI))  # rounded to 64 bits once reduced
            want[i, j, 0], want[i, j, 1] = math.cos(ang), math.sin(ang)
    m = kw.get("mscale", 1.0)
    assert float((got - want * m).abs().max()) <= m * 2.0**-22


@pytest.mark.parametrize("k", [True, False])
def test_more_heads_than_a_grid_has_rows(k):
    """100000 heads of one token: a thread walks many of them."""
    H, D = 100000, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    x = [torch.randn(1, H, 1, D, generator=g, device="cuda").bfloat16() for _ in range(2)]
    rope = llsa.make_rope(D)
    tab = torch.empty(1, D // 2, 2, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    pos = torch.tensor([[1234]], dtype=torch.int32, device="cuda")
    llsa.llsa_rope_table(rope, 1, pos.data_ptr(), tab.data_ptr(), s)
    out = [torch.full_like(t, float("nan")) for t in x]
    llsa.llsa_rope(rope, 1, H, 1, D, llsa.BF16, tab.data_ptr(), 1, x[0].data_ptr(), x[1].data_ptr() if k else None,
                   out[0].data_ptr(), out[1].data_ptr() if k else None, False, s)
    torch.cuda.synchronize()
    for t, y in zip(x[: 1 + k], out):
        want, mag = bt.rotate(t.double(), tab.double(), D, False)
        bt.within(y, want, bt.rotate_bound(want, mag, True), "rotation")
