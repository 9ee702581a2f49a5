"""Rotary positions on the GPU against 64-bit forms: the table, the rotation
and its adjoint, and the rotation with the pyramid (equal to llsa_rope and
llsa_pool bit for bit)."""

import pytest
import torch

import block_testlib as bt
import hierarchical_top_sparse_llsa_b200 as llsa

pytestmark = pytest.mark.gpu

DT = {"f32": (torch.float32, llsa.F32), "bf16": (torch.bfloat16, llsa.BF16)}


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _table(rope, rows, pos=None, half=None):
    t = torch.full((rows, half, 2), float("nan"), device="cuda")
    llsa.llsa_rope_table(rope, rows, None if pos is None else pos.data_ptr(), t.data_ptr(), _stream())
    torch.cuda.synchronize()
    return t


TABLES = [
    dict(rot=64, rows=777),
    dict(rot=64, rows=1),
    dict(rot=2, rows=5000),
    dict(rot=6, rows=333),  # an odd number of pairs
    dict(rot=64, rows=1024, axes=2),  # Z-order pixels
    dict(rot=44, rows=4099, axes=2),  # 11 pairs an axis, not a whole square
    dict(rot=128, rows=300, span=2**31 - 1),  # as far as an int32 goes
    dict(rot=128, rows=300, span=1 << 20, scaling=1, factor=4.0),
    dict(rot=64, rows=300, span=1 << 20, scaling=2, factor=8.0),
    dict(rot=2, rows=30, span=1 << 20, scaling=2, factor=8.0),  # one pair: the base is not stretched
    dict(rot=128, rows=300, span=1 << 17, scaling=3, factor=4.0, orig_len=8192),
    dict(rot=96, rows=300, span=1 << 17, axes=2, scaling=3, factor=2.5, orig_len=1024, base=500000.0),
]


@pytest.mark.parametrize("c", TABLES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_table(c):
    c = dict(c)
    rot, rows, axes, span = c.pop("rot"), c.pop("rows"), c.pop("axes", 1), c.pop("span", 0)
    rope = llsa.make_rope(rot, axes=axes, **c)
    pos = None
    if span:
        g = torch.Generator().manual_seed(1)
        pos = torch.randint(-span, span, (rows, axes), generator=g, dtype=torch.int64).clamp(-(2**31), 2**31 - 1)
        pos[0] = -(2**31) if span > 2**30 else span
        pos = pos.to(torch.int32).cuda()
    got = _table(rope, rows, pos, rot // 2)
    if pos is not None:
        p = pos.cpu().double()
    else:
        p = torch.arange(rows, dtype=torch.float64)[:, None] if axes == 1 else bt.zorder_xy(rows)
    m = 0.1 * torch.log(torch.tensor(c["factor"])).item() + 1 if c.get("scaling") == 3 else 1.0
    want = bt.rope_table(p, rot, axes, m, **c)
    # 2^-22 m as the header states; both sides' fp64 angles are off by 2^-52
    # of themselves
    bound = (2.0**-22 * m + 2.0**-51 * p.abs().max() * m) * torch.ones_like(want)
    bt.within(got.cpu(), want, bound, "table")


def test_table_mscale():
    rope = llsa.make_rope(64, mscale=1.75)
    want = bt.rope_table(torch.arange(50, dtype=torch.float64)[:, None], 64, 1, 1.75)
    bt.within(_table(rope, 50, None, 32).cpu(), want, torch.full_like(want, 2.0**-22 * 1.75), "table")


ROTATIONS = [
    # B, H, N, D, rot, interleaved, per_batch
    (1, 1, 1, 64, 64, False, False),
    (1, 16, 1, 128, 128, True, False),  # one token, the heads shared out
    (2, 3, 77, 64, 64, False, True),
    (3, 5, 129, 128, 64, False, False),
    (2, 2, 33, 64, 16, False, False),
    (1, 4, 100, 128, 24, False, True),  # partners off the 16-byte chunks (bf16)
    (1, 4, 100, 64, 6, False, False),   # an odd number of pairs
    (2, 3, 65, 64, 2, False, False),
    (2, 3, 65, 64, 6, True, True),
    (1, 2, 51, 128, 40, True, False),
    (1, 2, 2100, 64, 62, False, False),
    (2, 12, 4096, 64, 64, False, False),
]


def _inputs(B, H, N, D, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(B, H, N, D, generator=g, device="cuda").to(dt) for _ in range(3)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", ROTATIONS, ids=str)
def test_rotation(c, dtype):
    B, H, N, D, rot, inter, per_batch = c
    dt, code = DT[dtype]
    q, k, _ = _inputs(B, H, N, D, dt, 3)
    rows = B * N if per_batch else N
    rope = llsa.make_rope(rot, layout=llsa.ROPE_INTERLEAVED if inter else llsa.ROPE_HALF)
    tab = _table(rope, rows, None, rot // 2)
    for adjoint in (False, True):
        out = [torch.full_like(q, float("nan")) for _ in range(2)]
        llsa.llsa_rope(rope, B, H, N, D, code, tab.data_ptr(), rows, q.data_ptr(), k.data_ptr(), out[0].data_ptr(),
                       out[1].data_ptr(), adjoint, _stream())
        torch.cuda.synchronize()
        for x, y, what in ((q, out[0], "q"), (k, out[1], "k")):
            want, mag = bt.rotate(x.double(), tab.double(), rot, inter, adjoint)
            bt.within(y, want, bt.rotate_bound(want, mag, dtype == "bf16"), f"{what} adjoint={adjoint}")
            assert torch.equal(y[..., rot:], x[..., rot:])  # passes through
        # one tensor alone, and both in place: the same bits
        one = torch.full_like(q, float("nan"))
        llsa.llsa_rope(rope, B, H, N, D, code, tab.data_ptr(), rows, k.data_ptr(), None, one.data_ptr(), None, adjoint,
                       _stream())
        q2, k2 = q.clone(), k.clone()
        llsa.llsa_rope(rope, B, H, N, D, code, tab.data_ptr(), rows, q2.data_ptr(), k2.data_ptr(), q2.data_ptr(),
                       k2.data_ptr(), adjoint, _stream())
        torch.cuda.synchronize()
        assert torch.equal(one, out[1]) and torch.equal(q2, out[0]) and torch.equal(k2, out[1])


def test_special_values_stay_in_their_pairs():
    # an infinity or NaN reaches its own pair only, and channels past rot_dim
    # keep their bits, signed zeros and NaN payloads included
    q, _, _ = _inputs(1, 1, 8, 64, torch.bfloat16, 5)
    q[0, 0, 3, 5] = float("inf")
    q[0, 0, 4, 40] = float("nan")
    q[0, 0, 5, 60] = -0.0
    q.view(torch.int16)[0, 0, 6, 61] = 0x7FA1
    for inter in (False, True):
        rope = llsa.make_rope(32, layout=int(inter))
        tab = _table(rope, 8, None, 16)
        out = torch.empty_like(q)
        llsa.llsa_rope(rope, 1, 1, 8, 64, llsa.BF16, tab.data_ptr(), 8, q.data_ptr(), None, out.data_ptr(), None,
                       False, _stream())
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16)[..., 32:], q.view(torch.int16)[..., 32:])
        bad = ~torch.isfinite(out[0, 0, :, :32].float())
        pair = [4, 5] if inter else [5, 21]
        assert sorted(bad[3].nonzero().flatten().tolist()) == pair and int(bad.sum()) == 2


POOLS = [
    # B, H, N, D, L, rot, interleaved, per_batch
    (1, 2, 1024, 64, 2, 64, False, False),
    (2, 3, 48, 64, 1, 64, False, True),
    (1, 1, 16, 128, 1, 128, True, False),
    (2, 2, 4096, 128, 3, 64, False, False),
    (1, 3, 512, 64, 2, 6, True, True),
    (1, 3, 512, 64, 2, 24, False, False),  # bf16: two calls inside
    (1, 16, 65536, 64, 3, 64, False, False),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", POOLS, ids=str)
def test_rope_pool_is_rope_then_pool(c, dtype):
    B, H, N, D, L, rot, inter, per_batch = c
    dt, code = DT[dtype]
    q, k, v = _inputs(B, H, N, D, dt, 4)
    rows = B * N if per_batch else N
    rope = llsa.make_rope(rot, layout=int(inter), axes=2 if rot % 4 == 0 else 1)
    tab = _table(rope, rows, None, rot // 2)
    desc = llsa.make_desc(B, H, N, D, L, 4, code)
    ref, buf = (llsa.LlsaBuffers(desc, "cuda", with_bwd=False) for _ in range(2))
    rq, rk = torch.empty_like(q), torch.empty_like(k)
    llsa.llsa_rope(rope, B, H, N, D, code, tab.data_ptr(), rows, q.data_ptr(), k.data_ptr(), rq.data_ptr(),
                   rk.data_ptr(), False, _stream())
    llsa.llsa_pool(desc, rq.data_ptr(), rk.data_ptr(), v.data_ptr(), ref.pyramid, _stream())
    for in_place in (False, True):
        a, b = (q.clone(), k.clone())
        oq, ok = (a, b) if in_place else (torch.full_like(q, float("nan")), torch.full_like(k, float("nan")))
        for lv in (buf.pq, buf.pk, buf.pv):
            for t in lv.values():
                t.fill_(float("nan"))
        llsa.llsa_rope_pool(desc, rope, tab.data_ptr(), rows, a.data_ptr(), b.data_ptr(), v.data_ptr(), oq.data_ptr(),
                            ok.data_ptr(), buf.pyramid, _stream())
        torch.cuda.synchronize()
        assert torch.equal(oq, rq) and torch.equal(ok, rk)
        for got, want in ((buf.pq, ref.pq), (buf.pk, ref.pk), (buf.pv, ref.pv)):
            for l in want:
                assert torch.equal(got[l], want[l]), f"level {l}"


def test_adjoint_is_the_gradient():
    # <dy, R x> = <R^T dy, x>, and a central difference of <dy, R x>: R is
    # linear, so a step h along z moves it by h <dy, R z>
    B, H, N, D, rot = 1, 2, 40, 64, 48
    x, dy, z = _inputs(B, H, N, D, torch.float32, 6)
    rope = llsa.make_rope(rot, axes=2)
    tab = _table(rope, N, None, rot // 2)

    def apply(t, adjoint):
        out = torch.empty_like(t)
        llsa.llsa_rope(rope, B, H, N, D, llsa.F32, tab.data_ptr(), N, t.data_ptr(), None, out.data_ptr(), None,
                       adjoint, _stream())
        torch.cuda.synchronize()
        return out.double()

    back = apply(dy, True)
    h = 2.0**-6
    up, down = apply(x + h * z, False), apply(x - h * z, False)
    diff = float(((up - down) * dy.double()).sum() / (2 * h))
    want = float((back * z.double()).sum())
    # each rotation is off by at most 2 u of its products and its argument was
    # rounded once; the difference divides that by h
    mag = float((3.0 * (x.abs() + z.abs()).double() * 2).sum(-1).max()) * N * H * float(dy.abs().max())
    assert abs(diff - want) <= 8 * bt.U * mag / h


def test_rope_in_a_graph_and_on_another_stream():
    B, H, N, D = 1, 4, 256, 64
    q, k, v = _inputs(B, H, N, D, torch.bfloat16, 7)
    rope = llsa.make_rope(64)
    tab = _table(rope, N, None, 32)
    desc = llsa.make_desc(B, H, N, D, 2, 4, llsa.BF16)
    buf = llsa.LlsaBuffers(desc, "cuda", with_bwd=False)
    oq, ok = torch.empty_like(q), torch.empty_like(k)

    def call():
        llsa.llsa_rope_pool(desc, rope, tab.data_ptr(), N, q.data_ptr(), k.data_ptr(), v.data_ptr(), oq.data_ptr(),
                            ok.data_ptr(), buf.pyramid, _stream())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    want = [t.clone() for t in (oq, ok, buf.pq[1], buf.pk[2], buf.pv[2])]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for t in (oq, ok, buf.pq[1], buf.pk[2], buf.pv[2]):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for t, w in zip((oq, ok, buf.pq[1], buf.pk[2], buf.pv[2]), want):
        assert torch.equal(t, w)


@pytest.mark.parametrize("rot", [32, 64, 128])
@pytest.mark.parametrize("rows", [1, 255, 257, 18944, 18945, 37901, 65536])
def test_table_zorder_equals_positions(rows, rot):
    """The Z-order's table, computed entry by entry or by squares, is the one of the same positions, bit for bit."""
    i = torch.arange(rows, dtype=torch.int64, device="cuda")
    pos = torch.stack([sum(((i >> (2 * b + a)) & 1) << b for b in range(8)) for a in range(2)], 1).int()
    rope = llsa.make_rope(rot, axes=2)
    a, b = _table(rope, rows, None, rot // 2), _table(rope, rows, pos.contiguous(), rot // 2)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
