"""Cross attention on the GPU (forward and backward, bf16 and fp32) against
the 64-bit form, with bounds derived from the kernels' arithmetic."""

import math

import pytest
import torch

import block_testlib as bt
import hierarchical_top_sparse_llsa_b200 as llsa

pytestmark = pytest.mark.gpu

DT = {"f32": (torch.float32, llsa.F32), "bf16": (torch.bfloat16, llsa.BF16)}


def make(B, H, Hkv, N, S, D, dtype, seed=0, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype][0]

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x = dict(q=gain * rnd(B, H, N, D), k=rnd(B, Hkv, S, D), v=rnd(B, Hkv, S, D) + 0.5, do=rnd(B, H, N, D))
    return {n: t.to(dt) for n, t in x.items()}


def _p(t):
    return None if t is None or t.numel() == 0 else t.data_ptr()


def run(x, kv_len=None, mask=None, scale=0.0, residual=False, grads=True):
    """Both calls; every output starts as NaN."""
    q, k, v = x["q"], x["k"], x["v"]
    B, H, N, D = q.shape
    Hkv, S = k.shape[1:3]
    code = llsa.BF16 if q.dtype == torch.bfloat16 else llsa.F32
    desc = llsa.make_cross(B, H, Hkv, N, S, D, code, scale)
    s = torch.cuda.current_stream().cuda_stream
    nan = float("nan")
    o, lse = torch.full_like(q, nan), torch.full((B, H, N), nan, device="cuda")
    res = torch.full(q.shape, nan, dtype=torch.bfloat16, device="cuda") if residual else None
    fb, bb = llsa.llsa_cross_fwd_workspace_bytes(desc), llsa.llsa_cross_bwd_workspace_bytes(desc)
    ws = torch.full((max(fb, bb, 4) // 4 + 64,), nan, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    llsa.llsa_cross_attn_fwd(desc, _p(q), _p(k), _p(v), _p(kv_len), _p(mask), _p(o), _p(res), _p(lse), _p(ws), fb,
                             _p(st), s)
    out = {"o": o, "lse": lse}
    if residual:
        out["res"] = res
    if grads:
        ws.fill_(nan)
        g = {n: torch.full_like(x[n], nan) for n in "qkv"}
        llsa.llsa_cross_attn_bwd(desc, _p(q), _p(k), _p(v), _p(kv_len), _p(mask), _p(o), _p(res), _p(lse),
                                 _p(x["do"]), _p(g["q"]), _p(g["k"]), _p(g["v"]), _p(ws), bb, _p(st), s)
        out.update({"d" + n: t for n, t in g.items()})
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    return out


def check(x, out, kv_len=None, mask=None, scale=None, residual=False):
    bf16 = x["q"].dtype == torch.bfloat16
    want = bt.cross(x["q"], x["k"], x["v"], kv_len, mask, scale, x["do"], bf16, residual)
    for name, (t, bound) in want.items():
        if t.numel():
            bt.within(out[name], t, bound, name)


SHAPES = [
    # B, H, Hkv, N, S, D
    (1, 1, 1, 1, 1, 64),
    (1, 2, 2, 5, 3, 128),
    (2, 3, 3, 64, 64, 64),
    (1, 2, 1, 65, 77, 64),
    (2, 4, 2, 127, 128, 128),
    (1, 2, 2, 128, 129, 64),
    (1, 3, 1, 129, 15, 128),
    (2, 2, 2, 200, 256, 64),
    (1, 4, 4, 255, 257, 64),
    (1, 2, 1, 300, 333, 128),
    (3, 8, 2, 97, 512, 64),
    (1, 1, 1, 1, 4097, 64),     # one token over a long sequence: the keys are split
    (2, 6, 3, 3, 1000, 128),
    (1, 16, 4, 17, 2500, 128),
    (1, 1, 1, 3000, 1, 64),     # one key
    (1, 2, 2, 2500, 80, 64),
    (1, 2, 2, 1111, 700, 128),
    (2, 1, 1, 1025, 16, 128),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(shape, dtype):
    x = make(*shape, dtype)
    check(x, run(x))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(4, 2, 1, 150, 200, 64), (4, 2, 2, 70, 300, 128), (4, 4, 2, 2, 1500, 64)], ids=str)
def test_masks(shape, dtype):
    B, _, _, _, S, _ = shape
    x = make(*shape, dtype, seed=1)
    g = torch.Generator(device="cuda").manual_seed(2)
    # none, all but one, one, more than there are
    lens = torch.tensor([0, S - 1, 1, S + 9], dtype=torch.int32, device="cuda")
    mask = (torch.rand(B, S, generator=g, device="cuda") < 0.6).to(torch.uint8) * 3
    mask[1] = 0                 # an entry that sees nothing
    mask[3, : S // 2] = 0       # whole tiles hidden in front
    for kl, m in ((lens, None), (None, mask), (lens.flip(0).contiguous(), mask), (-lens, None)):
        # what is not seen holds values that would spoil any sum they entered
        ok = bt.seen(B, S, kl, m, "cuda")
        y = dict(x)
        for n in "kv":
            y[n] = x[n].clone()
            y[n].masked_fill_(~ok[:, None, :, None], float("nan"))
            y[n][:, :, ::7].masked_fill_(~ok[:, None, ::7, None], float("inf"))
        out = run(y, kl, m)
        check(y, out, kl, m)
        empty = ~ok.any(1)
        assert (out["o"][empty] == 0).all() and (out["dq"][empty] == 0).all()
        assert (out["lse"][empty] == -math.inf).all()
        hidden = (~ok)[:, None, :, None].expand_as(out["dk"])
        assert (out["dk"][hidden] == 0).all() and (out["dv"][hidden] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_states_at_all(dtype):
    x = make(2, 3, 3, 70, 0, 64, dtype)
    out = run(x)
    assert (out["o"] == 0).all() and (out["lse"] == -math.inf).all() and (out["dq"] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.03, 0.6])
def test_scale_and_peaked_rows(dtype, scale):
    # at 0.6 rows sit on one or two keys; the maximum moves from tile to tile
    x = make(1, 2, 2, 140, 520, 64, dtype, seed=3, gain=2.0)
    x["k"] = x["k"] * torch.linspace(0.2, 1.0, 520, device="cuda")[:, None].to(x["k"].dtype)
    check(x, run(x, scale=scale), scale=scale)


def test_residual():
    x = make(1, 4, 2, 200, 150, 64, "bf16", seed=4, gain=2.0)
    plain, res = run(x), run(x, residual=True)
    assert torch.equal(plain["o"], res["o"]) and torch.equal(plain["lse"], res["lse"])
    check(x, res, residual=True)
    # o + res holds the kernel's fp32 O to a bf16 step of the residual
    want, bound = bt.cross(x["q"], x["k"], x["v"])["o"]
    p_abs = bound - (want.abs() + bound) * bt.UB  # the bound without the store's rounding
    err = (res["o"].double() + res["res"].double() - want).abs()
    assert (err <= p_abs + want.abs() * 2.0**-15 + 1e-6).all()
    assert (res["res"].double().abs() <= want.abs() * bt.UB + bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(2, 4, 2, 333, 300, 64), (1, 2, 2, 9, 3000, 128)], ids=str)
def test_runs_are_identical(shape, dtype):
    x = make(*shape, dtype, seed=5)
    a, b = run(x), run(x)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_gradients_against_differences():
    # fp32: a step along a random direction moves <dO, O> by the gradient;
    # central differences of the GPU's own forward, whose fp32 rounding the
    # step divides
    x = make(1, 2, 1, 37, 45, 64, "f32", seed=6)
    out = run(x)
    h = 2.0**-5
    for name in "qkv":
        g = torch.Generator(device="cuda").manual_seed(7)
        z = torch.randn(x[name].shape, generator=g, device="cuda")
        z = z / z.norm()

        def loss(sign):
            y = dict(x, **{name: x[name] + sign * h * z})
            return (run(y, grads=False)["o"].double() * x["do"].double()).sum()

        # O(h^4) from a second, doubled step (Richardson)
        one = (loss(1) - loss(-1)) / (2 * h)
        two = (loss(2) - loss(-2)) / (4 * h)
        diff = float((4 * one - two) / 3)
        want = float((out["d" + name].double() * z.double()).sum())
        o, bound = bt.cross(x["q"], x["k"], x["v"], bf16=False)["o"]
        noise = float((bound * x["do"].double().abs()).sum()) / h
        # the fourth-order remainder: the loss along a unit step has derivatives
        # of at most the size of sum |dO||V| times |z q| powers below 1 / 8
        rest = h**4 * float((x["do"].double().abs().sum(-1)).max()) * float(x["v"].abs().max())
        assert abs(diff - want) <= noise + rest, name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graph_and_streams(dtype):
    shape = (1, 4, 4, 300, 200, 64)
    x = make(*shape, dtype, seed=8)
    want = run(x)
    B, H, Hkv, N, S, D = shape
    desc = llsa.make_cross(B, H, Hkv, N, S, D, DT[dtype][1])
    # two captured graphs with workspaces of their own, replayed side by side
    states = []
    for _ in range(2):
        o, lse = torch.empty_like(x["q"]), torch.empty(B, H, N, device="cuda")
        g = {n: torch.empty_like(x[n]) for n in "qkv"}
        fb, bb = llsa.llsa_cross_fwd_workspace_bytes(desc), llsa.llsa_cross_bwd_workspace_bytes(desc)
        ws = torch.empty(max(fb, bb, 1), dtype=torch.uint8, device="cuda")
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            s = torch.cuda.current_stream().cuda_stream
            llsa.llsa_cross_attn_fwd(desc, _p(x["q"]), _p(x["k"]), _p(x["v"]), None, None, _p(o), None, _p(lse),
                                     _p(ws), fb, None, s)
            llsa.llsa_cross_attn_bwd(desc, _p(x["q"]), _p(x["k"]), _p(x["v"]), None, None, _p(o), None, _p(lse),
                                     _p(x["do"]), _p(g["q"]), _p(g["k"]), _p(g["v"]), _p(ws), bb, None, s)
        states.append((graph, torch.cuda.Stream(), dict(o=o, lse=lse, dq=g["q"], dk=g["k"], dv=g["v"]), ws))
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, side, out, _ in states:
            with torch.cuda.stream(side):
                for t in out.values():
                    t.fill_(float("nan"))
                graph.replay()
        torch.cuda.synchronize()
        for _, _, out, _ in states:
            for n in out:
                assert torch.equal(out[n], want[n]), n
