"""The operators of a conditioned block together, as a program calls them:
projection -> rotation with the pyramid -> selection -> sparse attention, cross
attention to a caption, and the backward down to the projection's output; and
cross attention at sizes where every CTA of the persistent kernels walks many
items."""

import math

import pytest
import torch

import block_testlib as bt
import hierarchical_top_sparse_llsa_b200 as llsa
from test_gpu_cross_attn import check, make, run

pytestmark = pytest.mark.gpu


def _p(t):
    return None if t is None else t.data_ptr()


def _stream():
    return torch.cuda.current_stream().cuda_stream


MANY = [
    # B, H, Hkv, N, S, D: thousands of row tiles, so that items, heads and
    # batch entries change inside a CTA
    (2, 14, 14, 16387, 70, 64),
    (1, 9, 3, 30001, 40, 64),
    (2, 12, 12, 9001, 130, 128),
    (3, 40, 40, 129, 257, 64),    # a head is a tile and one row
    (40, 4, 1, 33, 100, 128),     # batch entries change with every item
    (2, 5, 5, 257, 6000, 64),     # more keys than stay in shared memory
]


@pytest.mark.parametrize("shape", MANY, ids=str)
@pytest.mark.parametrize("masked", [False, True])
def test_many_items(shape, masked):
    B, _, _, _, S, _ = shape
    x = make(*shape, "bf16", seed=21)
    lens = mask = None
    if masked:
        g = torch.Generator(device="cuda").manual_seed(22)
        lens = torch.randint(0, S + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        mask = (torch.rand(B, S, generator=g, device="cuda") < 0.8).to(torch.uint8)
    a = run(x, lens, mask)
    check(x, a, lens, mask)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")  # larger than the L2 cache
    for cold in (False, True, True):  # the same every time, whatever order the loads arrive in
        if cold:
            flush.zero_()
        b = run(x, lens, mask)
        for n in a:
            assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(3, 4, 2, 50, 9, 64), (3, 2, 2, 300, 200, 128), (3, 2, 1, 2, 2000, 64)], ids=str)
def test_one_key_has_no_gradient_of_its_score(shape, dtype):
    # a query that sees one key has probability 1 whatever the score: dQ and
    # that key's dK are zero, exactly, and its dV is the sum of dO
    B, H, Hkv, N, S, D = shape
    x = make(*shape, dtype, seed=23)
    mask = torch.zeros(B, S, dtype=torch.uint8, device="cuda")
    mask[0, 0] = mask[1, S - 1] = 1
    mask[2] = 1
    lens = torch.tensor([S, S, 1], dtype=torch.int32, device="cuda")
    out = run(x, lens, mask)
    check(x, out, lens, mask)
    assert (out["dq"] == 0).all() and (out["dk"] == 0).all()
    one = make(B, H, Hkv, N, 1, D, dtype, seed=24)
    out = run(one)
    check(one, out)
    assert (out["dq"] == 0).all() and (out["dk"] == 0).all()


def test_gradients_where_many_keys_share_a_row():
    # flat rows over many keys with a large common part: Delta from the stored
    # bf16 O would be off by more than the gradient
    x = make(1, 2, 2, 130, 3001, 64, "bf16", seed=25, gain=0.3)
    for n in "kv":
        x[n] = (x[n].float() + 4.0).to(torch.bfloat16)
    out = run(x)
    check(x, out)
    want = bt.cross(x["q"], x["k"], x["v"], do=x["do"])
    for n in ("dq", "dk", "dv"):
        w = want[n][0]
        # roundings of P, dS and the result are independent: half a step each
        # in the worst case, and P and dS enter sums of many terms
        rel = float((out[n].double() - w).norm() / w.norm())
        assert rel <= 4 * bt.UB, (n, rel)


@pytest.mark.parametrize("dtype,code", [(torch.bfloat16, llsa.BF16), (torch.float32, llsa.F32)])
def test_block_chain(dtype, code):
    B, H, N, D, L, topk, S = 2, 2, 1024, 64, 2, 8, 77
    g = torch.Generator(device="cuda").manual_seed(26)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda").to(dtype)

    q, k, v, do = (rnd(B, H, N, D) for _ in range(4))
    ck, cv = rnd(B, H, S, D), rnd(B, H, S, D)
    lens = torch.tensor([S, 50], dtype=torch.int32, device="cuda")
    desc = llsa.make_desc(B, H, N, D, L, topk, code)
    rope = llsa.make_rope(D, axes=2)
    cross = llsa.make_cross(B, H, H, N, S, D, code)
    buf = llsa.LlsaBuffers(desc, "cuda")
    tab = torch.empty(N, D // 2, 2, device="cuda")
    rq, rk, o, co = (torch.empty_like(q) for _ in range(4))
    lse, clse = torch.empty(B, H, N, device="cuda"), torch.empty(B, H, N, device="cuda")
    grads = {n: torch.empty_like(t) for n, t in dict(do1=q, dq=q, dk=q, dv=q, ck=ck, cv=cv, uq=q, uk=q).items()}
    fb, bb = llsa.llsa_cross_fwd_workspace_bytes(cross), llsa.llsa_cross_bwd_workspace_bytes(cross)
    ws = torch.empty(max(fb, bb, 1), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        s = _stream()
        llsa.llsa_rope_table(rope, N, None, _p(tab), s)
        llsa.llsa_rope_pool(desc, rope, _p(tab), N, _p(q), _p(k), _p(v), _p(rq), _p(rk), buf.pyramid, s)
        llsa.llsa_select(desc, buf.pyramid, buf.indices, s)
        llsa.llsa_attn_fwd(desc, _p(rq), _p(rk), _p(v), buf.pyramid, buf.indices, _p(o), _p(lse), _p(st), s)
        # the sparse attention's output asks the caption
        llsa.llsa_cross_attn_fwd(cross, _p(o), _p(ck), _p(cv), _p(lens), None, _p(co), None, _p(clse), _p(ws), fb,
                                 _p(st), s)
        llsa.llsa_cross_attn_bwd(cross, _p(o), _p(ck), _p(cv), _p(lens), None, _p(co), None, _p(clse), _p(do),
                                 _p(grads["do1"]), _p(grads["ck"]), _p(grads["cv"]), _p(ws), bb, _p(st), s)
        llsa.llsa_index_transpose(desc, buf.indices, buf.csr, _p(buf.tr_ws), buf.tr_ws_bytes, _p(st), s)
        llsa.llsa_attn_bwd(desc, _p(rq), _p(rk), _p(v), buf.pyramid, _p(o), _p(lse), _p(grads["do1"]), buf.indices,
                           buf.csr, _p(grads["dq"]), _p(grads["dk"]), _p(grads["dv"]), _p(buf.ws), buf.ws_bytes,
                           _p(st), s)
        llsa.llsa_rope(rope, B, H, N, D, code, _p(tab), N, _p(grads["dq"]), _p(grads["dk"]), _p(grads["uq"]),
                       _p(grads["uk"]), True, s)

    step()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    half = bt.UB if dtype == torch.bfloat16 else bt.U
    # rotation and its adjoint, each against the values that it was given
    t64 = bt.rope_table(bt.zorder_xy(N), D, 2).cuda()
    for got, src, adj in ((rq, q, False), (rk, k, False), (grads["uq"], grads["dq"], True),
                          (grads["uk"], grads["dk"], True)):
        y, mag = bt.rotate(src.double(), t64, D, False, adj)
        err = (got.double() - y).abs()
        # the table's entries are within 2^-22 of the exact ones, so a pair
        # (a, b) moves by up to (|a| + |b|) 2^-22, however small a c or b s is
        a = src.double().abs()
        pair = (a[..., : D // 2] + a[..., D // 2 :]).repeat(1, 1, 1, 2)
        assert (err <= bt.rotate_bound(y, mag, dtype == torch.bfloat16) + pair * 2.0**-22 * (1 + half)).all()
    # cross attention of the sparse attention's output
    x = dict(q=o, k=ck, v=cv, do=do)
    out = dict(o=co, lse=clse, dq=grads["do1"], dk=grads["ck"], dv=grads["cv"])
    check(x, out, lens)
    assert all(torch.isfinite(t).all() for t in (o, *grads.values()))
    assert float(lse.abs().max()) < math.inf
    # a captured step gives the same bits
    want = {n: t.clone() for n, t in {**grads, "co": co, "o": o}.items()}
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for t in (*grads.values(), co, o, rq, rk):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for n, t in {**grads, "co": co, "o": o}.items():
        assert torch.equal(t, want[n]), n


def _banded(shape, dtype, band=4096):
    """A tensor inside a larger one of the value 7, and a check that the rest still has it."""
    n = math.prod(shape)
    whole = torch.full((n + 2 * band,), 7.0, dtype=dtype, device="cuda")
    inner = whole[band:band + n].view(shape)
    return inner, lambda: bool((whole[:band] == 7).all()) and bool((whole[band + n:] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(2, 6, 2, 131, 77, 64), (1, 2, 1, 1, 2049, 128), (3, 2, 2, 515, 1, 64),
                                   (1, 4, 4, 1023, 333, 128)], ids=str)
def test_replay_on_new_inputs_writes_outputs_alone(shape, dtype):
    """A captured forward and backward without a status word, replayed after
    its inputs changed: the values of the new inputs, and nothing around the
    outputs or the workspace is written."""
    B, H, Hkv, N, S, D = shape
    x, y = make(*shape, dtype, seed=31), make(*shape, dtype, seed=32)
    t = x["q"].dtype
    desc = llsa.make_cross(B, H, Hkv, N, S, D, llsa.BF16 if dtype == "bf16" else llsa.F32)
    fb, bb = llsa.llsa_cross_fwd_workspace_bytes(desc), llsa.llsa_cross_bwd_workspace_bytes(desc)
    bands = {n: _banded(x[n[1:] if n != "o" else "q"].shape, t) for n in ("o", "dq", "dk", "dv")}
    bands["lse"] = _banded((B, H, N), torch.float32)
    bands["ws"] = _banded((max(fb, bb, 256) // 4,), torch.float32)
    out = {n: b[0] for n, b in bands.items()}

    def step():
        s = _stream()
        llsa.llsa_cross_attn_fwd(desc, _p(x["q"]), _p(x["k"]), _p(x["v"]), None, None, _p(out["o"]), None,
                                 _p(out["lse"]), _p(out["ws"]), fb, None, s)
        llsa.llsa_cross_attn_bwd(desc, _p(x["q"]), _p(x["k"]), _p(x["v"]), None, None, _p(out["o"]), None,
                                 _p(out["lse"]), _p(x["do"]), _p(out["dq"]), _p(out["dk"]), _p(out["dv"]),
                                 _p(out["ws"]), bb, None, s)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    for n in x:
        x[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    want = run(y)
    for n, w in want.items():
        assert torch.equal(out[n], w), n
    for n, (_, whole) in bands.items():
        assert whole(), n
    check(y, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,rot,layout", [(64, 64, 0), (64, 20, 0), (128, 128, 1), (128, 6, 1)])
def test_rotation_writes_outputs_alone(D, rot, layout, dtype):
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    code = llsa.BF16 if dtype == "bf16" else llsa.F32
    B, H, N = 2, 3, 77
    rope = llsa.make_rope(rot, layout=layout)
    table, tab_ok = _banded((N, rot // 2, 2), torch.float32)
    llsa.llsa_rope_table(rope, N, None, _p(table), _stream())
    g = torch.Generator(device="cuda").manual_seed(33)
    q, k = (torch.randn(B, H, N, D, generator=g, device="cuda").to(t) for _ in "qk")
    (qo, q_ok), (ko, k_ok) = _banded(q.shape, t), _banded(k.shape, t)
    llsa.llsa_rope(rope, B, H, N, D, code, _p(table), N, _p(q), _p(k), _p(qo), _p(ko), 0, _stream())
    torch.cuda.synchronize()
    assert tab_ok() and q_ok() and k_ok()
    for x, got in ((q, qo), (k, ko)):
        y, mag = bt.rotate(x.double(), table.double(), rot, bool(layout))
        bt.within(got, y, bt.rotate_bound(y, mag, dtype == "bf16"), "rotation")
