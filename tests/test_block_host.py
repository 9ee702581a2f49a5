"""CPU-only checks of the calls around the self-attention (rotary positions,
cross attention): refusals before any launch, workspace sizes, and the 64-bit
forms that the GPU tests compare with, against differences and properties."""

import math

import pytest
import torch

import block_testlib as bt
import hierarchical_top_sparse_llsa_b200 as llsa

A, W = 1 << 20, 1 << 30  # addresses that no refused call reads


def _apart(i):
    return (i + 1) << 34


def rope_table(**kw):
    r = dict(rot_dim=64)
    r.update({k: v for k, v in kw.items() if k in ("rot_dim", "layout", "axes", "base", "scaling", "factor", "orig_len",
                                                   "mscale", "beta_fast", "beta_slow")})
    return llsa.llsa_rope_table(llsa.make_rope(**r), kw.get("rows", 10), kw.get("pos"), kw.get("table", A), check=False)


@pytest.mark.parametrize("kw,status", [
    (dict(rot_dim=0), llsa.ERR_INVALID_ARG),
    (dict(rot_dim=7), llsa.ERR_INVALID_ARG),
    (dict(rot_dim=130), llsa.ERR_UNSUPPORTED),
    (dict(layout=2), llsa.ERR_INVALID_ARG),
    (dict(axes=0), llsa.ERR_INVALID_ARG),
    (dict(axes=3), llsa.ERR_INVALID_ARG),
    (dict(rot_dim=6, axes=2), llsa.ERR_INVALID_ARG),  # three pairs for two axes
    (dict(base=1.0), llsa.ERR_INVALID_ARG),
    (dict(base=-5.0), llsa.ERR_INVALID_ARG),
    (dict(base=math.nan), llsa.ERR_INVALID_ARG),
    (dict(base=math.inf), llsa.ERR_INVALID_ARG),
    (dict(factor=0.5), llsa.ERR_INVALID_ARG),
    (dict(factor=math.nan), llsa.ERR_INVALID_ARG),
    (dict(scaling=4), llsa.ERR_INVALID_ARG),
    (dict(mscale=-1.0), llsa.ERR_INVALID_ARG),
    (dict(mscale=math.nan), llsa.ERR_INVALID_ARG),
    (dict(scaling=llsa.ROPE_SCALE_YARN, factor=2.0), llsa.ERR_INVALID_ARG),  # no trained length
    (dict(scaling=llsa.ROPE_SCALE_YARN, factor=2.0, orig_len=99, beta_fast=1.0, beta_slow=2.0), llsa.ERR_INVALID_ARG),
    (dict(rows=0), llsa.ERR_INVALID_ARG),
    (dict(table=None), llsa.ERR_INVALID_ARG),
    (dict(table=A + 8), llsa.ERR_INVALID_ARG),
    (dict(pos=A + 2), llsa.ERR_INVALID_ARG),
])
def test_rope_table_refusals(kw, status):
    assert rope_table(**kw) == status


def rope(**kw):
    a = dict(B=2, H=3, N=100, D=64, dtype=llsa.BF16, table=A, table_rows=100, q=_apart(0), k=_apart(1), q_out=_apart(2),
             k_out=_apart(3), rot_dim=64, layout=0)
    a.update(kw)
    r = llsa.make_rope(a.pop("rot_dim"), layout=a.pop("layout"))
    return llsa.llsa_rope(r, *(a[n] for n in ("B", "H", "N", "D", "dtype", "table", "table_rows", "q", "k", "q_out",
                                              "k_out")), check=False)


SIZE = 2 * 3 * 100 * 64 * 2  # bytes of one tensor above


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), llsa.ERR_UNSUPPORTED),
    (dict(D=64, rot_dim=128), llsa.ERR_INVALID_ARG),
    (dict(dtype=7), llsa.ERR_INVALID_ARG),
    (dict(B=0), llsa.ERR_INVALID_ARG),
    (dict(H=0), llsa.ERR_INVALID_ARG),
    (dict(N=0), llsa.ERR_INVALID_ARG),
    (dict(table_rows=99), llsa.ERR_INVALID_ARG),
    (dict(table_rows=300), llsa.ERR_INVALID_ARG),
    (dict(table=None), llsa.ERR_INVALID_ARG),
    (dict(q=None), llsa.ERR_INVALID_ARG),
    (dict(q_out=None), llsa.ERR_INVALID_ARG),
    (dict(k=None), llsa.ERR_INVALID_ARG),      # k_out without k
    (dict(k_out=None), llsa.ERR_INVALID_ARG),
    (dict(q=_apart(0) + 8), llsa.ERR_INVALID_ARG),
    (dict(k_out=_apart(3) + 2), llsa.ERR_INVALID_ARG),
    (dict(q_out=_apart(0) + 16), llsa.ERR_INVALID_ARG),             # over its input, shifted
    (dict(q_out=_apart(1)), llsa.ERR_INVALID_ARG),                  # over the other input
    (dict(k_out=_apart(2)), llsa.ERR_INVALID_ARG),                  # both outputs in one place
    (dict(k_out=_apart(2) + SIZE - 16), llsa.ERR_INVALID_ARG),
    (dict(rot_dim=33), llsa.ERR_INVALID_ARG),
])
def test_rope_refusals(kw, status):
    assert rope(**kw) == status


def rope_pool(desc=None, rot_dim=64, pyr=True, **kw):
    desc = desc or llsa.make_desc(1, 2, 1024, 64, 2, 4, llsa.BF16)
    p = llsa.LlsaPyramid()
    if pyr:
        for l in range(1, 3):
            p.q[l] = p.k[l] = p.v[l] = _apart(10)
    a = dict(table=A, table_rows=1024, q=_apart(0), k=_apart(1), v=_apart(2), q_out=_apart(3), k_out=_apart(4))
    a.update(kw)
    return llsa.llsa_rope_pool(desc, llsa.make_rope(rot_dim), a["table"], a["table_rows"], a["q"], a["k"], a["v"],
                               a["q_out"], a["k_out"], p, check=False)


@pytest.mark.parametrize("kw,status", [
    (dict(desc=llsa.make_desc(1, 2, 1000, 64, 2, 4, llsa.BF16)), llsa.ERR_INVALID_ARG),
    (dict(desc=llsa.make_desc(1, 2, 1024, 96, 2, 4, llsa.BF16)), llsa.ERR_UNSUPPORTED),
    (dict(rot_dim=128), llsa.ERR_INVALID_ARG),
    (dict(pyr=False), llsa.ERR_INVALID_ARG),
    (dict(v=None), llsa.ERR_INVALID_ARG),
    (dict(q_out=None), llsa.ERR_INVALID_ARG),
    (dict(q_out=_apart(2)), llsa.ERR_INVALID_ARG),  # over V
    (dict(k_out=_apart(0)), llsa.ERR_INVALID_ARG),
    (dict(table_rows=1000), llsa.ERR_INVALID_ARG),
    (dict(v=_apart(2) + 4), llsa.ERR_INVALID_ARG),
])
def test_rope_pool_refusals(kw, status):
    assert rope_pool(**kw) == status


def _apart_pyramid(**kw):
    p = llsa.LlsaPyramid()
    for i, (l, n) in enumerate((l, n) for l in (1, 2) for n in "qkv"):
        getattr(p, n)[l] = _apart(10 + i)
    for name, ptr in kw.items():
        getattr(p, name[0])[int(name[1])] = ptr
    return p


# Outputs over the table or the pyramid.  Q has 1024 rows x 2 heads x 64 bf16
# (256 KB), the table 1024 x 32 pairs (256 KB), level 1 of Q 32 KB.
@pytest.mark.parametrize("kw,pyr", [
    (dict(q_out=A + 1024), {}),
    (dict(k_out=A + 256 * 1024 - 16), {}),
    ({}, dict(q1=A)),
    ({}, dict(q1=_apart(0) + 256)),
    ({}, dict(k2=_apart(1))),
    ({}, dict(v2=_apart(2) + 16)),
    ({}, dict(q1=_apart(3) + 4096)),
    ({}, dict(v2=_apart(4))),
    ({}, dict(k1=_apart(10) + 32 * 1024 - 16)),
    ({}, dict(q2=_apart(11))),
])
def test_rope_pool_refuses_overlap(kw, pyr):
    a = dict(table=A, q=_apart(0), k=_apart(1), v=_apart(2), q_out=_apart(3), k_out=_apart(4))
    a.update(kw)
    d = llsa.make_desc(1, 2, 1024, 64, 2, 4, llsa.BF16)
    st = llsa.llsa_rope_pool(d, llsa.make_rope(64), a["table"], 1024, a["q"], a["k"], a["v"], a["q_out"], a["k_out"],
                             _apart_pyramid(**pyr), check=False)
    assert st == llsa.ERR_INVALID_ARG


def test_rope_table_refuses_pos_over_the_table():
    r = llsa.make_rope(64, axes=2)  # 10 rows: 2560 bytes, and 80 of positions
    for pos in (A, A + 2556, A - 76):
        assert llsa.llsa_rope_table(r, 10, pos, A, check=False) == llsa.ERR_INVALID_ARG


@pytest.mark.parametrize("out", [dict(q_out=A + 16), dict(k_out=A + 12672 - 16)])
def test_rope_refuses_outputs_over_the_table(out):
    """99 rows of 32 pairs: 25344 bytes a table, 12672 of them of rot_dim 32."""
    a = dict(q_out=_apart(2), k_out=_apart(3))
    a.update(out)
    st = llsa.llsa_rope(llsa.make_rope(32), 1, 2, 99, 64, llsa.BF16, A, 99, _apart(0), _apart(1), a["q_out"],
                        a["k_out"], 0, check=False)
    assert st == llsa.ERR_INVALID_ARG


def desc(**kw):
    a = dict(B=2, H=4, Hkv=2, N=100, S=77, D=64, dtype=llsa.BF16)
    a.update(kw)
    return llsa.make_cross(**a)


BAD_DESC = [
    (dict(B=0), llsa.ERR_INVALID_ARG), (dict(H=0), llsa.ERR_INVALID_ARG), (dict(Hkv=0), llsa.ERR_INVALID_ARG),
    (dict(H=4, Hkv=3), llsa.ERR_INVALID_ARG), (dict(N=0), llsa.ERR_INVALID_ARG), (dict(S=-1), llsa.ERR_INVALID_ARG),
    (dict(D=96), llsa.ERR_UNSUPPORTED), (dict(D=0), llsa.ERR_INVALID_ARG), (dict(dtype=2), llsa.ERR_INVALID_ARG),
    (dict(flags=1), llsa.ERR_INVALID_ARG), (dict(sm_scale=-1.0), llsa.ERR_INVALID_ARG),
    (dict(sm_scale=math.nan), llsa.ERR_INVALID_ARG), (dict(sm_scale=math.inf), llsa.ERR_INVALID_ARG),
    (dict(B=1 << 16, H=1 << 15, Hkv=1, N=2), llsa.ERR_UNSUPPORTED),
    (dict(B=1 << 10, S=1 << 21), llsa.ERR_UNSUPPORTED),
]
FWD = ("q", "k", "v", "kv_len", "mask", "o", "res", "lse", "ws")
BWD = ("q", "k", "v", "kv_len", "mask", "o", "res", "lse", "do", "dq", "dk", "dv", "ws")


def cross(which, d=None, ws_bytes=1 << 40, **kw):
    names = FWD if which == "fwd" else BWD
    a = {n: _apart(i) for i, n in enumerate(BWD)}
    a.update(kv_len=None, mask=None, res=None)
    a.update(kw)
    f = llsa.llsa_cross_attn_fwd if which == "fwd" else llsa.llsa_cross_attn_bwd
    return f(d if d is not None else desc(), *(a[n] for n in names), ws_bytes, check=False)


@pytest.mark.parametrize("which", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,status", BAD_DESC, ids=str)
def test_cross_descriptor_refusals(which, kw, status):
    assert cross(which, desc(**kw)) == status
    assert llsa.llsa_cross_fwd_workspace_bytes(desc(**kw)) == 0
    assert llsa.llsa_cross_bwd_workspace_bytes(desc(**kw)) == 0


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_cross_pointer_refusals(which):
    inv = llsa.ERR_INVALID_ARG
    need = ("q", "k", "v", "o", "lse") + (("do", "dq", "dk", "dv") if which == "bwd" else ())
    for n in need:
        assert cross(which, **{n: None}) == inv, n
        if n != "lse":
            assert cross(which, **{n: A + 8}) == inv, n
    assert cross(which, lse=A + 2) == inv
    assert cross(which, kv_len=A + 2) == inv
    assert cross(which, res=A + 8) == inv
    out = "o" if which == "fwd" else "dq"
    assert cross(which, **{out: _apart(0)}) == inv  # over q
    assert cross(which, **{out: _apart(1) + 16}) == inv
    if which == "bwd":
        assert cross(which, dk=_apart(2)) == inv
        assert cross(which, dv=_apart(BWD.index("dk"))) == inv


def test_cross_workspace_refusals():
    d = desc(N=3, S=5000)
    for which, need in (("fwd", llsa.llsa_cross_fwd_workspace_bytes(d)), ("bwd", llsa.llsa_cross_bwd_workspace_bytes(d))):
        assert need > 0
        assert cross(which, d, ws_bytes=need - 1) == llsa.ERR_WORKSPACE
        assert cross(which, d, ws=None) == llsa.ERR_INVALID_ARG
        assert cross(which, d, ws=W + 128) == llsa.ERR_INVALID_ARG


# ----------------------------------------------- the 64-bit forms themselves
def test_cross_form_against_differences():
    g = torch.Generator().manual_seed(0)
    B, H, Hkv, N, S, D = 2, 4, 2, 5, 9, 64
    x = {n: torch.randn(B, h, t, D, generator=g, dtype=torch.float64) for n, h, t in
         (("q", H, N), ("k", Hkv, S), ("v", Hkv, S), ("do", H, N))}
    lens = torch.tensor([9, 4], dtype=torch.int32)
    mask = (torch.rand(B, S, generator=g) < 0.7).to(torch.uint8)
    ref = bt.cross(x["q"], x["k"], x["v"], lens, mask, 0.3, x["do"])
    h = 1e-5
    for n in "qkv":
        z = torch.randn(x[n].shape, generator=g, dtype=torch.float64)
        vals = [(bt.cross(**{**{m: x[m] for m in "qkv"}, n: x[n] + sign * h * z}, kv_len=lens, mask=mask,
                          scale=0.3)["o"][0] * x["do"]).sum() for sign in (1, -1)]
        diff = float(vals[0] - vals[1]) / (2 * h)
        want = float((ref["d" + n][0] * z).sum())
        assert abs(diff - want) < 1e-6 * max(1.0, abs(want)), n


def test_rotation_form_turns_pairs():
    x = torch.randn(1, 2, 6, 64, dtype=torch.float64)
    tab = bt.rope_table(torch.arange(6, dtype=torch.float64)[:, None], 32)
    for inter in (False, True):
        y, _ = bt.rotate(x, tab, 32, inter)
        back, _ = bt.rotate(y, tab, 32, inter, adjoint=True)
        assert torch.allclose(back, x, atol=1e-14)  # orthogonal
        i, j = (2, 3) if inter else (1, 17)  # pair 1 of token 5
        t = 5 * 10000.0 ** (-1 / 16)
        assert math.isclose(y[0, 1, 5, i], x[0, 1, 5, i] * math.cos(t) - x[0, 1, 5, j] * math.sin(t), abs_tol=1e-14)
        assert torch.equal(y[..., 32:], x[..., 32:])


def test_frequency_scalings():
    plain = bt.inv_freq(32)
    assert torch.allclose(bt.inv_freq(32, scaling=1, factor=4.0), plain / 4)
    ntk = bt.inv_freq(32, scaling=2, factor=4.0)
    assert ntk[0] == 1 and math.isclose(ntk[-1], plain[-1] / 4, rel_tol=1e-12)  # the slowest is stretched in full
    yarn = bt.inv_freq(32, scaling=3, factor=4.0, orig_len=2048)
    assert yarn[0] == plain[0] and math.isclose(yarn[-1], plain[-1] / 4, rel_tol=1e-12)
    assert ((yarn <= plain) & (yarn >= plain / 4 * (1 - 1e-12))).all()


def test_cross_fp32_backward_without_parts_needs_no_workspace():
    # as many tiles as SMs several times over: nothing is cut
    d = desc(B=8, H=16, Hkv=16, N=1024, S=77, dtype=llsa.F32)
    assert llsa.llsa_cross_bwd_workspace_bytes(d) == 0
    d.dtype = llsa.BF16  # Delta and a number per entry
    assert llsa.llsa_cross_bwd_workspace_bytes(d) >= 8 * 16 * 1024 * 4


@pytest.mark.parametrize("scale", [2.0**-121, 1e-38, 1e-45])
def test_cross_bf16_backward_refuses_scales_that_lse_cannot_be_divided_by(scale):
    d = desc()
    d.sm_scale = scale
    assert 0 < d.sm_scale < 2.0**-120
    assert cross("bwd", d) == llsa.ERR_UNSUPPORTED


def test_binding_refuses_a_library_without_its_calls(monkeypatch):
    """A library built before a call was added has the same version: the
    binding names what is missing."""
    import _ctypes  # any shared object that is not this library

    monkeypatch.setattr(llsa, "_lib", None)
    monkeypatch.setattr(llsa, "LIB_PATH", _ctypes.__file__)
    with pytest.raises(llsa.LlsaError, match="llsa_cross_attn_bwd.*rebuild"):
        llsa.lib()
