"""Cross attention on the GPU where its answer hangs on how the work is cut:
NaN among split keys, no states at all, items without rows for every tile."""

import math

import pytest
import torch

import block_testlib as bt
import hierarchical_top_sparse_llsa_b200 as llsa
from test_gpu_cross_attn import check, make, run

pytestmark = pytest.mark.gpu


# the keys in one piece, and split over the SMs
WHOLE_AND_SPLIT = [(1, 2, 2, 300, 40, 64), (1, 2, 2, 300, 40, 128), (1, 2, 1, 5, 3000, 64), (2, 4, 2, 3, 5000, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", WHOLE_AND_SPLIT, ids=str)
def test_nan_query_shows(shape, dtype):
    """A NaN query has scores that are all NaN: O and lse of its row are NaN,
    and no other row's are."""
    x = make(*shape, dtype, seed=41)
    clean = run(x, grads=False)
    x["q"][0, 1, 2, 3] = float("nan")
    out = run(x, grads=False)
    for n in ("o", "lse"):
        assert torch.isnan(out[n][0, 1, 2]).all(), n
        out[n][0, 1, 2] = clean[n][0, 1, 2]
        assert torch.equal(out[n], clean[n]), n
    # and its gradients
    out = run(x)
    assert torch.isnan(out["dq"][0, 1, 2]).all()
    out["dq"][0, 1, 2] = 0
    assert torch.isfinite(out["dq"]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", WHOLE_AND_SPLIT, ids=str)
def test_nan_keys_show(shape, dtype):
    """One NaN state that is seen reaches every query of its heads, also where
    it is the only one that its split of the keys sees."""
    B, H, Hkv, N, S, D = shape
    for at, hide in ((S // 2, False), (S - 1, True)):
        x = make(*shape, dtype, seed=42)
        mask = torch.ones(B, S, dtype=torch.uint8, device="cuda")
        if hide:  # the back half but for the last state
            mask[:, S // 2 : S - 1] = 0
        x["k"][0, 0, at, 5] = float("nan")
        out = run(x, None, mask, grads=False)
        heads = H // Hkv
        assert torch.isnan(out["o"][0, :heads]).all() and torch.isnan(out["lse"][0, :heads]).all()
        assert torch.isfinite(out["o"][0, heads:]).all() and torch.isfinite(out["o"][1:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hkv,N,D", [(1, 1, 1, 129, 64), (2, 6, 2, 1000, 64), (2, 4, 1, 43, 128), (1, 2, 2, 5000, 128),
                                         (1, 1, 1, 1, 64)])
def test_no_states_for_any_number_of_queries(B, H, Hkv, N, D, dtype):
    out = run(make(B, H, Hkv, N, 0, D, dtype, seed=43))
    assert (out["o"] == 0).all() and (out["lse"] == -math.inf).all() and (out["dq"] == 0).all()


# Items that have rows for one or two of the four query tiles (D = 64) come
# before items that have them all, at the start of a CTA's run too, with key
# tiles that fill the ring of slots exactly, nearly, or not
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("N", [520, 700, 1100])
@pytest.mark.parametrize("S", [40, 330, 384, 390])
def test_items_without_rows_for_every_tile(S, N, masked):
    x = make(6, 37, 37, N, S, 64, "bf16", seed=44)
    lens = mask = None
    if masked:
        g = torch.Generator(device="cuda").manual_seed(45)
        lens = torch.tensor([S, S - 1, S // 2, S, 1, S], dtype=torch.int32, device="cuda")
        mask = (torch.rand(6, S, generator=g, device="cuda") < 0.7).to(torch.uint8)
    a = run(x, lens, mask, grads=False)
    want = bt.cross(x["q"], x["k"], x["v"], lens, mask)
    for n in ("o", "lse"):
        bt.within(a[n], *want[n], n)
    for _ in range(3):
        b = run(x, lens, mask, grads=False)
        assert torch.equal(a["o"], b["o"]) and torch.equal(a["lse"], b["lse"])


def test_fp32_backward_without_a_workspace():
    shape = (8, 16, 16, 1024, 77, 64)
    x = make(*shape, "f32", seed=46)
    B, H, Hkv, N, S, D = shape
    d = llsa.make_cross(B, H, Hkv, N, S, D, llsa.F32)
    assert llsa.llsa_cross_fwd_workspace_bytes(d) == 0 and llsa.llsa_cross_bwd_workspace_bytes(d) == 0
    o, lse = torch.empty_like(x["q"]), torch.empty(B, H, N, device="cuda")
    g = {n: torch.empty_like(x[n]) for n in "qkv"}
    q, k, v, do = (x[n].data_ptr() for n in ("q", "k", "v", "do"))
    s = torch.cuda.current_stream().cuda_stream
    llsa.llsa_cross_attn_fwd(d, q, k, v, None, None, o.data_ptr(), None, lse.data_ptr(), None, 0, None, s)
    llsa.llsa_cross_attn_bwd(d, q, k, v, None, None, o.data_ptr(), None, lse.data_ptr(), do, g["q"].data_ptr(),
                             g["k"].data_ptr(), g["v"].data_ptr(), None, 0, None, s)
    torch.cuda.synchronize()
    want = bt.cross(x["q"], x["k"], x["v"], do=x["do"], bf16=False)
    for n, t in (("o", o), ("lse", lse), ("dq", g["q"]), ("dk", g["k"]), ("dv", g["v"])):
        bt.within(t, *want[n], n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [2.0**-120, 2.0**-40, 2.0**-10, 4.0])
def test_smallest_and_large_scales(scale, dtype):
    shape = (1, 2, 1, 150, 200, 64)
    x = make(*shape, dtype, seed=47)
    check(x, run(x, scale=scale), scale=scale)
