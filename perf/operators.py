"""What is measured of the operators around the sparse self-attention of a
conditioned transformer block: rotary positions (the cos/sin table, the
rotation and its adjoint, the rotation with the pooled pyramid) and cross
attention to an encoder's states (forward and backward).

Where `own` is false, run() computes an operator in plain torch; where it is
true, it makes the library's calls.  Tensors are contiguous
[B, H, tokens, D], tokens in Z-order, as everywhere in this library."""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_NONE, _LINEAR, _NTK, _YARN = 0, 1, 2, 3  # frequency scalings


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the table of a 256x256-pixel image: axial positions from the Z-order
        _table("table, 256x256 pixels, axial", rows=65536, rot=64, axes=2, given=False),
        # the table of a ragged batch far into a context stretched four times
        _table("table, far positions, YaRN", rows=1000, rot=128, scaling=_YARN, factor=4.0, orig_len=8192, span=32768),
        # Q and K of the 128x128-pixel workload before selection
        _rope("rotate Q and K, 128x128 pixels", B=2, H=12, N=16384, D=64, dtype="bf16", rot=64),
        # dQ and dK of a short odd sequence, half of each head rotated
        _rope("adjoint of dQ and dK, short", B=1, H=2, N=1023, D=64, dtype="f32", rot=32, interleaved=True, adjoint=True),
        # the headline workload: rotation and pyramid in front of the selection
        _pool("rotate and pool, 256x256 pixels", B=1, H=16, N=65536, D=64, L=3, dtype="bf16", rot=64),
        # the 32x32-pixel fp32 workload, interleaved pairs, part of the head
        _pool("rotate and pool, 32x32 pixels", B=1, H=2, N=1024, D=64, L=2, dtype="f32", rot=32, interleaved=True),
        # every pixel of a 256x256 image attends to a caption of 256 tokens
        _cross("cross forward, 256x256 pixels", "fwd", B=1, H=16, Hkv=16, N=65536, S=256, D=64, dtype="bf16"),
        # 128x128 pixels, captions of at most 77 tokens, padded and masked
        _cross("cross forward, padded captions", "fwd", B=2, H=12, Hkv=12, N=16384, S=77, D=64, dtype="bf16",
               ragged=True, mask=True),
        # a few query tokens read a long encoder sequence; shared key heads
        _cross("cross forward, few queries", "fwd", B=2, H=16, Hkv=4, N=17, S=20000, D=128, dtype="bf16"),
        # gradients of the large forward above
        _cross("cross backward, 256x256 pixels", "bwd", B=1, H=16, Hkv=16, N=65536, S=256, D=64, dtype="bf16"),
        # odd lengths, padded and masked keys, shared key heads
        _cross("cross backward, odd, shared heads", "bwd", B=2, H=8, Hkv=4, N=4095, S=333, D=128, dtype="bf16",
               ragged=True, mask=True),
        # a training step's two calls in fp32, at the 32x32-pixel workload
        _cross("cross step, fp32, 32x32 pixels", "step", B=1, H=2, Hkv=2, N=1024, S=77, D=64, dtype="f32"),
    ]


def _table(name=None, rows=1, rot=64, axes=1, given=True, scaling=_NONE, factor=1.0, orig_len=0, span=65536):
    c = dict(op="table", rows=rows, rot=rot, axes=axes, given=given, scaling=scaling, factor=factor,
             orig_len=orig_len, span=span)
    return dict(c, name=name) if name else c


def _rope(name=None, B=1, H=1, N=1, D=64, dtype="bf16", rot=64, interleaved=False, adjoint=False, per_batch=False):
    c = dict(op="rope", B=B, H=H, N=N, D=D, dtype=dtype, rot=rot, interleaved=interleaved, adjoint=adjoint,
             per_batch=per_batch)
    return dict(c, name=name) if name else c


def _pool(name=None, B=1, H=1, N=256, D=64, L=2, dtype="bf16", rot=64, interleaved=False):
    c = dict(op="rope_pool", B=B, H=H, N=N, D=D, L=L, dtype=dtype, rot=rot, interleaved=interleaved)
    return dict(c, name=name) if name else c


def _cross(name=None, which="fwd", B=1, H=1, Hkv=1, N=1, S=1, D=64, dtype="bf16", ragged=False, mask=False):
    c = dict(op="cross", which=which, B=B, H=H, Hkv=Hkv, N=N, S=S, D=D, dtype=dtype, ragged=ragged, mask=mask)
    return dict(c, name=name) if name else c


def _spread(rng, lo, hi):
    """A whole number whose logarithm is spread evenly."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("table", "rope", "rope", "rope_pool", "cross", "cross", "cross", "cross"))
    D = rng.choice((64, 128))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    rot = rng.choice((D, D, D // 2, 16, 24))
    interleaved = rng.random() < 0.5
    if op == "table":
        scaling = rng.choice((_NONE, _LINEAR, _NTK, _YARN))
        return _table(rows=_spread(rng, 200, 65536), rot=rot, axes=rng.choice((1, 2)) if rot % 4 == 0 else 1,
                      given=rng.random() < 0.6, scaling=scaling,
                      factor=1.0 if scaling == _NONE else rng.choice((2.0, 4.0, 7.5)),
                      orig_len=8192 if scaling == _YARN else 0, span=_spread(rng, 1024, 1 << 20))
    B, H = rng.randint(1, 4), rng.randint(1, 16)
    item = 2 if dtype == "bf16" else 4
    most = (1 << 27) // (B * H * D * item)  # tokens: 128 MiB a tensor
    if op == "rope":
        N = _spread(rng, 1, min(most, 65536))
        return _rope(B=B, H=H, N=N, D=D, dtype=dtype, rot=rot, interleaved=interleaved,
                     adjoint=rng.random() < 0.5, per_batch=rng.random() < 0.3)
    if op == "rope_pool":
        L = rng.choice((1, 2, 2, 3))
        N = 16**L * _spread(rng, 1, min(most, 65536) // 16**L)
        return _pool(B=B, H=H, N=N, D=D, L=L, dtype=dtype, rot=rot, interleaved=interleaved)
    Hkv = rng.choice((1, 2, 3, 4, 8))
    H = Hkv * rng.choice((1, 1, 2, 4))
    B = rng.randint(1, 3)
    which = rng.choice(("fwd", "fwd", "bwd", "step"))
    # query-key pairs of all heads, spread over a wide range, and a split of it
    pairs = math.exp(rng.uniform(math.log(1e3), math.log(9e7 if dtype == "bf16" else 2e7))) / (B * H)
    S = _spread(rng, 1, 20000 if rng.random() < 0.3 else 700)
    N = max(1, min(65536, (1 << 27) // (B * H * D * item), int(pairs / S)))
    return _cross(which=which, B=B, H=H, Hkv=Hkv, N=N, S=S, D=D, dtype=dtype, ragged=rng.random() < 0.5,
                  mask=rng.random() < 0.4)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _lens(case):
    """Valid keys of each batch entry: falling from S to about S / 2."""
    B, S = case["B"], case["S"]
    return [S - (b * S) // (2 * B) for b in range(B)] if case["ragged"] else [S] * B


def _zorder_xy(rows):
    """x (the even bits) and y (the odd bits) of Z-order tokens 0..rows-1."""
    t = torch.arange(rows, device="cuda")
    bits = torch.arange(16, device="cuda")
    x = (((t[:, None] >> (2 * bits)) & 1) << bits).sum(1)
    y = (((t[:, None] >> (2 * bits + 1)) & 1) << bits).sum(1)
    return torch.stack([x, y], 1)


def _positions(rows, axes):
    return torch.arange(rows, device="cuda")[:, None] if axes == 1 else _zorder_xy(rows)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "table":
        rows, axes = case["rows"], case["axes"]
        if case["given"]:  # runs of consecutive tokens from random starts
            start = torch.randint(0, case["span"], (1, axes), generator=g, device="cuda")
            step = torch.randint(0, 3, (rows, axes), generator=g, device="cuda")
            s["pos"] = (start + step.cumsum(0)).to(torch.int32).contiguous()
        # the plain fixed positions take nothing from the seed: the base does
        s["base"] = 10000.0 + float(torch.randint(0, 1000, (1,), generator=g, device="cuda"))
        s["table"] = torch.empty(rows, case["rot"] // 2, 2, device="cuda")
        return s
    t = _TYPES[case["dtype"]]
    B, H, N, D = case["B"], case["H"], case["N"], case["D"]
    if case["op"] in ("rope", "rope_pool"):
        # a projection's output: channels of unlike size around offsets
        chan = 0.5 + _randn(g, 2, 1, H, 1, D).abs()
        off = 0.3 * _randn(g, 2, 1, H, 1, D)
        s["q"], s["k"] = ((chan[i] * _randn(g, B, H, N, D) + off[i]).to(t) for i in (0, 1))
        axes = 2 if case["op"] == "rope_pool" and case["rot"] % 4 == 0 else 1
        rows = B * N if case.get("per_batch") else N
        pos = _positions(rows, axes)
        if axes == 1:  # a run of tokens somewhere in a context
            pos = pos + torch.randint(0, 100000, (1,), generator=g, device="cuda")
        s["rope_table"] = _plain_table(pos, case["rot"], axes, 10000.0, _NONE, 1.0, 0).float().contiguous()
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        if case["op"] == "rope_pool":
            s["v"] = _randn(g, B, H, N, D).to(t)
        return s
    Hkv, S = case["Hkv"], case["S"]
    s["q"] = (1.5 * _randn(g, B, H, N, D)).to(t)
    s["k"] = (_randn(g, B, Hkv, S, D) + 0.5 * _randn(g, B, Hkv, 1, D)).to(t)
    s["v"] = (_randn(g, B, Hkv, S, D) + 0.3 * _randn(g, B, Hkv, 1, D)).to(t)
    s["kv_len"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
    s["mask"] = (torch.rand(B, S, generator=g, device="cuda") < 0.9).to(torch.uint8) if case["mask"] else None
    s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(B, H, N, device="cuda")
    if case["which"] != "fwd":
        s["do"] = _randn(g, B, H, N, D).to(t)
        s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in ("q", "k", "v"))
    if case["which"] == "bwd":  # what the forward left
        o, s["lse"] = _plain_fwd(s)
        s["o"] = o.to(t)
    return s


# ------------------------------------------------------------- plain forms
def _inv_freq(n, base, scaling, factor, orig_len):
    """Frequencies of n pairs (64 bits): base^(-i/n), scaled."""
    i = torch.arange(n, device="cuda", dtype=torch.float64)
    if scaling == _NTK and n > 1:
        base = base * factor ** (n / (n - 1))
    f = torch.pow(torch.tensor(base, device="cuda", dtype=torch.float64), -i / n)
    if scaling == _LINEAR:
        f = f / factor
    if scaling == _YARN:
        # pairs that turn often within orig_len keep their frequency, pairs
        # that turn less than once are stretched, a ramp between
        lo = n * math.log(orig_len / (32.0 * 2 * math.pi)) / math.log(base)
        hi = n * math.log(orig_len / (1.0 * 2 * math.pi)) / math.log(base)
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), n - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
    return f


def _plain_table(pos, rot, axes, base, scaling, factor, orig_len):
    n = rot // 2 // axes
    f = _inv_freq(n, base, scaling, factor, orig_len)
    ang = (pos.double()[:, :, None] * f).reshape(pos.shape[0], rot // 2)
    m = 0.1 * math.log(factor) + 1.0 if scaling == _YARN else 1.0
    return torch.stack([ang.cos() * m, ang.sin() * m], -1)


def _rotate(x, table, rot, interleaved, adjoint):
    """The rotation in fp32: products and sums rounded one by one."""
    B, _, N, D = x.shape
    x = x.float()
    tab = table.view(-1, N, rot // 2, 2)[:, None]
    c, sn = tab[..., 0], tab[..., 1]
    if adjoint:
        sn = -sn
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
        y = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _means(x, L, first):
    """The pyramid of x: levels first..L, each the mean of 16 of the one below."""
    x = x.float()
    levels = [x := x.unflatten(2, (-1, 16)).mean(3) for _ in range(L)]
    return levels[first - 1 :]


def _valid(s):
    """bool [B, S]: the keys that may be attended to."""
    B, S = s["case"]["B"], s["case"]["S"]
    ok = torch.ones(B, S, dtype=torch.bool, device="cuda")
    if s["kv_len"] is not None:
        ok = ok & (torch.arange(S, device="cuda") < s["kv_len"][:, None])
    if s["mask"] is not None:
        ok = ok & (s["mask"] != 0)
    return ok


def _grouped(x, Hkv):
    return x.float().unflatten(1, (Hkv, -1))


def _plain_scores(s):
    """q . k / sqrt(D), -inf where masked: [B, Hkv, H / Hkv, N, S]."""
    c = s["case"]
    x = _grouped(s["q"], c["Hkv"]) @ s["k"].float()[:, :, None].transpose(-1, -2)
    return (x * (1.0 / math.sqrt(c["D"]))).masked_fill(~_valid(s)[:, None, None, None], -math.inf)


def _plain_fwd(s):
    x = _plain_scores(s)
    m = x.amax(-1, keepdim=True)
    m0 = m.masked_fill(m == -math.inf, 0.0)
    p = (x - m0).exp()
    l = p.sum(-1, keepdim=True)
    o = (p @ s["v"].float()[:, :, None]) / l.masked_fill(l == 0, 1.0)
    return o.flatten(1, 2), (m + l.log()).squeeze(-1).flatten(1, 2)


def _plain_bwd(s, lse):
    c = s["case"]
    Hkv, scale = c["Hkv"], 1.0 / math.sqrt(c["D"])
    q, do = _grouped(s["q"], Hkv), _grouped(s["do"], Hkv)
    k, v = s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    lse = lse.unflatten(1, (Hkv, -1))[..., None]
    p = (_plain_scores(s) - lse.masked_fill(lse == -math.inf, 0.0)).exp()
    dv = (p.transpose(-1, -2) @ do).sum(2)
    dp = do @ v.transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    dq = (ds @ k) * scale
    dk = (ds.transpose(-1, -2) @ q).sum(2) * scale
    return dq.flatten(1, 2), dk, dv


def _run_plain(s):
    c = s["case"]
    if c["op"] == "table":
        pos = s["pos"] if c["given"] else _positions(c["rows"], c["axes"])
        return _plain_table(pos, c["rot"], c["axes"], s["base"], c["scaling"], c["factor"], c["orig_len"]).float()
    t = _TYPES[c["dtype"]]
    if c["op"] == "rope":
        return [_rotate(s[x], s["rope_table"], c["rot"], c["interleaved"], c["adjoint"]).to(t) for x in ("q", "k")]
    if c["op"] == "rope_pool":
        q, k = (_rotate(s[x], s["rope_table"], c["rot"], c["interleaved"], False).to(t) for x in ("q", "k"))
        return {"q": q, "k": k, "pq": _means(q, c["L"], 1), "pk": _means(k, c["L"], 1), "pv": _means(s["v"], c["L"], 2)}
    if c["which"] == "fwd":
        o, lse = _plain_fwd(s)
        return {"o": o.to(t), "lse": lse}
    o, lse = (s["o"], s["lse"]) if c["which"] == "bwd" else _plain_fwd(s)
    dq, dk, dv = _plain_bwd(s, lse)
    out = {"dq": dq.to(t), "dk": dk.to(t), "dv": dv.to(t)}
    return out if c["which"] == "bwd" else dict(out, o=o.to(t), lse=lse)


# ------------------------------------------------------- the library's calls
def _ptr(t):
    return None if t is None else t.data_ptr()


def _beta_slow(c, base):
    """The turns at which the library's YaRN ramp ends where the plain form's
    does: at the last pair, if one turn (0: the default) lies past it."""
    if c["scaling"] != _YARN:
        return 0.0
    n = c["rot"] // 2 // c["axes"]
    past = n * math.log(c["orig_len"] / (2 * math.pi)) / math.log(base) > n - 1
    return c["orig_len"] / (2 * math.pi) * base ** (-(n - 1) / n) * (1 + 1e-9) if past else 0.0


def _plan(s):
    """The descriptors, buffers and workspaces that a program keeps."""
    import hierarchical_top_sparse_llsa_b200 as llsa

    c = s["case"]
    p = {"llsa": llsa}
    if c["op"] == "table":
        p["rope"] = llsa.make_rope(c["rot"], axes=c["axes"], base=s["base"], scaling=c["scaling"], factor=c["factor"],
                                   orig_len=c["orig_len"], beta_slow=_beta_slow(c, s["base"]))
        return p
    dtype = llsa.BF16 if c["dtype"] == "bf16" else llsa.F32
    if c["op"] in ("rope", "rope_pool"):
        layout = llsa.ROPE_INTERLEAVED if c["interleaved"] else llsa.ROPE_HALF
        p["rope"] = llsa.make_rope(c["rot"], layout=layout)
        p["dtype"] = dtype
        if c["op"] == "rope_pool":
            p["desc"] = llsa.make_desc(c["B"], c["H"], c["N"], c["D"], c["L"], 8, dtype)
            p["buf"] = llsa.LlsaBuffers(p["desc"], "cuda", with_bwd=False)
        return p
    p["desc"] = llsa.make_cross(c["B"], c["H"], c["Hkv"], c["N"], c["S"], c["D"], dtype)
    p["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    p["fwd_bytes"], p["bwd_bytes"] = (f(p["desc"]) for f in (llsa.llsa_cross_fwd_workspace_bytes,
                                                             llsa.llsa_cross_bwd_workspace_bytes))
    need = max(p["fwd_bytes"] if c["which"] != "bwd" else 0, p["bwd_bytes"] if c["which"] != "fwd" else 0, 1)
    p["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return p


def _run_own(s):
    if "plan" not in s:
        s["plan"] = _plan(s)
    c, p = s["case"], s["plan"]
    llsa, stream = p["llsa"], torch.cuda.current_stream().cuda_stream
    if c["op"] == "table":
        llsa.llsa_rope_table(p["rope"], c["rows"], _ptr(s.get("pos")), _ptr(s["table"]), stream)
        return s["table"]
    if c["op"] == "rope":
        llsa.llsa_rope(p["rope"], c["B"], c["H"], c["N"], c["D"], p["dtype"], _ptr(s["rope_table"]),
                       s["rope_table"].shape[0], _ptr(s["q"]), _ptr(s["k"]), _ptr(s["q_out"]), _ptr(s["k_out"]),
                       c["adjoint"], stream)
        return [s["q_out"], s["k_out"]]
    if c["op"] == "rope_pool":
        b, L = p["buf"], c["L"]
        llsa.llsa_rope_pool(p["desc"], p["rope"], _ptr(s["rope_table"]), s["rope_table"].shape[0], _ptr(s["q"]),
                            _ptr(s["k"]), _ptr(s["v"]), _ptr(s["q_out"]), _ptr(s["k_out"]), b.pyramid, stream)
        return {"q": s["q_out"], "k": s["k_out"], "pq": [b.pq[l] for l in range(1, L + 1)],
                "pk": [b.pk[l] for l in range(1, L + 1)], "pv": [b.pv[l] for l in range(2, L + 1)]}
    qkv = (_ptr(s["q"]), _ptr(s["k"]), _ptr(s["v"]), _ptr(s["kv_len"]), _ptr(s["mask"]))
    out = {}
    if c["which"] != "bwd":
        llsa.llsa_cross_attn_fwd(p["desc"], *qkv, _ptr(s["o"]), None, _ptr(s["lse"]), _ptr(p["ws"]), p["fwd_bytes"],
                                 _ptr(p["status"]), stream)
        out.update(o=s["o"], lse=s["lse"])
    if c["which"] != "fwd":
        llsa.llsa_cross_attn_bwd(p["desc"], *qkv, _ptr(s["o"]), None, _ptr(s["lse"]), _ptr(s["do"]), _ptr(s["dq"]),
                                 _ptr(s["dk"]), _ptr(s["dv"]), _ptr(p["ws"]), p["bwd_bytes"], _ptr(p["status"]), stream)
        out.update(dq=s["dq"], dk=s["dk"], dv=s["dv"])
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "table":
        out = c["rows"] * c["rot"] // 2
        return {"bytes": 8 * out + (4 * c["rows"] * c["axes"] if c["given"] else 0), "flops": 4 * out}
    e = 2 if c["dtype"] == "bf16" else 4
    B, H, N, D = c["B"], c["H"], c["N"], c["D"]
    x = B * H * N * D  # elements of Q
    if c["op"] in ("rope", "rope_pool"):
        rows = B * N if c.get("per_batch") else N
        table = rows * c["rot"] * 4
        if c["op"] == "rope":
            return {"bytes": 4 * x * e + table, "flops": 6 * B * H * N * c["rot"]}
        levels = sum(x // 16**l * 4 * (3 if l > 1 else 2) for l in range(1, c["L"] + 1))
        return {"bytes": 5 * x * e + table + levels, "flops": 6 * B * H * N * c["rot"] + 3 * x}
    keys = sum(_lens(c))
    kv = c["Hkv"] * keys * D
    side = B * H * N * 4 + (4 * B if c["ragged"] else 0) + (B * c["S"] if c["mask"] else 0)
    pairs = H * N * keys * D
    kv_all = B * c["Hkv"] * c["S"] * D
    fwd = {"bytes": (2 * x + 2 * kv) * e + side, "flops": 4 * pairs}
    bwd = {"bytes": (4 * x + 2 * kv + 2 * kv_all) * e + side, "flops": 10 * pairs}
    if c["which"] == "fwd":
        return fwd
    if c["which"] == "bwd":
        return bwd
    # a step reads q, k, v and dO once and writes o, lse and the gradients
    return {"bytes": (4 * x + 2 * kv + 2 * kv_all) * e + side, "flops": 14 * pairs}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "table":
        return _exact_table(s)
    if c["op"] in ("rope", "rope_pool"):
        return _exact_rope(s)
    return _exact_cross(s)


def _exact_table(s):
    c = s["case"]
    rows, axes, half = c["rows"], c["axes"], c["rot"] // 2
    n = half // axes
    if c["given"]:
        pos = s["pos"].double()
    elif axes == 1:
        pos = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None]
    else:
        xy = [[0, 0] for _ in range(rows)]
        for t in range(rows):
            for bit in range(t.bit_length()):
                xy[t][bit & 1] |= ((t >> bit) & 1) << (bit >> 1)
        pos = torch.tensor(xy, dtype=torch.float64, device="cuda")
    base, factor, freq = s["base"], c["factor"], []
    for i in range(n):
        if c["scaling"] == _NTK and n > 1:
            f = (base * factor ** (n / (n - 1.0))) ** (-float(i) / n)
        else:
            f = base ** (-float(i) / n)
        if c["scaling"] == _LINEAR:
            f = f / factor
        elif c["scaling"] == _YARN:
            # index of the pair that turns r times within orig_len positions
            at = [n * math.log(c["orig_len"] / (2 * math.pi * r), base) for r in (32.0, 1.0)]
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), n - 1)
            keep = 1.0 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f * keep + (f / factor) * (1.0 - keep)
        freq.append(f)
    out = torch.empty(rows, half, 2, dtype=torch.float64, device="cuda")
    m = 1.0 + 0.1 * math.log(factor) if c["scaling"] == _YARN else 1.0
    for a in range(axes):
        for i in range(n):
            ang = pos[:, a] * freq[i]
            out[:, a * n + i, 0] = torch.cos(ang) * m
            out[:, a * n + i, 1] = torch.sin(ang) * m
    return out


def _exact_rope(s):
    c = s["case"]
    B, H, N, D, rot = c["B"], c["H"], c["N"], c["D"], c["rot"]
    tab = s["rope_table"].double().view(-1, N, rot // 2, 2)
    z = torch.complex(tab[..., 0], tab[..., 1])  # a pair as a complex number, turned by z
    if c.get("adjoint"):
        z = z.conj()
    done = []
    for name in ("q", "k"):
        x = s[name].double()
        y = x.clone()
        first = slice(0, rot, 2) if c["interleaved"] else slice(0, rot // 2)
        second = slice(1, rot, 2) if c["interleaved"] else slice(rot // 2, rot)
        for h in range(H):
            w = torch.complex(x[:, h, :, first], x[:, h, :, second]) * z
            y[:, h, :, first], y[:, h, :, second] = w.real, w.imag
        done.append(y)
    if c["op"] == "rope":
        return done

    def pyramid(x, first):
        return [x.view(B, H, N // 16**l, 16**l, D).mean(3) for l in range(first, c["L"] + 1)]

    v = pyramid(s["v"].double(), 2)
    if c["dtype"] == "bf16":
        # levels of Q and K are means of stored, rounded values: 64 bits do
        # not settle which way a value next to a rounding border went
        none = [None] * c["L"]
        return {"q": done[0], "k": done[1], "pq": none, "pk": none, "pv": v}
    return {"q": done[0], "k": done[1], "pq": pyramid(done[0], 1), "pk": pyramid(done[1], 1), "pv": v}


def _exact_cross(s):
    c = s["case"]
    B, H, Hkv, N, S, D = (c[x] for x in ("B", "H", "Hkv", "N", "S", "D"))
    q, k, v = (s[x].double() for x in ("q", "k", "v"))
    o, lse = torch.zeros_like(q), torch.full((B, H, N), -math.inf, dtype=torch.float64, device="cuda")
    grads = c["which"] != "fwd"
    if grads:
        do = s["do"].double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b in range(B):
        keep = [j < (int(s["kv_len"][b]) if s["kv_len"] is not None else S) for j in range(S)]
        if s["mask"] is not None:
            keep = [a and m != 0 for a, m in zip(keep, s["mask"][b].tolist())]
        at = torch.tensor([j for j, a in enumerate(keep) if a], dtype=torch.long, device="cuda")
        if at.numel() == 0:
            continue
        for h in range(H):
            kh, vh = k[b, h // (H // Hkv), at], v[b, h // (H // Hkv), at]
            x = q[b, h] @ kh.T / D**0.5
            lse[b, h] = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[b, h][:, None])
            o[b, h] = p @ vh
            if grads:
                dp = do[b, h] @ vh.T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / D**0.5
                dq[b, h] = ds @ kh
                dk[b, h // (H // Hkv), at] += ds.T @ q[b, h]
                dv[b, h // (H // Hkv), at] += p.T @ do[b, h]
    if c["which"] == "fwd":
        return {"o": o, "lse": lse}
    out = {"dq": dq, "dk": dk, "dv": dv}
    return out if c["which"] == "bwd" else dict(out, o=o, lse=lse)
