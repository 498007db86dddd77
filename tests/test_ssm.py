"""The selective state-space mixer (ssm_prefill, ssm_decode) against the token-by-token recurrence in
64 bits, and its refusals.

Tolerances.  A matrix product takes each float32 operand as two bfloat16 parts, which leave at most
2^-18 of it (half a step of the second part, itself at most half a step, 2^-9, of the first), and
drops the product of the two second parts, at most 2^-18: 3 * 2^-18 of every term.  A term passes
two such products at most on its way into y (state, then read-out) and is otherwise touched by
float32 roundings, float32 sums of up to 128 terms and the exponentials of a decay, together below
2^-16 of the sum of the absolute terms: 2^-15 of the magnitude bounds an element.  The errors of
the terms are unlike each other, so that in the 2-norm an output is held to 3 * 2^-18 + 2^-20 of it.
A bfloat16 y is rounded once more, by at most 2^-8 of each value and so of the 2-norm.
"""
import ctypes

import pytest
import torch

import linear_attention_layer_causal_b200 as gdn
import ops_ref as ref

L2 = 3 * 2.0 ** -18 + 2.0 ** -20
ELEM = 2.0 ** -15
ACT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(cfg, lens, seed, *, wide=False, gate=True, init=True, extras=True, dt_shift=0.0, dev="cuda"):
    """Inputs of one call as a dict of keyword arguments (rows that are slices of wider ones when wide)."""
    g = torch.Generator().manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g).to(dev)
    H, P, S, C = cfg.num_heads, cfg.head_dim, cfg.state_dim, cfg.conv_dim
    N, B, act = sum(lens), len(lens), ACT[cfg.act_dtype]
    if wide:
        proj = randn(N, H * P + C + -(-H // 8) * 8 + 16).to(act)
        z, xbc, dt = proj[:, :H * P].unflatten(1, (H, P)), proj[:, H * P:H * P + C], proj[:, H * P + C:H * P + C + H]
    else:
        z, xbc, dt = randn(N, H, P).to(act), randn(N, C).to(act), randn(N, H).to(act)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    d = dict(xbc=xbc, dt=(dt.float() + dt_shift).to(act) if dt_shift else dt, conv_w=0.5 * randn(C, 4),
             A_log=torch.log(1 + 15 * torch.rand(H, generator=g)).to(dev), z=z if gate else None,
             initial_state=0.1 * randn(B, H, P, S) if init else None,
             initial_conv=randn(B, 3, C).to(act) if init else None)
    if extras:
        d.update(conv_b=0.1 * randn(C), dt_bias=randn(H) - 3, D=1 + 0.1 * randn(H))
    return d, torch.tensor(cu, dtype=torch.int32, device=dev)


def want(cfg, d, lens):
    return ref.ssm(cfg, d["xbc"], d["dt"], lens, d["conv_w"], d["A_log"], d.get("conv_b"), d.get("dt_bias"),
                   d.get("D"), d["z"], d["initial_state"], d["initial_conv"])


def prefill(cfg, d, cu, **kw):
    a = {k: v for k, v in d.items() if k not in ("xbc", "dt", "conv_w", "A_log")}
    return gdn.ssm_prefill(cfg, d["xbc"], d["dt"], cu, d["conv_w"], d["A_log"], **{**a, **kw})


def near(got, exact, mag, what, skip=None):
    g, e = got.double(), exact
    if e.numel() == 0:
        return
    assert torch.isfinite(g).all(), f"{what}: not finite"
    step = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    over = (g - e).abs() - (ELEM * mag + step * e.abs())
    assert float(over.max()) <= 0, f"{what}: an element is {float(over.max()):.2e} over its bound"
    rel = float((g - e).norm() / e.norm().clamp(min=1e-300))
    limit = L2 + step
    assert rel <= limit, f"{what}: {rel:.2e} in the 2-norm, {limit:.2e} allowed"


def check(cfg, d, lens, out):
    e = want(cfg, d, lens)
    near(out["y"], e["y"], e["y_mag"], "y")
    if "final_state" in out:
        near(out["final_state"], e["state"], e["state_mag"], "final state")
    if "final_conv" in out:
        assert torch.equal(out["final_conv"], e["conv"])


CASES = [
    # lens, H, G, P, S, dtype, gate, init, extras, wide
    ([1], 1, 1, 64, 64, "f32", True, False, True, False),
    ([2], 2, 1, 64, 128, "bf16", True, True, True, True),
    ([3], 3, 1, 64, 64, "f32", False, True, False, False),
    ([63], 4, 2, 64, 128, "f32", True, True, True, True),
    ([64], 2, 2, 128, 128, "f32", True, False, True, False),
    ([65], 3, 3, 128, 64, "bf16", False, True, True, True),
    ([130, 0, 1, 64, 257], 5, 1, 64, 64, "f32", True, True, True, True),
    ([0, 17, 0, 0, 80, 0], 6, 2, 64, 128, "f32", True, True, True, False),
    ([500], 3, 1, 128, 128, "f32", True, True, True, False),
    ([15, 16, 17, 31, 32, 33, 47, 48, 49], 2, 1, 64, 64, "f32", True, True, False, True),
    ([700, 90], 9, 3, 64, 128, "bf16", True, True, True, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,G,P,S,dtype,gate,init,extras,wide", CASES)
def test_prefill(lens, H, G, P, S, dtype, gate, init, extras, wide):
    cfg = gdn.SsmConfig(G, H, P, S, act_dtype=dtype)
    d, cu = make(cfg, lens, 100 + H + sum(lens), gate=gate, init=init, extras=extras, wide=wide)
    check(cfg, d, lens, prefill(cfg, d, cu, return_final_state=True, return_final_conv=True))


@pytest.mark.gpu
@pytest.mark.parametrize("segments", [1, 2, 3, 16])
@pytest.mark.parametrize("S", [64, 128])
def test_prefill_in_segments(segments, S):
    """Any number of segments gives the same results, sequences shorter than the cut among them."""
    lens = [600, 0, 1, 65, 129]
    cfg = gdn.SsmConfig(1, 3, 64, S, act_dtype="f32", segments=segments)
    d, cu = make(cfg, lens, 7, wide=True)
    check(cfg, d, lens, prefill(cfg, d, cu, return_final_state=True, return_final_conv=True))


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [-12.0, 6.0, 60.0])
def test_prefill_decay_extremes(shift):
    """Heads that forget nothing over the sequence, and heads that forget all within a token."""
    cfg = gdn.SsmConfig(1, 2, 64, 64, act_dtype="f32")
    d, cu = make(cfg, [300], 11, dt_shift=shift)
    check(cfg, d, [300], prefill(cfg, d, cu, return_final_state=True))


@pytest.mark.gpu
def test_step_length_is_clamped():
    cfg = gdn.SsmConfig(1, 2, 64, 64, act_dtype="f32", dt_min=0.02, dt_max=0.05)
    d, cu = make(cfg, [150], 12)
    check(cfg, d, [150], prefill(cfg, d, cu, return_final_state=True))


@pytest.mark.gpu
def test_prefill_large_and_small_values():
    """States near 1e30 and inputs near 1e-20 in one call: nothing overflows on the way."""
    cfg = gdn.SsmConfig(2, 4, 64, 64, act_dtype="f32")
    d, cu = make(cfg, [100, 70], 13, gate=False)
    d["initial_state"][0] *= 1e30
    d["xbc"][100:] *= 1e-20
    d["initial_conv"][1] *= 1e-20
    d["conv_b"] = None
    out = prefill(cfg, d, cu, return_final_state=True)
    e = want(cfg, d, [100, 70])
    for n, (a, b) in enumerate(((0, 100), (100, 170))):
        near(out["y"][a:b], e["y"][a:b], e["y_mag"][a:b], f"y {n}")
        near(out["final_state"][n], e["state"][n], e["state_mag"][n], f"state {n}")


@pytest.mark.gpu
def test_prefill_keeps_nan_in_its_sequence_and_head():
    cfg = gdn.SsmConfig(1, 3, 64, 64, act_dtype="f32")
    lens = [70, 90]
    d, cu = make(cfg, lens, 14)
    clean = prefill(cfg, d, cu, return_final_state=True)
    d["dt"][100, 1] = float("nan")  # sequence 1, token 30, head 1
    out = prefill(cfg, d, cu, return_final_state=True)
    assert torch.equal(out["y"][:70], clean["y"][:70])
    assert torch.equal(out["final_state"][0], clean["final_state"][0])
    for h in (0, 2):
        assert torch.equal(out["y"][:, h], clean["y"][:, h])
        assert torch.equal(out["final_state"][1, h], clean["final_state"][1, h])
    assert out["y"][100:, 1].isnan().all() and out["final_state"][1, 1].isnan().all()
    near(out["y"][70:100, 1], want(cfg, d, lens)["y"][70:100, 1],
         want(cfg, d, lens)["y_mag"][70:100, 1], "tokens before the NaN")


@pytest.mark.gpu
def test_prefill_in_place_and_rows_behind_the_last_sequence():
    cfg = gdn.SsmConfig(1, 2, 64, 128, act_dtype="f32")
    lens = [66, 2]
    d, cu = make(cfg, lens, 15)
    e = want(cfg, d, lens)
    N = 68
    pad = {k: torch.cat([d[k], torch.full((9, *d[k].shape[1:]), float("nan"), device="cuda")]) for k in ("xbc", "dt", "z")}
    y = torch.full((N + 9, 2, 64), 7.0, device="cuda")
    S0, C0 = d["initial_state"].clone(), d["initial_conv"].clone()
    out = prefill(cfg, {**d, **pad, "initial_state": S0, "initial_conv": C0}, cu, y=y, final_state=S0, final_conv=C0)
    assert out["final_state"] is S0 and out["final_conv"] is C0
    assert (y[N:] == 7.0).all()
    near(y[:N], e["y"], e["y_mag"], "y")
    near(S0, e["state"], e["state_mag"], "state")
    assert torch.equal(C0, e["conv"])


@pytest.mark.gpu
def test_no_tokens_pass_the_state_through():
    cfg = gdn.SsmConfig(1, 2, 64, 64)
    d, cu = make(cfg, [0, 0], 16)
    out = prefill(cfg, d, cu, return_final_state=True, return_final_conv=True)
    assert torch.equal(out["final_state"], d["initial_state"])
    assert torch.equal(out["final_conv"], d["initial_conv"])
    out = prefill(cfg, {**d, "initial_state": None, "initial_conv": None}, cu, return_final_state=True, return_final_conv=True)
    assert (out["final_state"] == 0).all() and (out["final_conv"] == 0).all()
    assert prefill(cfg, {**make(cfg, [], 16)[0]}, cu[:1])["y"].numel() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_in_two_pieces_and_decode_continue_it(dtype):
    cfg = gdn.SsmConfig(2, 6, 64, 128, act_dtype=dtype)
    d, cu = make(cfg, [200], 17)
    e = want(cfg, d, [200])
    first = {**d, **{k: d[k][:131] for k in ("xbc", "dt", "z")}}
    o = prefill(cfg, first, torch.tensor([0, 131], dtype=torch.int32, device="cuda"), return_final_state=True, return_final_conv=True)
    state, conv = o["final_state"], o["final_conv"]
    ys = [o["y"]]
    for a, b in ((131, 195),):
        piece = {**d, **{k: d[k][a:b] for k in ("xbc", "dt", "z")}, "initial_state": state, "initial_conv": conv}
        o = prefill(cfg, piece, torch.tensor([0, b - a], dtype=torch.int32, device="cuda"), final_state=state, final_conv=conv)
        ys.append(o["y"])
    for t in range(195, 200):
        ys.append(gdn.ssm_decode(cfg, d["xbc"][t:t + 1], d["dt"][t:t + 1], state, conv, d["conv_w"], d["A_log"],
                                 conv_b=d["conv_b"], dt_bias=d["dt_bias"], D=d["D"], z=d["z"][t:t + 1]))
    near(torch.cat(ys), e["y"], e["y_mag"], "y")
    near(state, e["state"], e["state_mag"], "state")
    assert torch.equal(conv, e["conv"])


@pytest.mark.gpu
@pytest.mark.parametrize("batch,H,G,P,S,dtype,gate,extras,wide", [
    (1, 1, 1, 64, 64, "f32", True, True, False),
    (3, 5, 1, 64, 128, "f32", True, True, True),
    (2, 6, 3, 128, 64, "bf16", False, True, True),
    (7, 3, 3, 128, 128, "f32", True, False, False),
    (200, 9, 1, 64, 128, "bf16", True, True, True),     # several units in a block, the last block shorter
    (130, 11, 1, 128, 64, "f32", True, True, True),
    (400, 4, 4, 64, 64, "bf16", True, True, False),     # one block per group: it advances every window
])
def test_decode(batch, H, G, P, S, dtype, gate, extras, wide):
    cfg = gdn.SsmConfig(G, H, P, S, act_dtype=dtype)
    d, _ = make(cfg, [1] * batch, 20 + batch, gate=gate, extras=extras, wide=wide)
    e = want(cfg, d, [1] * batch)
    state, conv = d["initial_state"].clone(), d["initial_conv"].clone()
    y = gdn.ssm_decode(cfg, d["xbc"], d["dt"], state, conv, d["conv_w"], d["A_log"], conv_b=d.get("conv_b"),
                       dt_bias=d.get("dt_bias"), D=d.get("D"), z=d["z"])
    near(y, e["y"], e["y_mag"], "y")
    near(state, e["state"], e["state_mag"], "state")
    assert torch.equal(conv, e["conv"])


@pytest.mark.gpu
def test_another_stream_and_graph_replays():
    """Two captured prefills with their own workspaces, replayed in turn and beside an eager call."""
    cfg = gdn.SsmConfig(1, 3, 64, 64, act_dtype="f32")
    sides = []
    s = torch.cuda.Stream()
    for seed, lens in ((30, [150, 20]), (31, [1, 90])):
        d, cu = make(cfg, lens, seed)
        ws = torch.empty(gdn.ssm_prefill_workspace_size(cfg, 2, sum(lens)), dtype=torch.uint8, device="cuda")
        y, st = torch.empty(sum(lens), 3, 64, device="cuda"), torch.empty(2, 3, 64, 64, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            prefill(cfg, d, cu, y=y, final_state=st, workspace=ws)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            prefill(cfg, d, cu, y=y, final_state=st, workspace=ws)
        sides.append((d, lens, y, st, g, (cu, ws)))  # a graph's operands have to live as long as it
    for _ in range(2):
        for d, lens, y, st, g, _kept in sides:
            y.zero_(), st.zero_()
            d["xbc"].mul_(0.5)  # new inputs in the captured buffers
            g.replay()
        torch.cuda.synchronize()
        for d, lens, y, st, g, _kept in sides:
            e = want(cfg, d, lens)
            near(y, e["y"], e["y_mag"], "replayed y")
            near(st, e["state"], e["state_mag"], "replayed state")


@pytest.mark.gpu
def test_decode_in_a_graph():
    cfg = gdn.SsmConfig(1, 40, 64, 128)
    d, _ = make(cfg, [1] * 5, 33)
    state, conv, y = d["initial_state"].clone(), d["initial_conv"].clone(), torch.empty(5, 40, 64, dtype=torch.bfloat16, device="cuda")

    def step():
        gdn.ssm_decode(cfg, d["xbc"], d["dt"], state, conv, d["conv_w"], d["A_log"], conv_b=d["conv_b"],
                       dt_bias=d["dt_bias"], D=d["D"], z=d["z"], y=y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    state.copy_(d["initial_state"]), conv.copy_(d["initial_conv"])
    now = {**d}
    for _ in range(3):
        e = want(cfg, now, [1] * 5)
        g.replay()
        torch.cuda.synchronize()
        near(y, e["y"], e["y_mag"], "y")
        near(state, e["state"], e["state_mag"], "state")
        assert torch.equal(conv, e["conv"])
        now = {**now, "initial_state": state.clone(), "initial_conv": conv.clone()}


def test_reference_matches_a_closed_form():
    """The tests' recurrence: one head, constant input, no conv history, geometric sum."""
    cfg = gdn.SsmConfig(1, 1, 64, 64, act_dtype="f32")
    w = torch.zeros(cfg.conv_dim, 4)
    w[:, 3] = 1
    xbc = torch.ones(9, cfg.conv_dim)
    e = ref.ssm(cfg, xbc, torch.zeros(9, 1), [9], w, torch.zeros(1))
    s, ln2 = 1 / (1 + torch.exp(torch.tensor(-1.0, dtype=torch.float64))), torch.log(torch.tensor(2.0, dtype=torch.float64))
    total = ln2 * s * s * sum(0.5 ** i for i in range(9))  # delta = ln 2, decay = 1/2
    assert torch.allclose(e["state"], total.expand(1, 1, 64, 64), rtol=1e-14)
    assert torch.allclose(e["y"][-1], (64 * total * s).expand(1, 64), rtol=1e-14)


# ---------------------------------------------------------------- refusals

def test_workspace_size_refusals():
    n = ctypes.c_size_t(0)

    def code(cfg, batch=1, N=10):
        return gdn.lib().gdn_ssm_prefill_workspace_size(ctypes.byref(cfg._c()), batch, N, ctypes.byref(n))
    C, I, U = gdn.SsmConfig, gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED
    assert code(C(1, 2, 64, 64)) == gdn.GDN_OK
    for bad in (C(0, 2, 64, 64), C(3, 4, 64, 64), C(1, 2, 64, 64, dt_min=-1.0), C(1, 2, 64, 64, dt_min=float("nan")),
                C(1, 2, 64, 64, dt_min=0.2, dt_max=0.1), C(1, 2, 64, 64, segments=-1), C(1, 2, 64, 64, segments=17)):
        assert code(bad) == I, bad
    for bad in (C(1, 2, 32, 64), C(1, 2, 64, 256), C(1, 2, 64, 64, conv_kernel=3), C(1, 20000, 64, 64)):
        assert code(bad) == U, bad
    assert code(C(1, 2, 64, 64), batch=-1) == I and code(C(1, 2, 64, 64), N=-1) == I
    assert code(C(1, 2, 64, 64), batch=0) == I and code(C(1, 2, 64, 64), N=1 << 31) == U
    assert gdn.ssm_prefill_workspace_size(C(1, 2, 64, 64), 3, 0) == 0


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="argument-error cases run only without a GPU")


@no_gpu
def test_abi_refusals():
    L, P = gdn.lib(), 1 << 20
    cfg = gdn.SsmConfig(1, 3, 64, 64)
    par = gdn._SsmParams(P, P, P, P, P)
    I, U, W = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_WORKSPACE
    C = cfg.conv_dim
    ok = dict(xbc=P, xs=C, dt=P, ds=3, z=P, zs=192, cu=P, batch=1, N=10, S0=P, C0=P, y=P, S1=P, C1=P, ws=P, wsb=1 << 30)

    def pre(par=par, cfg=cfg, **over):
        return L.gdn_ssm_prefill(ctypes.byref(cfg._c()), ctypes.byref(par), *{**ok, **over}.values(), None)
    for over in (dict(xbc=None), dict(dt=None), dict(y=None), dict(cu=None), dict(xbc=P + 8), dict(z=P + 8), dict(dt=P + 1),
                 dict(xs=C - 1), dict(xs=C + 4), dict(ds=2), dict(zs=191), dict(zs=196), dict(xs=1 << 40), dict(S0=P + 8),
                 dict(C0=P + 8), dict(S1=P + 4), dict(C1=P + 2), dict(batch=-1), dict(N=-1), dict(batch=0), dict(cu=P + 2)):
        assert pre(**over) == I, over
    assert pre(batch=70000) == U and pre(N=1 << 31) == U
    for over in (dict(ws=None), dict(wsb=100), dict(ws=P + 16)):
        assert pre(**over) == W, over
    assert pre(par=gdn._SsmParams(None, P, P, P, P)) == I and pre(par=gdn._SsmParams(P, P + 4, P, P, P)) == I
    assert pre(par=gdn._SsmParams(P, P, None, P, P)) == I
    dec = dict(xbc=P, xs=C, dt=P, ds=3, z=P, zs=192, state=P, conv=P, batch=2, y=P)

    def step(**over):
        return L.gdn_ssm_decode(ctypes.byref(cfg._c()), ctypes.byref(par), *{**dec, **over}.values(), None)
    for over in (dict(state=None), dict(conv=None), dict(state=P + 8), dict(batch=-1), dict(xbc=None), dict(xs=8)):
        assert step(**over) == I, over
    assert step(batch=70000) == U and step(batch=0) == gdn.GDN_OK


def test_binding_refuses_tensors_off_the_device():
    cfg = gdn.SsmConfig(1, 2, 64, 64, act_dtype="f32")
    d, cu = make(cfg, [4], 1, dev="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        prefill(cfg, d, cu)


@pytest.mark.gpu
def test_binding_refuses_wrong_shapes_types_and_strides():
    cfg = gdn.SsmConfig(1, 2, 64, 64, act_dtype="f32")
    d, cu = make(cfg, [4], 1)
    for key, bad in (("xbc", d["xbc"].bfloat16()), ("xbc", d["xbc"][:, :-8]), ("dt", d["dt"][:, :1]),
                     ("z", d["z"].transpose(1, 2).contiguous().transpose(1, 2)), ("conv_w", d["conv_w"][:-1]),
                     ("A_log", d["A_log"].double()), ("initial_state", d["initial_state"].transpose(2, 3)),
                     ("initial_conv", d["initial_conv"][:, :2]), ("D", d["D"].cpu())):
        with pytest.raises(ValueError):
            prefill(cfg, {**d, key: bad}, cu)
    with pytest.raises(ValueError):
        prefill(cfg, d, cu.long())
    with pytest.raises(gdn.GdnError):  # row strides that are no multiple of 16 bytes
        odd = torch.zeros(4, cfg.conv_dim + 1, device="cuda")[:, :-1]
        prefill(cfg, {**d, "xbc": odd}, cu)
    with pytest.raises(gdn.GdnError):
        prefill(cfg, d, cu, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("segments", [1, 4, 16])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_with_segments_and_short_sequences(segments, dtype):
    """States and windows advance in place, whichever segment has a short sequence's only chunk."""
    lens = [1, 64, 2, 130, 0, 3, 65, 700] + 24 * [1, 5]
    cfg = gdn.SsmConfig(2, 6, 64, 64, act_dtype=dtype, segments=segments)
    d, cu = make(cfg, lens, 40 + segments)
    e = want(cfg, d, lens)
    S0, C0 = d["initial_state"].clone(), d["initial_conv"].clone()
    out = prefill(cfg, {**d, "initial_state": S0, "initial_conv": C0}, cu, final_state=S0, final_conv=C0)
    near(out["y"], e["y"], e["y_mag"], "y")
    near(S0, e["state"], e["state_mag"], "state")
    assert torch.equal(C0, e["conv"])


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 37, 63, 64, 100])
def test_a_non_finite_channel_of_x_stays_in_its_row(at, value):
    """x of one channel and token is not finite: that channel's outputs from there on, and no others."""
    cfg = gdn.SsmConfig(1, 2, 64, 64, act_dtype="f32")
    d, cu = make(cfg, [150], 15, gate=False)
    clean = prefill(cfg, d, cu, return_final_state=True)
    xbc = d["xbc"].clone()
    xbc[at, 70] = value  # head 1, channel 6
    out = prefill(cfg, {**d, "xbc": xbc}, cu, return_final_state=True)
    others = [c for c in range(128) if c != 70]
    y, y0 = out["y"].flatten(1), clean["y"].flatten(1)
    assert torch.equal(y[:, others], y0[:, others])
    assert torch.equal(y[:at, 70], y0[:at, 70])
    assert not y[at:, 70].isfinite().any()
    S, S0 = out["final_state"].flatten(1, 2)[0], clean["final_state"].flatten(1, 2)[0]
    assert torch.equal(S[others], S0[others]) and not S[70].isfinite().any()


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["B", "C"])
def test_a_non_finite_column_of_b_or_c(which):
    """From a bad B on every output of its group; a bad C is read by four tokens and the state has no part of it."""
    cfg = gdn.SsmConfig(2, 4, 64, 64, act_dtype="f32")
    d, cu = make(cfg, [150], 17, gate=False)
    clean = prefill(cfg, d, cu, return_final_state=True)
    xbc, at = d["xbc"].clone(), 40
    xbc[at, 4 * 64 + (2 * 64 if which == "C" else 0) + 64 + 5] = float("nan")  # group 1, column 5
    out = prefill(cfg, {**d, "xbc": xbc}, cu, return_final_state=True)
    y, y0 = out["y"], clean["y"]
    end = at + 4 if which == "C" else 150
    assert torch.equal(y[:, :2], y0[:, :2])
    assert torch.equal(y[:at], y0[:at]) and torch.equal(y[end:], y0[end:])
    assert y[at:end, 2:].isnan().all()
    S, S0 = out["final_state"][0], clean["final_state"][0]
    if which == "C":
        assert torch.equal(S, S0)
    else:
        cols = [c for c in range(64) if c != 5]
        assert torch.equal(S[:2], S0[:2]) and torch.equal(S[2:, :, cols], S0[2:, :, cols])
        assert S[2:, :, 5].isnan().all()


@pytest.mark.gpu
def test_two_streams_at_once_without_given_workspaces():
    """Calls that overlap, each with a workspace of its own that is freed at once."""
    cfg = gdn.SsmConfig(1, 4, 64, 128, segments=4)
    lens = [900, 300]
    d, cu = make(cfg, lens, 18)
    d2, _ = make(cfg, lens, 19)
    one = prefill(cfg, d, cu, return_final_state=True)
    two = prefill(cfg, d2, cu, return_final_state=True)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(6):
        got.append((prefill(cfg, d, cu, return_final_state=True, stream=sa), one))
        got.append((prefill(cfg, d2, cu, return_final_state=True, stream=sb), two))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a["y"], b["y"]) and torch.equal(a["final_state"], b["final_state"])


@pytest.mark.gpu
def test_cu_seqlens_that_end_early_or_are_out_of_order():
    """Only the rows that some sequence has are written, and nothing outside the tensors is read."""
    cfg = gdn.SsmConfig(1, 2, 64, 64, act_dtype="f32")
    d, cu = make(cfg, [100, 50], 20)
    y = torch.full((150, 2, 64), 7.0, device="cuda")
    clean = prefill(cfg, d, cu)["y"]
    cu2 = torch.tensor([0, 100, 100], dtype=torch.int32, device="cuda")
    prefill(cfg, d, cu2, y=y)
    assert torch.equal(y[:100], clean[:100]) and (y[100:] == 7.0).all()
    y.fill_(7.0)
    cu2 = torch.tensor([0, 100, 1000], dtype=torch.int32, device="cuda")  # past the rows: the last one ends it
    prefill(cfg, d, cu2, y=y)
    assert torch.equal(y, clean)
    y.fill_(7.0)
    cu2 = torch.tensor([0, 100, 20], dtype=torch.int32, device="cuda")  # a negative length is none
    prefill(cfg, d, cu2, y=y)
    assert torch.equal(y[:100], clean[:100]) and (y[100:] == 7.0).all()


@pytest.mark.gpu
def test_status_words_are_clear_after_a_call():
    cfg = gdn.SsmConfig(1, 2, 64, 64)
    d, cu = make(cfg, [100], 21)
    need = gdn.ssm_prefill_workspace_size(cfg, 1, 100)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    prefill(cfg, d, cu, workspace=ws)
    torch.cuda.synchronize()
    assert (ws[:8] == 0).all()


@pytest.mark.gpu
def test_prefill_and_decode_past_32_bit_offsets():
    """Rows, outputs and states whose offsets pass 2^31 elements give what the same rows give alone."""
    cfg = gdn.SsmConfig(1, 128, 64, 64, segments=1)
    N, C = 262200, cfg.conv_dim
    total = N + 70
    assert total * 64 * 128 > 2 ** 31
    xbc = torch.zeros(total, C, dtype=torch.bfloat16, device="cuda")
    d, _ = make(cfg, [70], 23, init=False, gate=False)
    dt = torch.zeros(total, 128, dtype=torch.bfloat16, device="cuda")
    xbc[-70:], dt[-70:] = d["xbc"], d["dt"]
    cu = torch.tensor([0, N, total], dtype=torch.int32, device="cuda")
    out = prefill(cfg, {**d, "xbc": xbc, "dt": dt}, cu, return_final_state=True)
    alone = prefill(cfg, d, torch.tensor([0, 70], dtype=torch.int32, device="cuda"), return_final_state=True)
    assert torch.equal(out["y"][-70:], alone["y"])
    assert torch.equal(out["final_state"][1], alone["final_state"][0])
    del xbc, dt, out
    torch.cuda.empty_cache()

    B = 4200
    assert B * 128 * 64 * 64 > 2 ** 31
    state = torch.zeros(B, 128, 64, 64, device="cuda")
    state[-1] = alone["final_state"][0]
    conv = torch.zeros(B, 3, C, dtype=torch.bfloat16, device="cuda")
    xb = torch.zeros(B, C, dtype=torch.bfloat16, device="cuda")
    dt1 = torch.zeros(B, 128, dtype=torch.bfloat16, device="cuda")
    xb[-1], dt1[-1] = d["xbc"][0], d["dt"][0]
    kw = {k: d[k] for k in ("conv_b", "dt_bias", "D")}
    S1, C1 = state[-1:].clone(), conv[-1:].clone()
    y = gdn.ssm_decode(cfg, xb, dt1, state, conv, d["conv_w"], d["A_log"], **kw)
    y1 = gdn.ssm_decode(cfg, xb[-1:], dt1[-1:], S1, C1, d["conv_w"], d["A_log"], **kw)
    assert torch.equal(conv[-1:], C1)
    for a, b in ((state[-1], S1[0]), (y[-1].float(), y1[0].float())):
        assert float((a - b).norm()) <= 2.0 ** -8 * float(b.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("segments", [2, 7])
@pytest.mark.parametrize("P", [64, 128])
@pytest.mark.parametrize("S", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_segments_of_every_layout(dtype, S, P, segments):
    """Long segments (several chunks, so several buffers in use at once) of every kernel the library has."""
    lens = [1000, 70, 460]
    cfg = gdn.SsmConfig(2, 6, P, S, act_dtype=dtype, segments=segments)
    d, cu = make(cfg, lens, 30 + segments, wide=True)
    check(cfg, d, lens, prefill(cfg, d, cu, return_final_state=True, return_final_conv=True))


@pytest.mark.gpu
@pytest.mark.parametrize("segments", [1, 2])
def test_a_wait_that_runs_out_is_reported(segments):
    """With a bound of a few cycles on the waits between warps the call ends, says so, and the next one is whole."""
    cfg = gdn.SsmConfig(1, 2, 64, 64, act_dtype="f32", segments=segments)
    lens = [2000]
    d, cu = make(cfg, lens, 24)
    ws = torch.empty(gdn.ssm_prefill_workspace_size(cfg, 1, 2000), dtype=torch.uint8, device="cuda")
    clean = prefill(cfg, d, cu, workspace=ws, return_final_state=True)
    assert gdn.prefill_status(ws) == (gdn.GDN_OK, 0)
    gdn.wait_limit_next_call(100)
    prefill(cfg, d, cu, workspace=ws)
    assert gdn.prefill_status(ws)[0] == gdn.GDN_ERR_TIMEOUT
    again = prefill(cfg, d, cu, workspace=ws, return_final_state=True)
    assert gdn.prefill_status(ws) == (gdn.GDN_OK, 0)
    assert torch.equal(again["y"], clean["y"]) and torch.equal(again["final_state"], clean["final_state"])
