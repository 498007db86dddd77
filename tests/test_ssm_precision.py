"""The state-space mixer's prompts keep float32's precision, in the state whatever the activations and in
y where they are float32, over the ranges that their scaled 16-bit parts have to cover.

Tolerances.  A product takes an operand as two float16 parts, whose sum is off by at most 2^-22 of it, and drops the
product of the two second parts, at most 2^-22: 3 * 2^-22 of a term, twice on its way into y.  The
SiLUs and the masks (approximate exponentials and reciprocals, exponents of up to 16 rounded to 2^-24
of them) add 2^-20 of a term each at most, and the tensor core's sums of 24 instructions 24 * 2^-23
of the sum of the magnitudes: together below 2^-17 of the magnitude for an element.  In the 2-norm
these errors, unlike each other, are held to 2^-20 of the output (a float32 recurrence has 2^-23).
A step length is a float32, off by 2^-23 of it, and the decay e^G over many tokens with it by |G|
2^-23, here as in any float32 form: the tests that look at strongly decayed values alone clamp the
step to a power of two.
"""
import pytest
import torch

import linear_attention_layer_causal_b200 as gdn
import ops_ref as ref
from test_ssm import make, prefill, want

L2, ELEM = 2.0 ** -20, 2.0 ** -17
LAYOUTS = [(1, 3, 64, 64), (2, 6, 64, 128), (1, 3, 128, 64), (2, 4, 128, 128)]


def near(got, exact, mag, what, norm=True):
    over = (got.double() - exact).abs() - ELEM * mag
    assert torch.isfinite(got).all() and float(over.max()) <= 0, f"{what}: an element is {float(over.max()):.2e} over its bound"
    rel = float((got.double() - exact).norm() / exact.norm().clamp(min=1e-300))
    assert not norm or rel <= L2, f"{what}: {rel:.2e} in the 2-norm"


def check(cfg, d, lens, norm=True, **kw):
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    out = prefill(cfg, d, cu, return_final_state=True, **kw)
    e = want(cfg, d, lens)
    near(out["final_state"], e["state"], e["state_mag"], "state", norm)
    if cfg.act_dtype == "f32":
        near(out["y"], e["y"], e["y_mag"], "y", norm)
    else:
        assert float((out["y"].double() - e["y"]).norm() / e["y"].norm()) <= 2.0 ** -8 + 3 * 2.0 ** -18
    return out, e


@pytest.mark.gpu
@pytest.mark.parametrize("G,H,P,S", LAYOUTS)
@pytest.mark.parametrize("segments", [1, 3])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_layout(G, H, P, S, segments, dtype):
    cfg = gdn.SsmConfig(G, H, P, S, act_dtype=dtype, segments=segments)
    lens = [600, 1, 67]
    d, _ = make(cfg, lens, 50 + segments, wide=True)
    check(cfg, d, lens)


@pytest.mark.gpu
@pytest.mark.parametrize("G,H,P,S", LAYOUTS)
@pytest.mark.parametrize("segments", [1, 2])
@pytest.mark.parametrize("token", [0, 5, 63, 64, 150])
@pytest.mark.parametrize("most", [1.0, 2.5])
def test_a_single_token_that_is_not_zero(G, H, P, S, segments, token, most):
    """Everything in the state is one token's share, decayed by up to e^-8 or e^-20 a chunk: as exact as a large one.  So
    is y, except that a mask (2^-15 of the largest, and a part of 2^-25) is held to 2^-39 of its chunk's largest, which
    shows where nothing else is left: 2^-34 of the channel's largest allows for chunks and channels unlike each other."""
    cfg = gdn.SsmConfig(G, H, P, S, act_dtype="f32", segments=segments, dt_min=0.125, dt_max=0.125)
    d, _ = make(cfg, [180], 60, gate=False, init=False, extras=False)
    d["A_log"] = torch.log(torch.linspace(0.05, most, H, device="cuda"))
    keep = torch.zeros(180, 1, device="cuda")
    keep[token] = 1
    d["xbc"][:, :H * P] *= keep
    out = prefill(cfg, d, torch.tensor([0, 180], dtype=torch.int32, device="cuda"), return_final_state=True)
    e = want(cfg, d, [180])
    near(out["final_state"], e["state"], e["state_mag"], "state", False)
    rel = (out["final_state"].double() - e["state"]).norm(dim=(2, 3)) / e["state"].norm(dim=(2, 3))
    assert float(rel.max()) <= 2 * L2
    near(out["y"], e["y"], e["y_mag"] + 2.0 ** -17 * e["y_mag"].amax(0, keepdim=True), "y")


@pytest.mark.gpu
@pytest.mark.parametrize("G,H,P,S", LAYOUTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("segments", [1, 2])
def test_rows_of_very_different_size(G, H, P, S, dtype, segments):
    """Channels of x from 1e-12 to 1e9 and rows of the initial state from 1e-20 to 1e20, each row for itself."""
    cfg = gdn.SsmConfig(G, H, P, S, act_dtype=dtype, segments=segments, dt_min=2.0 ** -5, dt_max=2.0 ** -5)
    d, _ = make(cfg, [150], 61, gate=False)
    d["conv_b"] = None
    g = torch.Generator().manual_seed(3)
    d["conv_w"][:H * P] *= torch.exp2(torch.randint(-40, 30, (H * P, 1), generator=g)).float().cuda()
    d["initial_state"] *= torch.exp2(torch.randint(-66, 66, (1, H, P, 1), generator=g)).float().cuda()
    out, e = check(cfg, d, [150], norm=False)
    rel = (out["final_state"].double() - e["state"]).norm(dim=-1) / e["state"].norm(dim=-1)
    assert float(rel.max()) <= 2 * L2, float(rel.max())  # each row's 2-norm has fewer terms to even out


@pytest.mark.gpu
@pytest.mark.parametrize("scale_b,scale_c", [(1e-12, 1.0), (1e9, 1e-9), (1e15, 1.0), (1e-18, 1e-18)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_small_and_large_b_and_c(scale_b, scale_c, dtype):
    cfg = gdn.SsmConfig(2, 4, 64, 128, act_dtype=dtype)
    d, _ = make(cfg, [130], 62, gate=False, init=False)
    d["conv_b"] = None
    HP, GS = 4 * 64, 2 * 128
    d["conv_w"][HP:HP + GS] *= scale_b
    d["conv_w"][HP + GS:] *= scale_c
    check(cfg, d, [130])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [None, 0.0, 1e-12, 1e6, 1e20])
@pytest.mark.parametrize("dt", [-200.0, -20.0, 3.0])
def test_skip_and_step_of_any_size(D, dt):
    """D of any size beside the masks, and steps from exactly zero (the state stays) to 3."""
    cfg = gdn.SsmConfig(1, 2, 64, 64, act_dtype="f32")
    d, _ = make(cfg, [100], 63)
    d["dt"] = torch.full_like(d["dt"], dt)
    d["dt_bias"] = None
    d["D"] = None if D is None else torch.full_like(d["D"], D)
    out, e = check(cfg, d, [100], norm=dt != 3.0)  # (of 3 only a few tokens are left, which even nothing out)
    if dt == -200.0:
        assert torch.equal(out["final_state"], d["initial_state"])


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["x", "B", "C", "all"])
def test_zeros(what):
    """Parts that are zero give zeros, not a division by their largest value."""
    cfg = gdn.SsmConfig(1, 3, 64, 64, act_dtype="f32")
    for init in (True, False):
        d, cu = make(cfg, [90], 64, init=init)
        d["conv_b"] = None
        lo, hi = {"x": (0, 192), "B": (192, 256), "C": (256, 320), "all": (0, 320)}[what]
        d["conv_w"][lo:hi] = 0
        out = prefill(cfg, d, cu, return_final_state=True)
        e = want(cfg, d, [90])
        near(out["final_state"], e["state"], e["state_mag"], "state", init)
        near(out["y"], e["y"], e["y_mag"], "y", False)


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("segments", [1, 2])
def test_a_state_that_is_not_finite_stays_in_its_row(value, segments):
    """Its column in the state, its row in y; the other columns of that row of the state keep their values."""
    cfg = gdn.SsmConfig(1, 2, 64, 64, act_dtype="f32", segments=segments)
    d, cu = make(cfg, [150], 65, gate=False)
    clean = prefill(cfg, d, cu, return_final_state=True)
    d["initial_state"][0, 1, 6, 9] = value
    out = prefill(cfg, d, cu, return_final_state=True)
    rows = [r for r in range(128) if r != 70]
    assert torch.equal(out["y"].flatten(1)[:, rows], clean["y"].flatten(1)[:, rows])
    assert not out["y"].flatten(1)[:64, 70].isfinite().any()
    S, S0 = out["final_state"].flatten(1, 2)[0], clean["final_state"].flatten(1, 2)[0]
    assert torch.equal(S[rows], S0[rows]) and not S[70, 9].isfinite()
    others = [c for c in range(64) if c != 9]
    assert float((S[70, others] - S0[70, others]).abs().max()) <= 2.0 ** -20 * float(S0[70].abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompts_and_tokens_leave_the_same_state(dtype):
    """The state after a prompt against the one that the same tokens leave one by one."""
    cfg = gdn.SsmConfig(1, 4, 64, 128, act_dtype=dtype)
    d, cu = make(cfg, [130], 66)
    whole = prefill(cfg, d, cu, return_final_state=True)
    state, conv = d["initial_state"].clone(), d["initial_conv"].clone()
    ys = [gdn.ssm_decode(cfg, d["xbc"][t:t + 1], d["dt"][t:t + 1], state, conv, d["conv_w"], d["A_log"], conv_b=d["conv_b"],
                         dt_bias=d["dt_bias"], D=d["D"], z=d["z"][t:t + 1]) for t in range(130)]
    assert float((state - whole["final_state"]).norm() / state.norm()) <= L2
    y = torch.cat(ys).float()
    limit = L2 if dtype == "f32" else 2.0 ** -8  # two roundings to bfloat16, of at most 2^-9 in the mean each
    assert float((y - whole["y"].float()).norm() / y.norm()) <= limit


@pytest.mark.gpu
def test_long_memory():
    """Steps of 1e-4: 5000 tokens that are all still there at the end, and cancel to a fiftieth of their magnitudes:
    errors of one sign do not, so that only the bound by the magnitudes holds."""
    cfg = gdn.SsmConfig(1, 2, 64, 64, act_dtype="f32")
    d, _ = make(cfg, [5000], 67, gate=False, init=False)
    d["dt"] = torch.full_like(d["dt"], -9.2)
    d["dt_bias"] = None
    check(cfg, d, [5000], norm=False)


@pytest.mark.gpu
def test_masks_and_skip_at_the_top_of_their_range():
    """C . B, the step and D all just below a power of two, so that each takes the most of what its scale allows and
    their sum twice that: still finite, and exact."""
    cfg = gdn.SsmConfig(1, 1, 64, 64, act_dtype="f32", dt_min=1.4426948, dt_max=1.4426948)  # times ln 2: 1 - 2^-22
    d, cu = make(cfg, [64], 68, gate=False, init=False, extras=False)
    top = 2.0 - 2.0 ** -20
    d["conv_w"].zero_()
    d["conv_w"][:, 3] = 1
    x = torch.linspace(1.0, 3.0, 4001, dtype=torch.float64)
    silu = x * torch.sigmoid(x)
    b = float(x[(silu - 1).abs().argmin()])  # SiLU(b) next to 1: 64 columns of 1 are 64, their neighbours below
    for shift in (-1e-3, -1e-4, 0.0, 1e-4, 1e-3):
        d["xbc"][:, 64:] = b + shift
        for D in (top, -top, 1.0, top * 2.0 ** -3, top * 2.0 ** 7):
            d["D"] = torch.full((1,), D, device="cuda")
            out = prefill(cfg, d, cu, return_final_state=True)
            e = want(cfg, d, [64])
            near(out["y"], e["y"], e["y_mag"], "y", False)
            near(out["final_state"], e["state"], e["state_mag"], "state", False)
