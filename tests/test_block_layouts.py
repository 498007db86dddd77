"""MixerBlock's row layout for every mixer, its refusals, and its run around Gated DeltaNet against the
definitions: the parts of the in-projection from the documented rows of in_w in 64 bits, the mixer
against the oracle, the out-projection from the mixer's output in 64 bits."""
import pytest
import torch

import linear_attention_layer_causal_b200 as gdn
import oracle
import ops_ref as ref
from linear_attention_layer_causal_b200 import block as B
from parity_util import assert_output_close, assert_state_close
from test_block import HIDDEN, make

GDN = [(gdn.Config(2, 4, 128), False), (gdn.Config(1, 1, 32), False), (gdn.Config(2, 6, 32), True), (gdn.Config(1, 3, 32), False),
       (gdn.Config(1, 5, 128), True), (gdn.Config(4, 4, 32), False)]
SSM = [(gdn.SsmConfig(2, 8, 64, 64), True), (gdn.SsmConfig(1, 3, 64, 128), False), (gdn.SsmConfig(1, 1, 64, 64), False)]


def parts_of(mixer):
    """name -> (first row, rows) of in_w, as in_projection_rows() lists the parts."""
    at, first = 0, {}
    for name, rows in B.in_projection_rows(mixer):
        first[name] = at
        at += rows
    if isinstance(mixer, gdn.SsmConfig):
        hp = mixer.num_heads * mixer.head_dim
        return {"z": (0, hp), "xbc": (hp, mixer.conv_dim), "dt": (hp + mixer.conv_dim, mixer.num_heads)}
    h = mixer.num_v_heads
    return {"qkv": (first["qkv"], mixer.conv_dim), "z": (first["z"], h * mixer.head_dim), "a": (first["a|b"], h), "b": (first["a|b"] + h, h)}


@pytest.mark.parametrize("mixer,_", GDN + SSM)
def test_every_part_is_whole_blocks(mixer, _):
    """A part's scales are rows of in_scale of its own."""
    at = 0
    for name, rows in B.in_projection_rows(mixer):
        assert rows > 0 and rows % 128 == 0, name
        at += rows
    ends = sorted((a, a + n) for a, n in parts_of(mixer).values())
    assert ends[-1][1] <= at and all(a[1] <= b[0] for a, b in zip(ends, ends[1:]))


@pytest.mark.parametrize("mixer", [gdn.Config(2, 6, 32), gdn.SsmConfig(2, 6, 64, 64)])
def test_wrong_shapes_are_refused_when_the_layer_is_made(mixer):
    blk, _ = make(mixer, 1, True, dev="cpu")
    good = dict(mixer=mixer, norm_w=blk.norm_w, in_w=blk.in_w, in_scale=blk.in_scale, out_w=blk.out_w, out_scale=blk.out_scale,
                params=blk.params, out_norm_w=blk.out_norm_w)
    B.MixerBlock(**good)
    B.MixerBlock(**{**good, "out_norm_w": None})
    for name in ("norm_w", "in_scale", "out_w", "out_scale", "out_norm_w"):
        with pytest.raises(ValueError, match=name):
            B.MixerBlock(**{**good, name: good[name][:-1]})
        if name != "out_norm_w":
            with pytest.raises(ValueError, match=name):
                B.MixerBlock(**{**good, name: None})
    with pytest.raises(ValueError, match="in_scale"):
        B.MixerBlock(**{**good, "in_scale": good["in_scale"][:, :-1]})
    with pytest.raises(ValueError, match="out_w"):
        B.MixerBlock(**{**good, "out_w": good["out_w"][:, :-16]})


def check_parts(blk, x, residual):
    """The mixer's inputs, each element against the 64-bit product of the documented rows."""
    n = gdn.rmsnorm_fp8(x, blk.norm_w, residual=residual, eps=blk.eps, weight_offset=blk.weight_offset)
    p, mag = ref.product(n["q"], n["scale"], blk.in_w, blk.in_scale)
    i = blk._inputs(blk._project(x, residual)[0])
    parts = parts_of(blk.mixer)
    assert set(i) == set(parts)
    for name, (at, rows) in parts.items():
        got, want = i[name].flatten(1).double(), p[:, at:at + rows]
        assert got.shape == want.shape
        assert float(((got - want).abs() - 2.0 ** -8 * want.abs() - 140 * 2.0 ** -23 * mag[:, at:at + rows]).max()) <= 0, name
    return i


def check_out(blk, y, hidden):
    """The layer's output from the mixer's output y: e4m3 keeps 2^-4 of an element and 2^-10 of its scale, a norm
    before it 2^-19; the product 140 roundings of 2^-23 and that to bfloat16."""
    v = y.flatten(1).double()
    if blk.out_norm_w is not None:
        v = ref.norm(y.flatten(1), blk.out_norm_w)["v"]
    w = blk.out_w.double() * ref.widen(blk.out_scale.double().repeat_interleave(128, 0)[:HIDDEN], v.shape[1])
    err = (2.0 ** -4 + 2.0 ** -18) * v.abs() + 2.0 ** -9 * ref.widen(ref.block_scale(v), v.shape[1])
    want = v @ w.T
    bound = (err + 140 * 2.0 ** -23 * v.abs()) @ w.abs().T
    assert float(((hidden.double() - want).abs() - (1 + 2.0 ** -8) * bound - 2.0 ** -8 * want.abs()).max()) <= 0
    # the errors are unlike each other: in the 2-norm half of the largest is left with room to spare
    assert float((hidden.double() - want).norm() / want.norm()) <= 2.0 ** -4


@pytest.mark.gpu
@pytest.mark.parametrize("mixer,out_norm", GDN)
def test_gated_deltanet_layer_against_its_definition(mixer, out_norm):
    blk, randn = make(mixer, 5, out_norm)
    shape = oracle.Shape(mixer.num_qk_heads, mixer.num_v_heads, mixer.head_dim, mixer.conv_kernel)
    lens = [70, 1, 0, 130]
    x, r = randn(201, HIDDEN).bfloat16().cuda(), randn(201, HIDDEN).bfloat16().cuda()
    cu = torch.tensor([0, 70, 71, 71, 201], dtype=torch.int32, device="cuda")
    hidden, residual, state, conv = blk.prefill(x, r, cu)
    assert torch.equal(residual, (x.float() + r.float()).bfloat16())
    i, w = check_parts(blk, x, r), blk.params
    par = [w[k] for k in ("conv_w", "A_log", "dt_bias", "norm_w")]
    e = oracle.prefill(shape, i["qkv"], i["a"], i["b"], i["z"], cu, *par)
    y = gdn.prefill(mixer, i["qkv"], i["a"], i["b"], i["z"], cu, **w)["y"]
    assert_output_close(y, e["y"])
    assert_state_close(state, e["state"])
    assert torch.equal(conv.double().cpu(), torch.from_numpy(e["conv_window"]))
    check_out(blk, y, hidden)

    # a token for each sequence
    x, r = randn(len(lens), HIDDEN).bfloat16().cuda(), randn(len(lens), HIDDEN).bfloat16().cuda()
    s0, c0 = state.clone(), conv.clone()
    hidden, residual = blk.decode(x, r, state, conv)
    i = check_parts(blk, x, r)
    e = oracle.decode(shape, i["qkv"], i["a"], i["b"], i["z"], *par, s0.cpu(), c0.cpu())
    s1, c1 = s0.clone(), c0.clone()
    y = gdn.decode(mixer, i["qkv"], i["a"], i["b"], i["z"], s1, c1, **w)
    assert_output_close(y, e["y"])
    assert torch.equal(state, s1) and torch.equal(conv, c1)
    assert_state_close(state, e["state"])
    check_out(blk, y, hidden)


@pytest.mark.gpu
@pytest.mark.parametrize("mixer,out_norm", SSM)
def test_state_space_layers_parts(mixer, out_norm):
    blk, randn = make(mixer, 6, out_norm)
    x = randn(75, HIDDEN).bfloat16().cuda()
    check_parts(blk, x, None)
    check_parts(blk, x, randn(75, HIDDEN).bfloat16().cuda())


@pytest.mark.gpu
@pytest.mark.parametrize("mixer,out_norm", SSM + GDN)
def test_prompt_and_tokens_agree(mixer, out_norm):
    """A prompt of 16 tokens against 13 and three single ones, in the 2-norm.  The mixer's inputs are equal.  Its two
    forms round differently: the state-space mixer's by some 2^-16, which moves one in 2^9 of y's values to the next
    bfloat16; where that is a block's largest, the block is quantised anew, and its values move by the e4m3 error of
    2^-5 in the mean.  A tenth of the blocks of a row so moved is 2^-6 of the whole, and not expected.  Gated
    DeltaNet's prompts are held to 2^-6.6 of its output (heads of 128 run in tf32), which may move every block: two
    e4m3 errors of 2^-5 that differ, below 2^-4."""
    blk, randn = make(mixer, 3, out_norm)
    x, r = randn(16, HIDDEN).bfloat16().cuda(), randn(16, HIDDEN).bfloat16().cuda()

    def cu(n):
        return torch.tensor([0, n], dtype=torch.int32, device="cuda")
    whole, _, whole_s, whole_c = blk.prefill(x, r, cu(16))
    out, _, state, conv = blk.prefill(x[:13].contiguous(), r[:13].contiguous(), cu(13))
    outs = [out]
    for t in range(13, 16):
        outs.append(blk.decode(x[t:t + 1].contiguous(), r[t:t + 1].contiguous(), state, conv)[0])
    got, want = torch.cat(outs).double(), whole.double()
    limit = 2.0 ** -6 if isinstance(mixer, gdn.SsmConfig) else 2.0 ** -4
    assert float((got - want).norm() / want.norm()) <= limit
    assert torch.equal(conv, whole_c)
    assert float((state.double() - whole_s.double()).norm() / whole_s.double().norm()) <= (2.0 ** -15 if isinstance(mixer, gdn.SsmConfig) else 1e-2)
