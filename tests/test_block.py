"""A run of the operators as a layer uses them: norm with residual, 8-bit in-projection, mixer, 8-bit
out-projection, for prompts and single tokens (block.MixerBlock)."""
import pytest
import torch

import linear_attention_layer_causal_b200 as gdn
import ops_ref as ref
from linear_attention_layer_causal_b200 import block as B

HIDDEN = 256


def make(mixer, seed, out_norm=False, dev="cuda"):
    g = torch.Generator().manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g)
    rows = sum(n for _, n in B.in_projection_rows(mixer))
    ssm = isinstance(mixer, gdn.SsmConfig)
    H, C = (mixer.num_heads, mixer.conv_dim) if ssm else (mixer.num_v_heads, mixer.conv_dim)
    width = H * mixer.head_dim
    in_w, in_s = ref.quant(randn(rows, HIDDEN) / HIDDEN ** 0.5, 128)
    out_w, out_s = ref.quant(randn(HIDDEN, width) / width ** 0.5, 128)
    p = dict(conv_w=0.5 * randn(C, 4), A_log=torch.log(1 + 15 * torch.rand(H, generator=g)), dt_bias=randn(H) - 2)
    p |= dict(D=1 + 0.1 * randn(H), conv_b=0.1 * randn(C)) if ssm else dict(norm_w=1 + 0.1 * randn(mixer.head_dim))
    blk = B.MixerBlock(mixer, 0.1 * randn(HIDDEN).to(dev), in_w.to(dev), in_s.to(dev), out_w.to(dev), out_s.to(dev),
                       {k: v.to(dev) for k, v in p.items()}, weight_offset=1.0,
                       out_norm_w=1 + 0.1 * randn(width).to(dev) if out_norm else None)
    return blk, randn


MIXERS = [(gdn.SsmConfig(2, 8, 64, 64), True), (gdn.SsmConfig(1, 3, 64, 128), False), (gdn.SsmConfig(1, 2, 128, 64), False),
          (gdn.Config(2, 4, 128), False)]


@pytest.mark.gpu
@pytest.mark.parametrize("mixer,out_norm", MIXERS)
def test_prompt_then_tokens_continue_it(mixer, out_norm):
    """13 tokens as a prompt and three single ones give what a prompt of 16 gives.  A product's row
    has the same bits at every row count up to 16 (one kernel, one split of k), so the inputs of the
    mixer are equal; its two forms round differently in float32, which may move a rounding to
    bfloat16 and then one to e4m3: at most a step, 2^-3, of an element of a row, so 2^-3 in the
    2-norm (it is some 1e-3)."""
    blk, randn = make(mixer, 3, out_norm)
    x, r = randn(16, HIDDEN).bfloat16().cuda(), randn(16, HIDDEN).bfloat16().cuda()

    def cu(n):
        return torch.tensor([0, n], dtype=torch.int32, device="cuda")
    whole, whole_r, whole_s, whole_c = blk.prefill(x, r, cu(16))
    out, res, state, conv = blk.prefill(x[:13].contiguous(), r[:13].contiguous(), cu(13))
    outs, ress = [out], [res]
    for t in range(13, 16):
        o, q = blk.decode(x[t:t + 1].contiguous(), r[t:t + 1].contiguous(), state, conv)
        outs.append(o)
        ress.append(q)
    assert torch.equal(torch.cat(ress), whole_r)
    assert torch.equal(whole_r, (x.float() + r.float()).bfloat16())
    assert torch.equal(conv, whole_c)
    got, want = torch.cat(outs).double(), whole.double()
    assert float((got - want).norm() / want.norm()) <= 2.0 ** -3
    assert float((state.double() - whole_s.double()).norm() / whole_s.double().norm()) <= 1e-2


@pytest.mark.gpu
@pytest.mark.parametrize("mixer,out_norm", MIXERS)
def test_steps_against_their_definitions(mixer, out_norm):
    """Every step of a ragged batch against its 64-bit definition on the inputs that it got."""
    blk, randn = make(mixer, 5, out_norm)
    lens = [70, 1, 0, 130]
    N = sum(lens)
    x = randn(N, HIDDEN).bfloat16().cuda()
    cu = torch.tensor([0, 70, 71, 71, 201], dtype=torch.int32, device="cuda")
    hidden, residual, state, conv = blk.prefill(x, None, cu)
    assert residual is x  # the first layer: nothing to add
    n = gdn.rmsnorm_fp8(x, blk.norm_w, weight_offset=1.0)
    e = ref.norm(x, blk.norm_w, offset=1.0)
    deq = n["q"].double() * ref.widen(n["scale"].double(), HIDDEN)
    assert float(((deq - e["v"]).abs() - (2.0 ** -4 + 2.0 ** -19) * e["v"].abs()
                  - 2.0 ** -10 * ref.widen(e["scale"], HIDDEN)).max()) <= 0
    rows = gdn.matmul_fp8(n["q"], n["scale"], blk.in_w, blk.in_scale)
    p, mag = ref.product(n["q"], n["scale"], blk.in_w, blk.in_scale)
    assert float(((rows.double() - p).abs() - 2.0 ** -8 * p.abs() - 140 * 2.0 ** -23 * mag).max()) <= 0
    if isinstance(mixer, gdn.SsmConfig):
        i = blk._inputs([rows])
        w = blk.params
        m = ref.ssm(mixer, i["xbc"], i["dt"], lens, w["conv_w"], w["A_log"], w["conv_b"], w["dt_bias"], w["D"], i["z"])
        assert float((state.double() - m["state"]).norm() / m["state"].norm()) <= 3 * 2.0 ** -18 + 2.0 ** -20
        assert torch.equal(conv, m["conv"])
        y = m["y"].reshape(N, -1)
        v = ref.norm(y, blk.out_norm_w, groups=mixer.num_groups)["v"] if out_norm else y
        wide = blk.out_w.double() * ref.widen(blk.out_scale.double().repeat_interleave(128, 0)[:HIDDEN], y.shape[1])
        # y's rounding to bfloat16 and its quantisation leave (2^-8 + 2^-4) of an element, and 2^-10 of its scale
        err = (2.0 ** -4 + 2.0 ** -7) * v.abs() + 2.0 ** -9 * ref.widen(ref.block_scale(v), y.shape[1])
        want = v @ wide.T
        assert float(((hidden.double() - want).abs() - err @ wide.abs().T - 2.0 ** -7 * want.abs()).max()) <= 0


@pytest.mark.gpu
def test_decode_of_a_layer_in_a_graph():
    """The whole single-token layer captured once and replayed on new inputs."""
    mixer = gdn.SsmConfig(2, 8, 64, 64)
    blk, randn = make(mixer, 8, True)
    x, r = torch.empty(5, HIDDEN, dtype=torch.bfloat16, device="cuda"), torch.empty(5, HIDDEN, dtype=torch.bfloat16, device="cuda")
    state, conv = torch.zeros(5, 8, 64, 64, device="cuda"), torch.zeros(5, 3, mixer.conv_dim, dtype=torch.bfloat16, device="cuda")
    x.normal_(), r.normal_()
    blk.decode(x, r, state, conv)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, res = blk.decode(x, r, state, conv)
    for t in range(3):
        x.copy_(randn(5, HIDDEN)), r.copy_(randn(5, HIDDEN))
        s0, c0 = state.clone(), conv.clone()
        g.replay()
        torch.cuda.synchronize()
        s1, c1 = s0.clone(), c0.clone()
        o, q = blk.decode(x, r, s1, c1)
        assert torch.equal(out, o) and torch.equal(res, q) and torch.equal(state, s1) and torch.equal(conv, c1)


def test_refusals():
    mixer = gdn.SsmConfig(2, 6, 64, 64)
    rows = sum(n for _, n in B.in_projection_rows(mixer))
    assert rows % 128 == 0 and rows >= 6 * 64 + mixer.conv_dim + 6
    w = torch.zeros(rows, HIDDEN, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="rows"):
        B.MixerBlock(mixer, None, w[:-1], None, None, None, {})
    with pytest.raises(ValueError, match="bfloat16"):
        B.MixerBlock(gdn.SsmConfig(2, 6, 64, 64, act_dtype="f32"), None, w, None, None, None, {})
