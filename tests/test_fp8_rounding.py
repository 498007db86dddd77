"""The 8-bit values of the norm and the plain quantisation, bit for bit: scale = max(amax / 448, 2^-126)
and q = e4m3(v / scale), both quotients rounded to float32 as IEEE division does.

The inputs are put where a neighbouring quotient shows: on ties of e4m3 (halfway between two of its
values) and next to them, under scales that are no powers of two.  Both sides compute the same
float32 operations, so nothing but equality is accepted.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

import linear_attention_layer_causal_b200 as gdn
import ops_ref as ref

# halfway points of e4m3: (2 k + 1) 2^-4 in each binade's steps of 2^-3, and of the subnormal steps of 2^-9
TIES = [m * 2.0 ** e for m in (17, 19, 21, 23, 25, 27, 29) for e in range(-10, 4)] + [k * 2.0 ** -10 for k in (1, 3, 5, 7, 9, 11, 13, 15)]


def expected(v):
    """(q, scale) of float32 rows v, by the definition in float32, on the CPU and by a tensor: a quotient by a
    Python number may be computed as a product with its reciprocal."""
    v = v.cpu()
    dim = v.shape[1]
    amax = torch.stack([v[:, i:i + 128].abs().amax(1) for i in range(0, dim, 128)], 1)
    scale = (amax / torch.full_like(amax, 448.0)).clamp(min=ref.TINY)
    quotient = v / ref.widen(scale, dim)
    return quotient.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def tie_rows(rows, dim, seed):
    """Each block's largest element is any float32, the others are ties times its scale or the floats beside them."""
    g = torch.Generator().manual_seed(seed)
    v = torch.empty(rows, dim)
    ties = torch.tensor(TIES)
    for i in range(0, dim, 128):
        n = min(128, dim - i)
        amax = torch.exp2(torch.empty(rows, 1).uniform_(-20, 20, generator=g))
        scale = amax / torch.full_like(amax, 448.0)
        t = ties[torch.randint(len(TIES), (rows, n), generator=g)] * (1 - 2.0 * torch.randint(0, 2, (rows, n), generator=g))
        near = (t * scale)
        step = torch.randint(-1, 2, (rows, n), generator=g)
        near = torch.where(step > 0, torch.nextafter(near, torch.tensor(float("inf"))),
                           torch.where(step < 0, torch.nextafter(near, torch.tensor(float("-inf"))), near))
        near[:, :1] = amax
        v[:, i:i + n] = near
    return v


def same_bits(q, scale, v):
    want_q, want_s = expected(v)
    assert torch.equal(scale.cpu(), want_s)
    assert torch.equal(q.view(torch.uint8).cpu(), want_q.view(torch.uint8))


def test_the_inputs_reach_ties():
    """Among the drawn quotients many are ties exactly, and rounding a product with the reciprocal would miss some."""
    v = tie_rows(64, 512, 1)
    q, scale = expected(v)
    s = ref.widen(scale, 512)
    quotient, product = v / s, v * (1.0 / s)
    assert int((quotient != product).sum()) > 1000
    other = product.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    assert int((other.view(torch.uint8) != q.view(torch.uint8)).sum()) > 100


def to_f32(x):
    """The float32 nearest to a Fraction (ties to even), away from its subnormal range."""
    if x == 0:
        return Fraction(0)
    n, d = abs(x).as_integer_ratio()
    e = n.bit_length() - d.bit_length() - 24
    n, d = (n << -e, d) if e < 0 else (n, d << e)
    while n >= d << 24:
        d, e = d << 1, e + 1
    q, r = divmod(n, d)
    q += 2 * r > d or (2 * r == d and q & 1)
    return (1 if x > 0 else -1) * q * Fraction(2) ** e


def test_the_remainder_step_stays_on_the_quotients_side_of_a_tie():
    """q = v inv, q - (q s - v) inv with one rounding each (a fused multiply-add): the kernel's quotient.

    Its error before the last rounding is some 2^-46 of the quotient, so it rounds as the quotient does
    except perhaps where v / s is that near to the middle between two floats, and e4m3 sees the
    difference only where one of the two is a tie T = t 2^e, t of five bits.  With v and s of 24 bits,
    v / s = (T + half a unit)(1 + d) and |d| <= 2^-45 leave s t 2^20 +- s = v 2^j +- c with a small c,
    hence s = +-c modulo 2^20: all of them are gone through, and the ties themselves."""
    near = 0
    for t in range(16, 32):
        tie = t << 19
        for sign in (-1, 1):
            mid = (t << 20) + sign  # in halves of T's unit
            for i in range(8, 17):
                for c in range(-64, 65):
                    s = (i << 20) + c
                    if not 1 << 23 <= s < 1 << 24:
                        continue
                    prod = s * mid
                    j = prod.bit_length() - 24
                    v = (prod + (1 << (j - 1))) >> j
                    x = Fraction(v << j, 2 * s)  # the quotient, in units of T
                    near += abs(x - Fraction(mid, 2)) < Fraction(mid, 2 << 44)
                    inv = Fraction(float(np.float32(1) / np.float32(s)))
                    q = to_f32(Fraction(v << j) / 2 * inv)
                    r = to_f32(q * s - Fraction(v << j, 2))
                    q = to_f32(q - r * inv)
                    want = to_f32(x)
                    assert (q > tie) - (q < tie) == (want > tie) - (want < tie), (t, sign, s, v)
        for s in range((1 << 23) + 1, 1 << 24, 40961):  # v / s = T where s is short enough
            s = s >> 5 << 5
            inv = Fraction(float(np.float32(1) / np.float32(s)))
            v = Fraction(s * tie)
            assert to_f32(v) == v
            q = to_f32(v * inv)
            assert to_f32(q - to_f32(q * s - v) * inv) == tie
    assert near > 100  # the search does reach such quotients


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim", [(3, 8), (64, 512), (5, 1544), (40, 2048), (700, 8192), (2, 16512)])
def test_quantised_bits(rows, dim):
    v = tie_rows(rows, dim, rows + dim).cuda()
    q, scale = gdn.quantize_fp8(v)
    same_bits(q, scale, v)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim", [(64, 512), (300, 2048)])
def test_quantised_bits_of_bfloat16_rows(rows, dim):
    x = tie_rows(rows, dim, rows).cuda().bfloat16()
    q, scale = gdn.quantize_fp8(x)
    same_bits(q, scale, x.float())


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim,groups", [(64, 512, 1), (1000, 1024, 8), (9, 4104, 1), (3, 40960, 2)])
def test_normed_bits(rows, dim, groups):
    """In float32 the norm's own output y is v: q and scale are of exactly that."""
    x, w = tie_rows(rows, dim, dim).cuda(), torch.randn(dim, generator=torch.Generator().manual_seed(2)).cuda()
    out = gdn.rmsnorm_fp8(x, w, groups=groups, return_y=True)
    same_bits(out["q"], out["scale"], out["y"])


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [256, 8192, 16512])
def test_quantised_bits_of_tiny_and_huge_blocks_and_zeros(dim):
    """Blocks whose quotients leave subnormal remainders, blocks near the largest float, zeros of both signs."""
    v = tie_rows(40, dim, 3)
    at = torch.arange(40)[:, None] * 6.0 - 120.0 - v.abs().amax(1, keepdim=True).log2().round()
    v = v * torch.exp2(at.clamp(max=0) / 2).float() * torch.exp2(at.clamp(max=0) / 2).float() * torch.exp2(at.clamp(min=0)).float()
    v[:, 3] = 0.0
    v[:, 5] = -0.0
    v[7] = 0.0
    assert v.isfinite().all() and float(v.abs().max()) > 1e33 and 0 < float(v[1].abs().max()) < 1e-33
    q, scale = gdn.quantize_fp8(v.cuda())
    same_bits(q, scale, v)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim,groups,dtype", [(700, 8192, 1, torch.float32), (1200, 8192, 2, torch.float32), (2000, 2048, 1, torch.float32),
                                                   (3000, 2048, 1, torch.bfloat16), (500, 16392, 1, torch.bfloat16), (40, 24576, 1, torch.float32)])
def test_many_rows_give_what_each_gives_alone(rows, dim, groups, dtype):
    """Blocks that take several rows, and parts that are read twice, against the rows one by one."""
    g = torch.Generator().manual_seed(dim)
    x, r = (torch.randn(rows, dim, generator=g).cuda().to(dtype) for _ in range(2))
    w = torch.randn(dim, generator=g).cuda()
    out = gdn.rmsnorm_fp8(x, w, residual=r, groups=groups, return_y=True)
    r2 = r.clone()
    gdn.rmsnorm_fp8(x, w, residual=r2, groups=groups, residual_out=r2)
    assert torch.equal(r2, out["residual"]) and torch.equal(r2, (x.float() + r.float()).to(dtype))
    for i in (0, 1, rows // 2, rows - 1):
        one = gdn.rmsnorm_fp8(x[i:i + 1], w, residual=r[i:i + 1], groups=groups, return_y=True)
        near = (one["y"].double() - out["y"][i:i + 1].double()).abs() <= (torch.finfo(dtype).eps + 2.0 ** -20) * out["y"][i:i + 1].double().abs()
        assert near.all()  # (a row alone may run with more threads, which sum its squares in another order)
        assert torch.equal(one["residual"], out["residual"][i:i + 1])
    if dtype == torch.float32:
        same_bits(out["q"], out["scale"], out["y"])
