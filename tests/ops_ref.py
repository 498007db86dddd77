"""Plain 64-bit forms of the state-space mixer, the norm with an 8-bit output and the 8-bit matrix
product, for the tests: torch float64 on the inputs' device, one token and one block at a time.

Besides the values, ssm() returns for y and the state a magnitude: the same recurrence on absolute
values, with sum |w x| + |b| in the place of each convolved channel.  It bounds the sum of the
absolute values of every term that enters an output, so an error bound per operation times the
magnitude bounds the output's error.
"""
import torch

FP8_MAX = 448.0
TINY = 2.0 ** -126


def silu(x):
    return x * torch.sigmoid(x)


def ssm(cfg, xbc, dt, lens, conv_w, A_log, conv_b=None, dt_bias=None, D=None, z=None, state=None, conv=None):
    """The recurrence over packed sequences: dict of y, state, conv (window), y_mag, state_mag."""
    H, P, S, G, C = cfg.num_heads, cfg.head_dim, cfg.state_dim, cfg.num_groups, cfg.conv_dim
    dev, f = xbc.device, torch.float64
    N, B = xbc.shape[0], len(lens)
    x64, dt64, w = xbc.to(f), dt.to(f), conv_w.to(f)
    b = torch.zeros(C, dtype=f, device=dev) if conv_b is None else conv_b.to(f)
    bias = torch.zeros(H, dtype=f, device=dev) if dt_bias is None else dt_bias.to(f)
    Dv = torch.zeros(H, dtype=f, device=dev) if D is None else D.to(f)
    y, y_mag = torch.zeros(N, H, P, dtype=f, device=dev), torch.zeros(N, H, P, dtype=f, device=dev)
    out_s = torch.zeros(B, H, P, S, dtype=f, device=dev)
    out_m = torch.zeros_like(out_s)
    out_c = torch.zeros(B, 3, C, dtype=xbc.dtype, device=dev)
    A = torch.exp(A_log.to(f))
    t = 0
    for n, L in enumerate(lens):
        h = torch.zeros(H, P, S, dtype=f, device=dev) if state is None else state[n].to(f).clone()
        m = h.abs()
        win = torch.zeros(3, C, dtype=xbc.dtype, device=dev) if conv is None else conv[n].clone()
        rows = torch.cat([win, xbc[t:t + L]])
        r64 = rows.to(f)
        for i in range(L):
            terms = r64[i:i + 4].T * w
            pre = terms.sum(1) + b
            u, um = silu(pre), terms.abs().sum(1) + b.abs()
            d = torch.logaddexp(dt64[t + i] + bias, torch.zeros((), dtype=f, device=dev)).clamp(cfg.dt_min, cfg.dt_max)
            a = torch.exp(-A * d)[:, None, None]

            def parts(v):
                return (v[:H * P].view(H, P), v[H * P:H * P + G * S].view(G, S).repeat_interleave(H // G, 0),
                        v[H * P + G * S:].view(G, S).repeat_interleave(H // G, 0))
            xv, bv, cv = parts(u)
            xm, bm, cm = parts(um)
            h = a * h + (d[:, None] * xv)[..., None] * bv[:, None]
            m = a * m + (d[:, None] * xm)[..., None] * bm[:, None]
            o = (h * cv[:, None]).sum(-1) + Dv[:, None] * xv
            om = (m * cm[:, None]).sum(-1) + Dv.abs()[:, None] * xm
            if z is not None:
                g = z[t + i].to(f)
                o, om = o * silu(g), om * g.abs()
            y[t + i], y_mag[t + i] = o, om
        out_s[n], out_m[n] = h, m
        out_c[n] = rows[-3:]
        t += L
    return {"y": y, "state": out_s, "conv": out_c, "y_mag": y_mag, "state_mag": out_m}


def norm(x, weight, residual=None, groups=1, eps=1e-6, offset=0.0):
    """dict of r (x + residual), v (the norm's output), scale, all float64."""
    r = x.double() + (0 if residual is None else residual.double())
    rows, dim = r.shape
    v = r
    if weight is not None:
        p = r.view(rows, groups, -1)
        v = (p / torch.sqrt((p * p).mean(-1, keepdim=True) + eps)).reshape(rows, dim) * (offset + weight.double())
    return {"r": r, "v": v, "scale": block_scale(v)}


def block_scale(v):
    cols = [v[:, i:i + 128].abs().amax(1) / FP8_MAX for i in range(0, v.shape[1], 128)]
    return torch.stack(cols, 1).clamp(min=TINY)


def widen(scale, dim):
    return scale.repeat_interleave(128, 1)[:, :dim]


def quant(t, rows):
    """t as e4m3 with one float32 scale for each block of `rows` x 128 (the inputs of a product)."""
    n, k = t.shape
    nb, kb = -(-n // rows), -(-k // 128)
    q = torch.empty(n, k, dtype=torch.float8_e4m3fn, device=t.device)
    s = torch.empty(nb, kb, device=t.device)
    for i in range(nb):
        for j in range(kb):
            blk = t[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128]
            s[i, j] = max(float(blk.abs().max()) / FP8_MAX, TINY)
            q[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128] = (blk / s[i, j]).clamp(-FP8_MAX, FP8_MAX).to(q.dtype)
    return q, s


def product(a, sa, w, sw):
    """(value, sum of the absolute values of its terms), float64."""
    A = a.double() * widen(sa.double(), a.shape[1])
    W = w.double() * widen(sw.double().repeat_interleave(128, 0)[:w.shape[0]], w.shape[1])
    return A @ W.T, A.abs() @ W.abs().T
