"""Cases that measure the selective state-space scan, the RMS norm with an 8-bit output and the
8-bit block-scaled matrix product.

`own` selects what run() computes with: False, the operators' plain forms in elementary torch
operations; True, the library's kernels through its Python binding.  Every operator is one that a
hybrid model's layer needs around and beside the token mixers of this library: the scan is a mixer
of its own (prompt and single-token form), the norm feeds the mixer's in-projection with 8-bit rows,
and the product is that projection.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
TINY = 2.0 ** -126
BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one short prompt of a small model: a call that is all launch and latency
        {"name": "scan, one short prompt", "op": "scan", "lens": "37", "heads": 8, "groups": 1, "P": 64,
         "S": 64, "dtype": "bf16", "gate": True, "init": False},
        # one 4096-token prompt at this library's 128 value heads: the ordinary prefill
        {"name": "scan, 4096 tokens", "op": "scan", "lens": "4096", "heads": 128, "groups": 8, "P": 64,
         "S": 128, "dtype": "bf16", "gate": True, "init": True},
        # a ragged batch of prompts, one of them empty and one a single token, float32 activations, an odd
        # number of heads in each group
        {"name": "scan, ragged float32", "op": "scan", "lens": "700,1,0,333,64,1291,65,2,511", "heads": 21,
         "groups": 7, "P": 128, "S": 64, "dtype": "f32", "gate": False, "init": True},
        # one long document on few heads: few chains, so the sequence has to be cut to fill the GPU
        {"name": "scan, long document", "op": "scan", "lens": "32768", "heads": 32, "groups": 1, "P": 64,
         "S": 128, "dtype": "bf16", "gate": True, "init": False},
        # one new token for one user, and for a full serving batch
        {"name": "step, one sequence", "op": "step", "batch": 1, "heads": 128, "groups": 8, "P": 64, "S": 128,
         "dtype": "bf16", "gate": True},
        {"name": "step, 256 sequences", "op": "step", "batch": 256, "heads": 128, "groups": 8, "P": 64,
         "S": 128, "dtype": "bf16", "gate": True},
        # the norm before a projection: one token, a prompt of the 8192-wide residual stream, and odd rows
        # of float32 whose last block is partial
        {"name": "norm, one row", "op": "norm", "rows": 1, "dim": 8192, "groups": 1, "dtype": "bf16",
         "residual": True},
        {"name": "norm, 4096 rows", "op": "norm", "rows": 4096, "dim": 8192, "groups": 1, "dtype": "bf16",
         "residual": True},
        {"name": "norm, ragged float32", "op": "norm", "rows": 777, "dim": 1544, "groups": 1, "dtype": "f32",
         "residual": False},
        # projections: one token through a 2048-wide layer's in-projection (q|k|v|z|a|b of 16 q/k and 32
        # value heads), a ragged mid-sized batch into float32, a prompt through the out-projection of 128
        # value heads of 128 into the 8192-wide stream
        {"name": "product, one row", "op": "product", "M": 1, "N": 12352, "K": 2048, "out": "bf16"},
        {"name": "product, ragged float32", "op": "product", "M": 301, "N": 1003, "K": 4112, "out": "f32"},
        {"name": "product, 4096 rows", "op": "product", "M": 4096, "N": 8192, "K": 16384, "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "step", "norm", "product", "product"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("scan", "step"):
        groups = rng.choice([1, 1, 2, 4, 8])
        heads = groups * _log_int(rng, 1, 128 // groups)
        P, S = rng.choice([64, 64, 128]), rng.choice([64, 128, 128])
        gate = rng.random() < 0.7
        if op == "step":
            batch = _log_int(rng, 1, min(256, max(1, (128 * 256 * 8192) // (heads * P * S))))
            return {"op": op, "batch": batch, "heads": heads, "groups": groups, "P": P, "S": S,
                    "dtype": dtype, "gate": gate}
        # at most the work of the 4096-token case: tokens times heads times state
        most = min(32768, (4096 * 128 * 64 * 128) // (heads * P * S))
        total = _log_int(rng, 1, most)
        n = rng.choice([1, 1, 2, 5, 16])
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        return {"op": op, "lens": ",".join(map(str, lens)), "heads": heads, "groups": groups, "P": P, "S": S,
                "dtype": dtype, "gate": gate, "init": rng.random() < 0.5}
    if op == "norm":
        groups = rng.choice([1, 1, 1, 2, 4])
        dim = groups * (128 * _log_int(rng, 1, 64 // groups) if groups > 1 else 8 * _log_int(rng, 1, 1024))
        return {"op": op, "rows": _log_int(rng, 1, 4096), "dim": dim, "groups": groups, "dtype": dtype,
                "residual": rng.random() < 0.6}
    return {"op": op, "M": _log_int(rng, 1, 4096), "N": _log_int(rng, 1, 8192),
            "K": 16 * _log_int(rng, 1, 1024), "out": rng.choice(["bf16", "bf16", "f32"])}


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


def _ceil(a, b):
    return -(-a // b)


# ----------------------------------------------------------------- inputs

def _mixer_weights(case, g, randn):
    H, P, S = case["heads"], case["P"], case["S"]
    conv_dim = H * P + 2 * case["groups"] * S
    dev = "cuda"
    # A in [1, 16] and steps whose softplus spans 1e-3 to 0.1 at dt = 0: heads that forget within a few
    # tokens beside heads that remember thousands
    u = torch.rand(H, generator=g, device=dev)
    step = torch.exp(math.log(1e-3) + u * (math.log(0.1) - math.log(1e-3)))
    return {
        "conv_w": 0.5 * randn(conv_dim, 4), "conv_b": 0.1 * randn(conv_dim),
        "A_log": torch.log(1 + 15 * torch.rand(H, generator=g, device=dev)),
        "dt_bias": torch.log(torch.expm1(step)), "D": 1 + 0.1 * randn(H),
    }


def _block_quant(t, block_rows):
    """8-bit weights with one scale for each block of `block_rows` x 128."""
    n, k = t.shape
    pad = torch.zeros(_ceil(n, block_rows) * block_rows, _ceil(k, BLOCK) * BLOCK, device=t.device)
    pad[:n, :k] = t
    v = pad.view(pad.shape[0] // block_rows, block_rows, pad.shape[1] // BLOCK, BLOCK)
    scale = torch.clamp(v.abs().amax(dim=(1, 3)) / FP8_MAX, min=TINY)
    q = (v / scale[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX).to(FP8)
    return q.view(pad.shape)[:n, :k].contiguous(), scale.contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": case}
    if case["op"] in ("scan", "step"):
        H, P, S, G = case["heads"], case["P"], case["S"], case["groups"]
        act = DTYPES[case["dtype"]]
        conv_dim = H * P + 2 * G * S
        rows = sum(_lens(case)) if case["op"] == "scan" else case["batch"]
        batch = len(_lens(case)) if case["op"] == "scan" else case["batch"]
        # one in-projection's rows, z | x|B|C | dt, whose parts the mixer reads in place
        zdim = H * P if case["gate"] else 0
        width = zdim + conv_dim + _ceil(H, 8) * 8
        proj = randn(rows, width).to(act)
        s["z"] = proj[:, :zdim].unflatten(1, (H, P)) if case["gate"] else None
        s["xbc"] = proj[:, zdim:zdim + conv_dim]
        s["dt"] = proj[:, zdim + conv_dim:zdim + conv_dim + H]
        s["w"] = _mixer_weights(case, g, randn)
        if case["op"] == "scan":
            cu = [0]
            for n in _lens(case):
                cu.append(cu[-1] + n)
            s["lens"] = _lens(case)
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
            s["state"] = 0.1 * randn(batch, H, P, S) if case["init"] else None
            s["conv"] = randn(batch, 3, conv_dim).to(act) if case["init"] else None
        else:
            s["state"] = 0.1 * randn(batch, H, P, S)
            s["conv"] = randn(batch, 3, conv_dim).to(act)
        return s
    if case["op"] == "norm":
        act = DTYPES[case["dtype"]]
        # a residual stream with a few channels far larger than the rest, as trained models have
        big = 1 + 20 * (torch.rand(case["dim"], generator=g, device=dev) < 0.01).float()
        s["x"] = randn(case["rows"], case["dim"]).to(act)
        s["residual"] = (2 * randn(case["rows"], case["dim"]) * big).to(act) if case["residual"] else None
        s["w"] = 0.1 * randn(case["dim"])  # zero-centred gains: the factor is 1 + w
        return s
    s["a"], s["a_scale"] = _block_quant(randn(case["M"], case["K"]), 1)
    s["b"], s["b_scale"] = _block_quant(randn(case["N"], case["K"]) / math.sqrt(case["K"]), BLOCK)
    return s


# -------------------------------------------------------------------- run

def run(s):
    return {"scan": _scan, "step": _step, "norm": _norm, "product": _product}[s["case"]["op"]](s)


def _config(c):
    import linear_attention_layer_causal_b200 as gdn
    return gdn.SsmConfig(c["groups"], c["heads"], c["P"], c["S"], act_dtype=c["dtype"])


def _scan(s):
    w = s["w"]
    if own:
        import linear_attention_layer_causal_b200 as gdn
        return gdn.ssm_prefill(_config(s["case"]), s["xbc"], s["dt"], s["cu"], w["conv_w"], w["A_log"],
                               conv_b=w["conv_b"], dt_bias=w["dt_bias"], D=w["D"], z=s["z"],
                               initial_state=s["state"], initial_conv=s["conv"], return_final_state=True,
                               return_final_conv=True)
    return _plain_scan(s)


def _step(s):
    w = s["w"]
    if own:
        import linear_attention_layer_causal_b200 as gdn
        y = gdn.ssm_decode(_config(s["case"]), s["xbc"], s["dt"], s["state"], s["conv"], w["conv_w"], w["A_log"],
                           conv_b=w["conv_b"], dt_bias=w["dt_bias"], D=w["D"], z=s["z"])
        return {"y": y, "state": s["state"], "conv": s["conv"]}
    return _plain_step(s)


def _norm(s):
    if own:
        import linear_attention_layer_causal_b200 as gdn
        out = gdn.rmsnorm_fp8(s["x"], s["w"], residual=s["residual"], groups=s["case"]["groups"],
                              eps=1e-6, weight_offset=1.0)
        return {k: out[k] for k in ("q", "scale", "residual") if k in out}
    return _plain_norm(s)


def _product(s):
    if own:
        import linear_attention_layer_causal_b200 as gdn
        return gdn.matmul_fp8(s["a"], s["a_scale"], s["b"], s["b_scale"],
                              out_dtype=DTYPES[s["case"]["out"]])
    return _plain_product(s)


# ------------------------------------------------------------ plain forms

def _plain_silu(x):
    return x / (1 + torch.exp(-x))


def _plain_softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _plain_scan(s):
    """The scan in chunks of 64 tokens over sequences padded to one length: masked products within a
    chunk, and the states entering the chunks as one product with their mutual decays."""
    c, w = s["case"], s["w"]
    H, P, S, G, Q = c["heads"], c["P"], c["S"], c["groups"], 64
    act, dev = s["xbc"].dtype, s["xbc"].device
    lens = torch.tensor(s["lens"], device=dev)
    starts = s["cu"][:-1].long()
    B, N = lens.numel(), s["xbc"].shape[0]
    nc = max(1, _ceil(max(s["lens"]), Q))
    T = nc * Q
    conv_dim = s["xbc"].shape[1]
    t = torch.arange(T, device=dev)
    valid = t[None, :] < lens[:, None]                                       # [B, T]
    at = torch.where(valid, starts[:, None] + t[None, :], torch.zeros_like(starts)[:, None])
    rows = s["xbc"][at].float() * valid[..., None]                           # [B, T, C]
    before = s["conv"].float() if s["conv"] is not None else torch.zeros(B, 3, conv_dim, device=dev)
    ext = torch.cat([before, rows], 1)
    u = w["conv_b"] + sum(w["conv_w"][:, i] * ext[:, i:i + T] for i in range(4))
    u = _plain_silu(u)
    final_conv = ext.gather(1, (lens[:, None] + torch.arange(3, device=dev))[..., None].expand(B, 3, conv_dim))
    x = u[..., :H * P].reshape(B, nc, Q, H, P)
    b = u[..., H * P:H * P + G * S].reshape(B, nc, Q, G, S)
    cc = u[..., H * P + G * S:].reshape(B, nc, Q, G, S)
    delta = _plain_softplus(s["dt"][at].float() + w["dt_bias"]) * valid[..., None]
    delta = delta.view(B, nc, Q, H)
    g = (-torch.exp(w["A_log"].double()) * delta.double()).cumsum(2)          # log decay within the chunk
    xd = x * delta[..., None]
    hpg = H // G
    mask = torch.tril(torch.ones(Q, Q, dtype=torch.bool, device=dev))
    gh = g.permute(0, 1, 3, 2)                                               # [B, nc, H, Q]
    L = torch.where(mask, torch.exp(torch.where(mask, gh[..., :, None] - gh[..., None, :], 0.0)).float(), 0.0)
    cb = torch.einsum("bcqgs,bckgs->bcgqk", cc, b).repeat_interleave(hpg, 2)
    y = torch.einsum("bchqk,bckhp->bcqhp", cb * L, xd)
    tail = torch.exp(g[:, :, -1:] - g).float()
    bh = b.repeat_interleave(hpg, 3)
    local = torch.einsum("bckhp,bckhs->bchps", xd * tail[..., None], bh)     # [B, nc, H, P, S]
    # states entering chunk i, and after the last: decays between chunk ends times the local states
    ends = torch.cat([torch.zeros(B, 1, H, dtype=torch.float64, device=dev), g[:, :, -1].cumsum(1)], 1)
    ends = ends.permute(0, 2, 1)                                             # [B, H, nc + 1]
    low = torch.tril(torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=dev))
    between = torch.where(low, torch.exp(torch.where(low, ends[..., :, None] - ends[..., None, :], 0.0)), 0.0).float()
    h0 = s["state"] if s["state"] is not None else torch.zeros(B, H, P, S, device=dev)
    enter = torch.einsum("bhij,bjhps->bihps", between, torch.cat([h0[:, None], local], 1))
    y = y + torch.einsum("bcqhs,bchps->bcqhp", cc.repeat_interleave(hpg, 3), enter[:, :-1]) * torch.exp(g).float()[..., None]
    y = (y + w["D"][:, None] * x).reshape(B, T, H, P)
    out = torch.empty(N, H, P, device=dev)
    out[at[valid]] = y[valid]
    if s["z"] is not None:
        out = out * _plain_silu(s["z"].float())
    return {"y": out.to(act), "final_state": enter[:, -1].contiguous(), "final_conv": final_conv.to(act)}


def _plain_step(s):
    c, w = s["case"], s["w"]
    H, P, S, G, B = c["heads"], c["P"], c["S"], c["groups"], c["batch"]
    act = s["xbc"].dtype
    ext = torch.cat([s["conv"], s["xbc"][:, None]], 1)                        # [B, 4, C]
    u = _plain_silu(w["conv_b"] + (ext.float() * w["conv_w"].T).sum(1))
    x = u[:, :H * P].view(B, H, P)
    b = u[:, H * P:H * P + G * S].view(B, G, S).repeat_interleave(H // G, 1)
    cc = u[:, H * P + G * S:].view(B, G, S).repeat_interleave(H // G, 1)
    delta = _plain_softplus(s["dt"].float() + w["dt_bias"])
    a = torch.exp(-torch.exp(w["A_log"]) * delta)
    new = s["state"] * a[..., None, None] + (x * delta[..., None])[..., None] * b[:, :, None]
    y = (new * cc[:, :, None]).sum(-1) + w["D"][:, None] * x
    if s["z"] is not None:
        y = y * _plain_silu(s["z"].float())
    s["state"].copy_(new)  # the resident state and window advance in place
    s["conv"].copy_(ext[:, 1:])
    return {"y": y.to(act), "state": s["state"], "conv": s["conv"]}


def _plain_norm(s):
    c = s["case"]
    r = s["x"].float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
    rows, dim = r.shape
    v = r.view(rows, c["groups"], -1)
    y = (v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6)).view(rows, dim) * (1 + s["w"])
    nb = _ceil(dim, BLOCK)
    pad = torch.nn.functional.pad(y, (0, nb * BLOCK - dim)).view(rows, nb, BLOCK)
    scale = torch.clamp(pad.abs().amax(-1) / FP8_MAX, min=TINY)
    q = (pad / scale[..., None]).clamp(-FP8_MAX, FP8_MAX).to(FP8).view(rows, -1)[:, :dim].contiguous()
    out = {"q": q, "scale": scale}
    if s["residual"] is not None:
        out["residual"] = r.to(s["x"].dtype)
    return out


def _plain_product(s):
    k = s["a"].shape[1]
    a = s["a"].float() * s["a_scale"].repeat_interleave(BLOCK, 1)[:, :k]
    n = s["b"].shape[0]
    b = s["b"].float() * s["b_scale"].repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return (a @ b.T).to(DTYPES[s["case"]["out"]])


# ------------------------------------------------------------------- work

def work(case):
    e = {"bf16": 2, "f32": 4}
    if case["op"] in ("scan", "step"):
        H, P, S, G = case["heads"], case["P"], case["S"], case["groups"]
        el = e[case["dtype"]]
        conv_dim = H * P + 2 * G * S
        n = sum(_lens(case)) if case["op"] == "scan" else case["batch"]
        batch = len(_lens(case)) if case["op"] == "scan" else case["batch"]
        row = conv_dim + H + H * P * (2 if case["gate"] else 1)
        reads_state = case["op"] == "step" or case["init"]
        state = batch * (H * P * S * 4 + 3 * conv_dim * el) * (2 if reads_state else 1)
        # a token's update and read-out of one state: a multiply-add and a multiply, and a multiply-add
        return {"bytes": n * row * el + state + conv_dim * 20, "flops": n * (5.0 * H * P * S + 8 * conv_dim)}
    if case["op"] == "norm":
        n, d = case["rows"], case["dim"]
        el = e[case["dtype"]]
        return {"bytes": n * d * (el * (3 if case["residual"] else 1) + 1) + n * _ceil(d, BLOCK) * 4 + 4 * d,
                "flops": 8.0 * n * d}
    M, N, K = case["M"], case["N"], case["K"]
    kb = _ceil(K, BLOCK)
    return {"bytes": M * K + N * K + 4 * kb * (M + _ceil(N, BLOCK)) + M * N * e[case["out"]],
            "flops": 2.0 * M * N * K}


# ------------------------------------------------------------------ exact

def exact(case, seed):
    s = prepare(case, seed)
    return {"scan": _exact_mixer, "step": _exact_mixer, "norm": _exact_norm, "product": _exact_product}[case["op"]](s)


def _exact_mixer(s):
    """Token by token, from the recurrence, in 64 bits."""
    c = s["case"]
    H, P, S, G = c["heads"], c["P"], c["S"], c["groups"]
    w = {k: v.double() for k, v in s["w"].items()}
    act = s["xbc"].dtype
    step = c["op"] == "step"
    lens = [1] * c["batch"] if step else s["lens"]
    begin = [sum(lens[:i]) for i in range(len(lens))]
    B, dev = len(lens), s["xbc"].device
    xbc = s["xbc"]
    window = s["conv"].double() if s["conv"] is not None else torch.zeros(B, 3, xbc.shape[1], dtype=torch.float64, device=dev)
    window = window.clone()
    h = s["state"].double() if s["state"] is not None else torch.zeros(B, H, P, S, dtype=torch.float64, device=dev)
    h = h.clone()
    y = torch.zeros(xbc.shape[0], H, P, dtype=torch.float64, device=dev)
    A = torch.exp(w["A_log"])
    order = sorted(range(B), key=lambda i: -lens[i])
    index = torch.tensor(order, device=dev)
    first = torch.tensor([begin[i] for i in order], device=dev)
    window, h = window[index], h[index]
    for t in range(max(lens)):
        n = sum(1 for v in lens if v > t) if B > 1 else 1
        rows = first[:n] + t
        new = xbc[rows].double()
        pre = (window[:n] * w["conv_w"][:, :3].T).sum(1) + new * w["conv_w"][:, 3] + w["conv_b"]
        u = pre * torch.sigmoid(pre)
        window[:n] = torch.cat([window[:n, 1:], new[:, None]], 1)
        x = u[:, :H * P].reshape(n, H, P)
        delta = torch.logaddexp(s["dt"][rows].double() + w["dt_bias"], torch.zeros((), dtype=torch.float64, device=dev))
        b = u[:, H * P:H * P + G * S].reshape(n, G, 1, 1, S).expand(n, G, H // G, 1, S).reshape(n, H, 1, S)
        cc = u[:, H * P + G * S:].reshape(n, G, 1, S, 1).expand(n, G, H // G, S, 1).reshape(n, H, S, 1)
        h[:n].mul_(torch.exp(-A * delta)[..., None, None]).add_((delta[..., None] * x)[..., None] * b)
        y[rows] = torch.matmul(h[:n], cc).squeeze(-1) + w["D"][:, None] * x
    if s["z"] is not None:
        z = s["z"].double()
        y = y * (z * torch.sigmoid(z))
    back = torch.argsort(index)
    window, h = window[back], h[back]
    if step:
        return {"y": y, "state": h, "conv": window.to(act).double()}
    return {"y": y, "final_state": h, "final_conv": window.to(act).double()}


def _exact_norm(s):
    c = s["case"]
    r = s["x"].double() + (s["residual"].double() if s["residual"] is not None else 0.0)
    rows, dim = r.shape
    parts = r.reshape(rows * c["groups"], dim // c["groups"])
    y = parts / torch.sqrt(torch.linalg.vector_norm(parts, dim=1, keepdim=True) ** 2 / parts.shape[1] + 1e-6)
    y = y.reshape(rows, dim) * (1 + s["w"].double())
    scales = [y[:, k:k + BLOCK].abs().max(1).values / FP8_MAX for k in range(0, dim, BLOCK)]
    scale = torch.stack(scales, 1).clamp(min=TINY)
    q = torch.cat([y[:, i * BLOCK:(i + 1) * BLOCK] / scale[:, i:i + 1] for i in range(scale.shape[1])], 1)
    out = {"q": q, "scale": scale}
    if s["residual"] is not None:
        out["residual"] = r
    return out


def _exact_product(s):
    M, K = s["a"].shape
    N = s["b"].shape[0]
    a, b = s["a"].double(), s["b"].double()
    for i in range(0, K, BLOCK):  # scale the blocks where they stand
        a[:, i:i + BLOCK] *= s["a_scale"][:, i // BLOCK, None].double()
        for j in range(0, N, BLOCK):
            b[j:j + BLOCK, i:i + BLOCK] *= s["b_scale"][j // BLOCK, i // BLOCK].double()
    return a @ b.T
