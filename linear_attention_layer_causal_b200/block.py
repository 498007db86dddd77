"""One layer around a token mixer, from residual stream to residual stream, with 8-bit projections:

    q = e4m3 of RMSNorm(hidden + residual)          rmsnorm_fp8
    in-projection                                   matmul_fp8
    token mixer (state-space, or Gated DeltaNet)    ssm_prefill / ssm_decode, prefill / decode
    e4m3 of the mixer's output (after an optional
    RMSNorm by groups)                              rmsnorm_fp8 or quantize_fp8
    out-projection                                  matmul_fp8

Only a composition of the library's calls; it computes nothing itself.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional, Union

from . import (BLOCK, Config, SsmConfig, decode, matmul_fp8, prefill, quantize_fp8, rmsnorm_fp8,
               ssm_decode, ssm_prefill)


def in_projection_rows(mixer: Union[Config, SsmConfig]) -> list:
    """Rows of the in-projection's weight by part, each part's padded to whole blocks of 128 (what
    the rows behind a part hold is not used).

    A state-space mixer reads its parts as slices of one product's rows, z | x|B|C | dt; Gated
    DeltaNet takes contiguous tensors, so that qkv, z and a|b are products of their own."""
    def pad(n):
        return -(-n // BLOCK) * BLOCK
    if isinstance(mixer, SsmConfig):
        hp = mixer.num_heads * mixer.head_dim
        return [("z|xbc|dt", pad(hp + mixer.conv_dim + mixer.num_heads))]
    return [("qkv", pad(mixer.conv_dim)), ("z", pad(mixer.num_v_heads * mixer.head_dim)),
            ("a|b", pad(2 * mixer.num_v_heads))]


def _heads(mixer):
    return mixer.num_heads if isinstance(mixer, SsmConfig) else mixer.num_v_heads


@dataclass
class MixerBlock:
    """Weights of one layer.  in_w [rows, hidden] e4m3 with in_scale [rows / 128, ceil(hidden / 128)],
    its rows as in_projection_rows() lists them; out_w [hidden, H P] (or [hidden, H_v d]) with
    out_scale; params: the mixer's keyword parameters (conv_w, A_log, ..).  Activations are
    bfloat16."""
    mixer: Union[Config, SsmConfig]
    norm_w: object
    in_w: object
    in_scale: object
    out_w: object
    out_scale: object
    params: dict
    out_norm_w: Optional[object] = None  # state-space mixer: RMSNorm by groups before the out-projection
    eps: float = 1e-6
    weight_offset: float = 0.0           # 1.0: zero-centred gains of norm_w

    def __post_init__(self):
        if self.mixer.act_dtype != "bf16":
            raise ValueError("MixerBlock runs bfloat16 activations")
        rows = sum(n for _, n in in_projection_rows(self.mixer))
        if self.in_w.shape[0] != rows:
            raise ValueError(f"in_w must have {rows} rows {in_projection_rows(self.mixer)}, got {self.in_w.shape[0]}")
        hidden, width = self.in_w.shape[1], _heads(self.mixer) * self.mixer.head_dim
        for name, shape in (("norm_w", (hidden,)), ("in_scale", (rows // BLOCK, -(-hidden // BLOCK))),
                            ("out_w", (hidden, width)), ("out_scale", (-(-hidden // BLOCK), -(-width // BLOCK))),
                            ("out_norm_w", (width,))):
            t = getattr(self, name)
            if t is None and name == "out_norm_w":
                continue
            if t is None or tuple(t.shape) != shape:
                raise ValueError(f"{name} must have the shape {shape}, got {None if t is None else tuple(t.shape)}")

    def _project(self, hidden, residual):
        n = rmsnorm_fp8(hidden, self.norm_w, residual=residual, eps=self.eps, weight_offset=self.weight_offset)
        parts, at = [], 0
        for _, rows in in_projection_rows(self.mixer):
            parts.append(matmul_fp8(n["q"], n["scale"], self.in_w[at:at + rows],
                                    self.in_scale[at // BLOCK:(at + rows) // BLOCK]))
            at += rows
        return parts, n.get("residual", hidden)

    def _inputs(self, parts):
        m = self.mixer
        if isinstance(m, SsmConfig):
            hp, (rows,) = m.num_heads * m.head_dim, parts
            return dict(z=rows[:, :hp].unflatten(1, (m.num_heads, m.head_dim)), xbc=rows[:, hp:hp + m.conv_dim],
                        dt=rows[:, hp + m.conv_dim:hp + m.conv_dim + m.num_heads])
        qkv, z, ab = parts
        h = m.num_v_heads
        return dict(qkv=qkv[:, :m.conv_dim].contiguous(), a=ab[:, :h].contiguous(), b=ab[:, h:2 * h].contiguous(),
                    z=z[:, :h * m.head_dim].contiguous().unflatten(1, (h, m.head_dim)))

    def _out(self, y):
        flat = y.flatten(1)
        if self.out_norm_w is not None:
            groups = self.mixer.num_groups if isinstance(self.mixer, SsmConfig) else 1
            n = rmsnorm_fp8(flat, self.out_norm_w, groups=groups, eps=self.eps)
            q, scale = n["q"], n["scale"]
        else:
            q, scale = quantize_fp8(flat)
        return matmul_fp8(q, scale, self.out_w, self.out_scale)

    def prefill(self, hidden, residual, cu_seqlens, *, initial_state=None, initial_conv=None):
        """Packed prompts: hidden, residual [N, hidden] (residual None at the first layer).  Returns
        (hidden, residual, state, conv window)."""
        parts, residual = self._project(hidden, residual)
        i, kw = self._inputs(parts), dict(initial_state=initial_state, initial_conv=initial_conv,
                                          return_final_state=True, return_final_conv=True)
        if isinstance(self.mixer, SsmConfig):
            o = ssm_prefill(self.mixer, i["xbc"], i["dt"], cu_seqlens, z=i["z"], **self.params, **kw)
        else:
            o = prefill(self.mixer, i["qkv"], i["a"], i["b"], i["z"], cu_seqlens, **self.params, **kw)
        return self._out(o["y"]), residual, o["final_state"], o["final_conv"]

    def decode(self, hidden, residual, state, conv_cache):
        """One token per sequence; `state` and `conv_cache` advance in place.  Returns (hidden, residual)."""
        parts, residual = self._project(hidden, residual)
        i = self._inputs(parts)
        if isinstance(self.mixer, SsmConfig):
            y = ssm_decode(self.mixer, i["xbc"], i["dt"], state, conv_cache, z=i["z"], **self.params)
        else:
            y = decode(self.mixer, i["qkv"], i["a"], i["b"], i["z"], state, conv_cache, **self.params)
        return self._out(y), residual
