"""Attention sublayers of a diffusion transformer on the library's kernels, and the block that holds one.

  SelfAttention    x -> to_qkv -> norm and rotation of q and k -> attention -> to_out
  CrossAttention   x -> to_q -> norm and rotation, over states that `encode` projected once (to_kv, norm of k): a text
                   encoder's states stay the same over all denoising steps, so their keys and values are kept
  FluxBlock        to_qkv .. to_out, then the MLP pair (fused across the GELU), as `compress` packs it

The projections are any of the package's layer classes (SvdqLinear, Fp8Linear, W8A8Linear, ...); between them run
svdq_qk_norm_rope (in place on the projection's output) and svdq_cross_attn.  Everything is enqueued, and every
intermediate allocated, on `stream` (default: the current stream), and the host waits for nothing (but in FluxBlock's
first call of a larger token count, for its rotation table).  The layers' workspaces serve one call at a time: a call on
another stream than the object's last call comes after what that stream has been given so far.  (Not in a capture, and
not after a raw handle's stream, which may be gone: there the caller sees to the order.)
"""
from __future__ import annotations

import functools

from . import SVDQ_OK, _layer_device, _stream_context, _current_handle, svdq_cross_attn, svdq_mlp_forward, svdq_mlp_fusable, \
    svdq_qk_norm_rope


def _after_last_call(self, handle: int):
    """The current stream, of this handle, waits for the stream of the object's last call, whose kernels use the same
    workspaces."""
    import torch

    with torch.cuda.device(self.device):
        if torch.cuda.is_current_stream_capturing():
            return
    stream = torch.cuda.current_stream(self.device)
    if self._last is not None:
        stream.wait_stream(self._last[1])
    raw = handle != 0 and stream.stream_id == handle
    self._last = None if raw else (handle, stream)


def _on_stream(f):
    """The method with its `stream` argument made the current stream of the object's device: its intermediates then
    belong to that stream."""

    @functools.wraps(f)
    def g(self, *args, stream=None, **kw):
        if stream is not None:
            with _stream_context(stream, self.device):
                return g(self, *args, **kw)
        handle = _current_handle(self.device)
        if self._last is None or self._last[0] != handle:
            _after_last_call(self, handle)
        return f(self, *args, **kw)

    return g


def rope_table(rows: int, rot_dim: int, theta: float = 10000.0, device=None):
    """Cosines and sines f32 [rows, rot_dim/2, 2] of the angles row * theta^(-2i/rot_dim), computed in binary64 (far
    positions lose their angle in binary32)."""
    import torch

    device = _layer_device(device)
    freq = theta ** (-torch.arange(rot_dim // 2, dtype=torch.float64, device=device) * 2 / rot_dim)
    angle = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * freq[None, :]
    return torch.stack((angle.cos(), angle.sin()), dim=-1).float().contiguous()


def _fits(heads: int, N: int, parts: int, what: str) -> int:
    if heads < 1 or N % (parts * heads):
        raise ValueError(f"{what}: {N} outputs are not {parts} x {heads} heads")
    return N // (parts * heads)


def _tokens(x, layer):
    if x.dim() != 3 or x.shape[2] != layer.K:
        raise ValueError(f"expected [batch, tokens, {layer.K}], got {tuple(x.shape)}")
    return x.shape[0], x.shape[1]


class SelfAttention:
    """Attention among a block's own tokens: `to_qkv` maps a token to heads * dim queries, as many keys and as many
    values, `to_out` takes the heads back.  q_norm and k_norm are bf16 [dim] weights of the head norms or None."""

    _last = None  # (handle, stream) of the last call

    def __init__(self, to_qkv, to_out, heads: int, q_norm=None, k_norm=None, eps: float = 1e-6,
                 pairs: str = "interleaved"):
        self.dim = _fits(heads, to_qkv.N, 3, "to_qkv")
        if to_out.K != heads * self.dim or to_out.device != to_qkv.device:
            raise ValueError("to_out does not take to_qkv's heads")
        self.to_qkv, self.to_out, self.heads, self.device = to_qkv, to_out, heads, to_out.device
        self.q_norm, self.k_norm, self.eps, self.pairs = q_norm, k_norm, eps, pairs

    @_on_stream
    def forward(self, x, rope=None, positions=None, kv_len=None, kv_mask=None):
        """x bf16 [B, S, K] -> [B, S, to_out.N]; rope and positions as in svdq_qk_norm_rope, kv_len and kv_mask as in
        svdq_cross_attn (tokens that no query sees)."""
        b, s = _tokens(x, self.to_qkv)
        qkv = self.to_qkv.forward(x).view(b, s, 3, self.heads, self.dim)
        q, k, v = qkv.unbind(2)
        svdq_qk_norm_rope(q, k, self.q_norm, self.k_norm, eps=self.eps, rope=rope, positions=positions,
                          pairs=self.pairs, out_q=q, out_k=k)
        o = svdq_cross_attn(q, k, v, kv_len=kv_len, kv_mask=kv_mask,
                            out=x.new_empty(b, s, self.heads, self.dim))
        return self.to_out.forward(o.view(b, s, self.to_out.K)).view(b, s, self.to_out.N)

    __call__ = forward


class CrossAttention:
    """Attention over an encoder's states: `to_q` maps a token to heads * dim queries, `to_kv` a state to
    kv_heads * dim keys and as many values (kv_heads: heads, or a divisor of it whose heads are shared)."""

    _last = None  # (handle, stream) of the last call

    def __init__(self, to_q, to_kv, to_out, heads: int, kv_heads: int | None = None, q_norm=None, k_norm=None,
                 eps: float = 1e-6, pairs: str = "interleaved"):
        kv_heads = heads if kv_heads is None else kv_heads
        self.dim = _fits(heads, to_q.N, 1, "to_q")
        if _fits(kv_heads, to_kv.N, 2, "to_kv") != self.dim or heads % kv_heads:
            raise ValueError(f"to_kv's {kv_heads} heads do not serve to_q's {heads} of {self.dim}")
        if to_out.K != heads * self.dim or not (to_q.device == to_kv.device == to_out.device):
            raise ValueError("to_out does not take to_q's heads")
        self.to_q, self.to_kv, self.to_out, self.heads, self.kv_heads = to_q, to_kv, to_out, heads, kv_heads
        self.device = to_out.device
        self.q_norm, self.k_norm, self.eps, self.pairs = q_norm, k_norm, eps, pairs

    @_on_stream
    def encode(self, states, rope=None, positions=None):
        """Keys and values [B, Sk, kv_heads, dim] of states bf16 [B, Sk, K], for any number of `forward` calls."""
        b, s = _tokens(states, self.to_kv)
        kv = self.to_kv.forward(states).view(b, s, 2, self.kv_heads, self.dim)
        k, v = kv.unbind(2)
        svdq_qk_norm_rope(k, None, self.k_norm, eps=self.eps, rope=rope, positions=positions, pairs=self.pairs,
                          out_q=k)
        return k, v

    @_on_stream
    def forward(self, x, keys_values, rope=None, positions=None, kv_len=None, kv_mask=None):
        """x bf16 [B, S, K] and what `encode` gave -> [B, S, to_out.N]; kv_len and kv_mask say which states count."""
        b, s = _tokens(x, self.to_q)
        k, v = keys_values
        q = self.to_q.forward(x).view(b, s, self.heads, self.dim)
        svdq_qk_norm_rope(q, None, self.q_norm, eps=self.eps, rope=rope, positions=positions, pairs=self.pairs,
                          out_q=q)
        o = svdq_cross_attn(q, k, v, kv_len=kv_len, kv_mask=kv_mask)
        return self.to_out.forward(o.view(b, s, self.to_out.K)).view(b, s, self.to_out.N)

    __call__ = forward


class FluxBlock:
    """The image stream's linears of a FLUX-style block with their attention, from the layers of a packed checkpoint
    (`compress.load`): to_qkv -> attention -> to_out -> MLP up -> GELU -> down.  q_norm and k_norm are bf16 [dim] weights of
    the head norms or None.  Tokens are rotated by their number, or by the caller's table (a row for each token of, say,
    several axes' angles side by side).  (Residuals, modulation and the block's normalizations belong to the caller.)"""

    _last = None  # (handle, stream) of the last call

    def __init__(self, layers: dict, heads: int, theta: float = 10000.0, prefix: str = "transformer_blocks.0.", q_norm=None,
                 k_norm=None, eps: float = 1e-6):
        self.attention = SelfAttention(layers[prefix + "attn.to_qkv"], layers[prefix + "attn.to_out.0"], heads, q_norm,
                                       k_norm, eps)
        self.up, self.down = layers[prefix + "ff.net.0.proj"], layers[prefix + "ff.net.2"]
        if svdq_mlp_fusable(self.up.handle, self.down.handle) != SVDQ_OK:
            raise ValueError("the MLP pair's shapes or formats cannot be fused (both NVFP4, static scale)")
        self.theta, self._ropes, self.device = theta, [], self.up.device

    def _table(self, tokens: int):
        """Cosines and sines of the first `tokens` rows or more.  A table for more tokens than any before is made once (half
        as long again as the one before: all of them come to 4.5 times what the longest call needs at most), and waited
        for."""
        import torch

        t = self._ropes[-1] if self._ropes else None
        if t is None or t.shape[0] < tokens:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError(f"no rotation table for {tokens} tokens yet: run the block once before the capture")
            rows = max(tokens, t.shape[0] * 3 // 2 if t is not None else 0)
            t = rope_table(rows, self.attention.dim, self.theta, self.up.device)
            torch.cuda.current_stream(self.up.device).synchronize()  # before any other stream uses it
            self._ropes.append(t)  # the shorter ones stay: a captured graph may read them
        return t

    @_on_stream
    def forward(self, x, rope=None, positions=None):
        """x bf16 [B, S, K] -> [B, S, down.N]; rope and positions as in svdq_qk_norm_rope (rope: by the token's number)."""
        import torch

        b, s = _tokens(x, self.attention.to_qkv)
        if rope is None and positions is not None:
            raise ValueError("positions need a rope table")
        h = self.attention.forward(x, rope=self._table(s) if rope is None else rope, positions=positions)
        y = x.new_empty(b * s, self.down.N)
        with torch.cuda.device(self.up.device):
            svdq_mlp_forward(self.up.handle, self.down.handle, h, b * s, y, self.up.workspace(b * s),
                             self.down.workspace(b * s))
        return y.view(b, s, self.down.N)

    __call__ = forward
