"""The attention block of a decoder on the library's calls.

``AttentionBlock`` runs the steps between a block's normed input and its output
projection: one projection to q, k and v; the norm and rotation of q and k with
the write of K and V into an int8 paged cache (one launch); attention over that
cache; the output projection.  The projections are layers of either kind, the
codebook layer (4-bit weights) or the int8 layer (for the ones kept at 8 bits,
or whose input width the rotation block does not divide).

Everything runs on the calls of :mod:`.binding`, on the current stream; with
:meth:`AttentionBlock.prepare` called for the token count, a step allocates
only its outputs and can be captured into a CUDA graph (a capture that would
have to allocate a workspace is refused).
"""

from __future__ import annotations

import torch

from . import binding as B


def _capturing(device: torch.device) -> bool:
    return device.type == "cuda" and torch.cuda.is_current_stream_capturing()


class _Workspaces:
    """Workspaces of a layer for any number of tokens, on each device: the last one serves every call that it is large
    enough for; where it is too small the next one is at least twice as large, and the earlier ones stay for captured
    graphs that name them.  None is made inside a capture: its zero fill would be recorded instead of run, and calls
    before the first replay would find words that must be zero as the memory held them."""

    def __init__(self, need):
        self._need = need
        self._held: list[torch.Tensor] = []
        self._of: dict[tuple[torch.device, int], torch.Tensor] = {}

    def get(self, m: int, device) -> torch.Tensor:
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        ws = self._of.get((device, m))
        if ws is None:
            need = self._need(m)
            if need == 0:
                raise B.W4A8Error("workspace", 2)
            ws = next((w for w in reversed(self._held) if w.device == device), None)
            if ws is None or ws.numel() < need:
                if _capturing(device):
                    raise RuntimeError(f"no workspace for {m} tokens yet: call prepare({m}) before the capture")
                ws = torch.zeros(need if ws is None else max(need, 2 * ws.numel()), dtype=torch.uint8, device=device)
                self._held.append(ws)
            self._of[device, m] = ws
        return ws


class CodebookLayer:
    """y = w4a8_linear(x) on a packed [N, K] layer (:func:`binding.pack_layout`)."""

    def __init__(self, packed: torch.Tensor, n: int, k: int):
        self.packed, self.n, self.k = packed, n, k
        self._workspaces = _Workspaces(lambda m: B.linear_workspace_bytes(m, k, n))

    def prepare(self, m: int) -> torch.Tensor:
        return self._workspaces.get(m, self.packed.device)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        return B.linear(x, self.packed, self.n, workspace=self.prepare(x.shape[0]))


class Int8Layer:
    """y = w4a8_int8_linear(x) on weights from :func:`binding.int8_quantize` (``rotate`` as they were quantised)."""

    def __init__(self, w_q: torch.Tensor, s_w: torch.Tensor, rotate: bool = True):
        self.w_q, self.s_w, self.rotate = w_q, s_w, rotate
        self.n, self.k = w_q.shape
        self._workspaces = _Workspaces(lambda m: B.int8_linear_workspace_bytes(m, self.k, self.n))

    def prepare(self, m: int) -> torch.Tensor:
        return self._workspaces.get(m, self.w_q.device)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        return B.int8_linear(x, self.w_q, self.s_w, rotate=self.rotate, workspace=self.prepare(x.shape[0]))


class AttentionBlock:
    """q, k, v = split(qkv(x)); K and V into the cache; y = out(attention(q)).

    ``qkv`` maps the hidden width to (heads + 2 kv_heads) * head_dim, q's heads
    first, then k's, then v's; ``out`` maps heads * head_dim back.  ``q_weight``,
    ``k_weight`` (fp32 [head_dim] or None), ``eps``, ``inv_freq``
    (:func:`binding.rope_frequencies`), ``interleaved``, ``rope_factor``, ``scale``
    and ``window`` as in :func:`binding.kv_update` and :func:`binding.kv_attention`.

    A block's layers and workspaces belong to one stream: two steps of one
    block must be ordered on the GPU.
    """

    def __init__(self, qkv, out, heads: int, kv_heads: int, head_dim: int, q_weight=None, k_weight=None,
                 eps: float = 1e-6, inv_freq=None, interleaved: bool = False, rope_factor: float = 1.0,
                 scale: float | None = None, window: int = 0):
        if qkv.n != (heads + 2 * kv_heads) * head_dim:
            raise ValueError(f"qkv has {qkv.n} outputs, not {(heads + 2 * kv_heads) * head_dim}")
        if out.k != heads * head_dim:
            raise ValueError(f"out takes {out.k} inputs, not {heads * head_dim}")
        self.qkv, self.out = qkv, out
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.rotation = dict(q_weight=q_weight, k_weight=k_weight, eps=eps, inv_freq=inv_freq, interleaved=interleaved,
                             rope_factor=rope_factor)
        self.scale, self.window = scale, window
        self._workspaces = _Workspaces(lambda m: B.kv_attention_workspace_bytes(m, heads, kv_heads, head_dim))

    def prepare(self, tokens: int, device=None) -> torch.Tensor:
        """Allocate what steps of that many tokens need (the attention's part on ``device``, by default the layers');
        returns the attention's workspace."""
        layers = [layer.prepare(tokens) for layer in (self.qkv, self.out)]
        return self._workspaces.get(tokens, layers[0].device if device is None else device)

    def __call__(self, x: torch.Tensor, cache: B.KvCache, block_table: torch.Tensor, q_start: torch.Tensor,
                 kv_len: torch.Tensor, positions: torch.Tensor | None = None) -> torch.Tensor:
        """bf16 x [T, hidden] -> bf16 y [T, hidden]; the batch as for :func:`binding.kv_update`.  Rows behind the
        last sequence come out undefined."""
        t, d = x.shape[0], self.head_dim
        workspace = self.prepare(t, x.device)
        rows = self.qkv(x).view(t, self.heads + 2 * self.kv_heads, d)
        q, k, v = rows.split([self.heads, self.kv_heads, self.kv_heads], 1)
        # q in place: its rows of the projection's output are not needed any more
        B.kv_update(cache, k, v, block_table, q_start, kv_len, q=q, q_out=q, positions=positions, **self.rotation)
        o = B.kv_attention(q, cache, block_table, q_start, kv_len, scale=self.scale, window=self.window,
                           workspace=workspace, out=x.new_empty((t, self.heads, d)))
        return self.out(o.view(t, self.heads * d))
