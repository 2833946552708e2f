"""Torch-facing convenience wrapper over the C ABI (argument marshalling only).

Tensors must already live on the CUDA device; this module only turns them into
pointers, sizes and the current stream and calls ``libtq.so``.  There is no CPU
path: a CPU tensor raises.
"""
from __future__ import annotations

import contextlib

import torch

from . import native

__all__ = ["Codec"]


def _ptr(t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device (the library has no CPU path)")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class Codec:
    """One set of codec tables (Pi, S, codebook) on the current device."""

    def __init__(self, head_dim: int, k_bits: int, v_bits: int, group: int, seed: int = 0, rotation: int = 0,
                 values: str = "group"):
        """rotation: native.TQ_ROTATION_DENSE (Haar) or native.TQ_ROTATION_HADAMARD;
        values: "group" (per-group scale / zero) or "mse" (rotation + Lloyd-Max codebook)."""
        self.head_dim, self.k_bits, self.v_bits, self.group, self.seed = head_dim, k_bits, v_bits, group, seed
        self.qjl = k_bits <= 3
        self.rotation = rotation
        self.values = values
        flags = (native.TQ_ROTATION_HADAMARD if rotation == native.TQ_ROTATION_HADAMARD else 0) | \
            (native.TQ_VALUES_MSE if values == "mse" else 0)
        self.device = torch.cuda.current_device() if torch.cuda.is_available() else 0
        self.handle = native.tq_init_ex(head_dim, k_bits, v_bits, group, seed, flags)

    def close(self):
        if getattr(self, "handle", None):
            native.tq_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---- layout -----------------------------------------------------------------
    def cache_layout(self, page_size: int):
        return native.tq_cache_layout(self.handle, page_size)

    def alloc_cache(self, num_blocks: int, num_kv_heads: int, page_size: int, device="cuda", fill: int = 0):
        kpb, vpb = self.cache_layout(page_size)
        kc = torch.full((num_blocks * num_kv_heads * kpb,), fill, dtype=torch.uint8, device=device)
        vc = torch.full((num_blocks * num_kv_heads * vpb,), fill, dtype=torch.uint8, device=device)
        return kc, vc

    # ---- calls ------------------------------------------------------------------
    def compress_kv(self, k, v, slot_mapping, k_cache, v_cache, page_size: int, num_blocks: int, stream=None):
        T, H, d = k.shape
        assert v.shape == k.shape and d == self.head_dim and k.dtype == torch.bfloat16
        assert k.stride(2) == 1 and k.stride(1) == d and v.stride(2) == 1 and v.stride(1) == d
        native.tq_compress_kv(self.handle, _ptr(k), _ptr(v), T, H, k.stride(0), v.stride(0), _ptr(slot_mapping),
                              _ptr(k_cache), _ptr(v_cache), page_size, num_blocks, _stream(stream))

    def dequant_kv(self, k_cache, v_cache, page_size: int, num_blocks: int, num_kv_heads: int, slots,
                   k_out=None, v_out=None, stream=None):
        T = slots.numel()
        shape = (T, num_kv_heads, self.head_dim)
        if k_out is None:
            k_out = torch.zeros(shape, dtype=torch.bfloat16, device=slots.device)
        if v_out is None:
            v_out = torch.zeros(shape, dtype=torch.bfloat16, device=slots.device)
        native.tq_dequant_kv(self.handle, _ptr(k_cache), _ptr(v_cache), page_size, num_blocks, num_kv_heads,
                             _ptr(slots), T, _ptr(k_out), _ptr(v_out), _stream(stream))
        return k_out, v_out

    def decode_splits(self, batch: int, num_kv_heads: int, max_blocks_per_seq: int, page_size: int) -> int:
        return native.tq_decode_splits(self.handle, batch, num_kv_heads, max_blocks_per_seq, page_size)

    def workspace(self, batch: int, num_q_heads: int, splits: int, device="cuda"):
        n = native.tq_decode_workspace_bytes(self.handle, batch, num_q_heads, splits)
        return torch.empty(n, dtype=torch.uint8, device=device)

    def decode_attention(self, q, k_cache, v_cache, block_table, seq_lens, num_kv_heads: int, page_size: int,
                         num_blocks: int, sm_scale: float, splits: int = 0, workspace=None, out=None, stream=None):
        B, Hq, d = q.shape
        assert d == self.head_dim and q.dtype == torch.bfloat16 and q.is_contiguous()
        maxb = block_table.shape[1]
        if splits == 0:
            splits = self.decode_splits(B, num_kv_heads, maxb, page_size)
        if workspace is None:
            workspace = self.workspace(B, Hq, splits, device=q.device)
        if out is None:
            out = torch.empty_like(q)
        native.tq_decode_attention(self.handle, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                   _ptr(seq_lens), B, Hq, num_kv_heads, page_size, maxb, num_blocks, float(sm_scale),
                                   splits, _ptr(workspace), workspace.numel(), _ptr(out), _stream(stream))
        return out

    def set_wait_limit(self, cycles: int):
        native.tq_set_wait_limit(self.handle, cycles)

    def prefill_attention(self, q, k_cache, v_cache, block_table, seq_lens, num_kv_heads: int, page_size: int,
                          num_blocks: int, sm_scale: float, splits: int = 0, workspace=None, out=None, stream=None):
        """Causal attention of the last q.shape[1] positions of every sequence over its compressed cache.

        q: [B, Tq, Hq, d] bf16; returns [B, Tq, Hq, d] bf16."""
        B, Tq, Hq, d = q.shape
        assert d == self.head_dim and q.dtype == torch.bfloat16 and q.is_contiguous()
        maxb = block_table.shape[1]
        if splits == 0:
            splits = native.tq_prefill_splits(self.handle, B, Tq, Hq, num_kv_heads, maxb, page_size)
        if workspace is None:
            workspace = self.workspace(B * Tq, Hq, splits, device=q.device)
        if out is None:
            out = torch.empty_like(q)
        native.tq_prefill_attention(self.handle, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                    _ptr(seq_lens), B, Tq, Hq, num_kv_heads, page_size, maxb, num_blocks,
                                    float(sm_scale), splits, _ptr(workspace), workspace.numel(), _ptr(out),
                                    _stream(stream))
        return out

    def decode_attention_bf16(self, q, k_pool, v_pool, block_table, seq_lens, num_kv_heads: int, page_size: int,
                              num_blocks: int, sm_scale: float, splits: int = 0, workspace=None, out=None,
                              stream=None):
        """Bypass decode over plain bf16 pools [num_blocks][num_kv_heads][page_size][head_dim]."""
        B, Hq, d = q.shape
        assert d == self.head_dim and q.dtype == torch.bfloat16 and q.is_contiguous()
        assert k_pool.dtype == torch.bfloat16 and v_pool.dtype == torch.bfloat16
        maxb = block_table.shape[1]
        if splits == 0:
            splits = self.decode_splits(B, num_kv_heads, maxb, page_size)
        if workspace is None:
            workspace = self.workspace(B, Hq, splits, device=q.device)
        if out is None:
            out = torch.empty_like(q)
        native.tq_decode_attention_bf16(self.handle, _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
                                        _ptr(seq_lens), B, Hq, num_kv_heads, page_size, maxb, num_blocks,
                                        float(sm_scale), splits, _ptr(workspace), workspace.numel(), _ptr(out),
                                        _stream(stream))
        return out

    # ---- plain bf16 pages and 8-bit pages ------------------------------------------
    def _need(self, ok, what: str):
        if not ok:
            raise ValueError(what)

    def _on_device(self, *tensors):
        """Every tensor on the handle's device (the current one when the Codec was made)."""
        for t in tensors:
            if t is not None and (not t.is_cuda or t.device.index != self.device):
                raise ValueError(f"tensor must be on cuda:{self.device}, the device of this Codec (there is no CPU path)")

    @contextlib.contextmanager
    def _launch(self, stream):
        """The handle's device current, and the stream to launch on: the caller's, or that device's current one.
        What is allocated inside belongs to that stream."""
        with torch.cuda.device(self.device):
            if stream is None:
                yield torch.cuda.current_stream(self.device).cuda_stream
                return
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=self.device)
            with torch.cuda.stream(stream):
                yield stream.cuda_stream

    def rope_table(self, rows: int, rot_dim: int, base: float = 10000.0):
        """cos | sin of positions 0 .. rows - 1, fp32 [rows, rot_dim], from angles in 64 bits."""
        dev = torch.device("cuda", self.device)
        inv = base ** (-torch.arange(rot_dim // 2, dtype=torch.float64, device=dev) * 2 / rot_dim)
        ang = torch.arange(rows, dtype=torch.float64, device=dev)[:, None] * inv
        return torch.cat([torch.cos(ang), torch.sin(ang)], 1).to(torch.float32)

    def alloc_pools_bf16(self, num_blocks: int, num_kv_heads: int, page_size: int):
        """Zeroed bf16 key and value pools [num_blocks][num_kv_heads][page_size][head_dim]."""
        shape = (num_blocks, num_kv_heads, page_size, self.head_dim)
        dev = torch.device("cuda", self.device)
        return torch.zeros(shape, dtype=torch.bfloat16, device=dev), torch.zeros(shape, dtype=torch.bfloat16, device=dev)

    def alloc_pools_fp8(self, num_blocks: int, num_kv_heads: int, page_size: int):
        """Zeroed e4m3 key and value pools and their scales (1.0): k_pool, v_pool, k_scales, v_scales."""
        shape = (num_blocks, num_kv_heads, page_size, self.head_dim)
        dev = torch.device("cuda", self.device)
        pools = [torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2)]
        return (*pools, *(torch.ones(shape[:2], dtype=torch.float32, device=dev) for _ in range(2)))

    def _rows(self, x, heads, what):
        """Token stride of x [T, heads, head_dim] with contiguous heads and rows."""
        T = x.shape[0]
        self._need(x.dim() == 3 and x.dtype == torch.bfloat16 and x.shape[1] == heads and x.shape[2] == self.head_dim,
                   f"{what} must be bf16 [T, heads, {self.head_dim}]")
        self._need(x.stride(2) == 1 and (heads == 1 or x.stride(1) == self.head_dim),
                   f"{what}: the heads of a token must be contiguous")
        return x.stride(0) if T > 1 else max(x.stride(0), heads * self.head_dim)

    def _pools(self, pools, dtype, num_kv_heads, page_size, num_blocks, scales=()):
        for p in pools:
            self._need(p.dtype == dtype and p.is_contiguous() and
                       p.numel() == num_blocks * num_kv_heads * page_size * self.head_dim,
                       f"pools must be contiguous {dtype} [num_blocks, num_kv_heads, page_size, head_dim]")
        for s in scales:
            self._need(s.dtype == torch.float32 and s.is_contiguous() and s.numel() == num_blocks * num_kv_heads,
                       "scales must be contiguous fp32 [num_blocks, num_kv_heads]")

    def _append_args(self, k, v, slot_mapping, q, q_out, positions, rope, interleaved):
        """Checked arguments of both appends up to the slots."""
        T, H = k.shape[0], k.shape[1]
        self._need(v.shape == k.shape, "k and v must have one shape")
        self._need(slot_mapping.dtype == torch.int64 and slot_mapping.is_contiguous() and slot_mapping.numel() == T,
                   "slot_mapping must be contiguous int64 [T]")
        ks, vs = self._rows(k, H, "k"), self._rows(v, H, "v")
        qp = qs = Hq = qo = 0
        if q is not None:
            Hq = q.shape[1]
            self._need(q.shape[0] == T, "q must have k's tokens")
            qs = self._rows(q, Hq, "q")
            if q_out is None:
                q_out = torch.zeros(T, Hq, self.head_dim, dtype=torch.bfloat16, device=q.device)
            self._need(q_out.dtype == torch.bfloat16 and q_out.is_contiguous() and q_out.shape == q.shape,
                       "q_out must be contiguous bf16 of q's shape")
            qp, qo = q.data_ptr(), q_out.data_ptr()
        else:
            self._need(q_out is None, "q_out without q")
        rp = rows = rot = pp = 0
        if rope is not None:
            self._need(rope.dim() == 2 and rope.dtype == torch.float32 and rope.is_contiguous(),
                       "rope must be contiguous fp32 [rows, rot_dim]")
            self._need(positions is not None and positions.dtype == torch.int64 and positions.is_contiguous() and
                       positions.numel() == T, "positions must be contiguous int64 [T]")
            rp, rows, rot, pp = rope.data_ptr(), rope.shape[0], rope.shape[1], positions.data_ptr()
        self._on_device(k, v, slot_mapping, q, q_out, positions if rope is not None else None, rope)
        style = native.TQ_ROPE_INTERLEAVED if interleaved else native.TQ_ROPE_HALF
        return q_out, (qp, k.data_ptr(), v.data_ptr(), T, Hq, H, qs, ks, vs, pp, rp, rows, rot, style,
                       slot_mapping.data_ptr()), qo

    def append_kv_bf16(self, k, v, slot_mapping, k_pool, v_pool, page_size: int, num_blocks: int, q=None, q_out=None,
                       positions=None, rope=None, interleaved: bool = False, stream=None):
        """Put keys (rotated by position where a rope table is given) and values into the bf16 pools.

        k, v: [T, Hkv, d] bf16, tokens strided; q: [T, Hq, d], rotated into q_out, which is returned (None without q).
        rope: fp32 [rows, rot_dim] as rope_table makes it; positions: int64 [T]."""
        with self._launch(stream) as st:
            q_out, args, qo = self._append_args(k, v, slot_mapping, q, q_out, positions, rope, interleaved)
            self._pools((k_pool, v_pool), torch.bfloat16, k.shape[1], page_size, num_blocks)
            self._on_device(k_pool, v_pool)
            native.tq_append_kv_bf16(self.handle, *args, k_pool.data_ptr(), v_pool.data_ptr(), page_size, num_blocks,
                                     qo, st)
        return q_out

    def append_kv_fp8(self, k, v, slot_mapping, k_pool, v_pool, k_scales, v_scales, page_size: int, num_blocks: int,
                      q=None, q_out=None, positions=None, rope=None, interleaved: bool = False, stream=None):
        """append_kv_bf16 into e4m3 pools with one scale per (page, kv head)."""
        with self._launch(stream) as st:
            q_out, args, qo = self._append_args(k, v, slot_mapping, q, q_out, positions, rope, interleaved)
            self._pools((k_pool, v_pool), torch.float8_e4m3fn, k.shape[1], page_size, num_blocks, (k_scales, v_scales))
            self._on_device(k_pool, v_pool, k_scales, v_scales)
            native.tq_append_kv_fp8(self.handle, *args, k_pool.data_ptr(), v_pool.data_ptr(), k_scales.data_ptr(),
                                    v_scales.data_ptr(), page_size, num_blocks, qo, st)
        return q_out

    def decode_splits_fp8(self, batch: int, num_kv_heads: int, max_blocks_per_seq: int, page_size: int) -> int:
        return native.tq_decode_splits_fp8(self.handle, batch, num_kv_heads, max_blocks_per_seq, page_size)

    def prefill_splits_fp8(self, batch: int, q_tokens: int, num_q_heads: int, num_kv_heads: int,
                           max_blocks_per_seq: int, page_size: int) -> int:
        return native.tq_prefill_splits_fp8(self.handle, batch, q_tokens, num_q_heads, num_kv_heads,
                                            max_blocks_per_seq, page_size)

    def workspace_fp8(self, batch: int, num_q_heads: int, splits: int):
        """Scratch of the attention over 8-bit pages (batch * q_tokens rows for prefill); empty where none is needed."""
        n = native.tq_workspace_bytes_fp8(self.handle, batch, num_q_heads, splits)
        return torch.empty(n, dtype=torch.uint8, device=torch.device("cuda", self.device))

    def _attention_fp8(self, q, tq, k_pool, v_pool, k_scales, v_scales, block_table, seq_lens, num_kv_heads, page_size,
                       num_blocks, sm_scale, splits, workspace, out, stream):
        B, Hq = q.shape[0], q.shape[-2]
        self._need(q.dtype == torch.bfloat16 and q.is_contiguous() and q.shape[-1] == self.head_dim,
                   f"q must be contiguous bf16 with head dim {self.head_dim}")
        self._need(block_table.dim() == 2 and block_table.dtype == torch.int32 and block_table.is_contiguous() and
                   block_table.shape[0] == B, "block_table must be contiguous int32 [B, max_blocks]")
        self._need(seq_lens.dtype == torch.int32 and seq_lens.is_contiguous() and seq_lens.numel() == B,
                   "seq_lens must be contiguous int32 [B]")
        self._pools((k_pool, v_pool), torch.float8_e4m3fn, num_kv_heads, page_size, num_blocks, (k_scales, v_scales))
        maxb = block_table.shape[1]
        with self._launch(stream) as st:
            if splits == 0:
                splits = self.decode_splits_fp8(B, num_kv_heads, maxb, page_size) if tq == 0 else \
                    self.prefill_splits_fp8(B, tq, Hq, num_kv_heads, maxb, page_size)
            if workspace is None:
                workspace = self.workspace_fp8(B * max(tq, 1), Hq, splits)
            if out is None:
                out = torch.empty_like(q)
            self._need(out.dtype == torch.bfloat16 and out.is_contiguous() and out.shape == q.shape,
                       "out must be contiguous bf16 of q's shape")
            self._on_device(q, k_pool, v_pool, k_scales, v_scales, block_table, seq_lens, workspace, out)
            pools = (k_pool.data_ptr(), v_pool.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                     block_table.data_ptr(), seq_lens.data_ptr())
            rest = (Hq, num_kv_heads, page_size, maxb, num_blocks, float(sm_scale), splits, workspace.data_ptr(),
                    workspace.numel() * workspace.element_size(), out.data_ptr(), st)
            if tq == 0:
                native.tq_decode_attention_fp8(self.handle, q.data_ptr(), *pools, B, *rest)
            else:
                native.tq_prefill_attention_fp8(self.handle, q.data_ptr(), *pools, B, tq, *rest)
        return out

    def decode_attention_fp8(self, q, k_pool, v_pool, k_scales, v_scales, block_table, seq_lens, num_kv_heads: int,
                             page_size: int, num_blocks: int, sm_scale: float, splits: int = 0, workspace=None,
                             out=None, stream=None):
        """Attention of one query token per sequence (q [B, Hq, d] bf16) over its 8-bit pages."""
        self._need(q.dim() == 3, "q must be [B, Hq, head_dim]")
        return self._attention_fp8(q, 0, k_pool, v_pool, k_scales, v_scales, block_table, seq_lens, num_kv_heads,
                                   page_size, num_blocks, sm_scale, splits, workspace, out, stream)

    def prefill_attention_fp8(self, q, k_pool, v_pool, k_scales, v_scales, block_table, seq_lens, num_kv_heads: int,
                              page_size: int, num_blocks: int, sm_scale: float, splits: int = 0, workspace=None,
                              out=None, stream=None):
        """Causal attention of the last q.shape[1] positions of every sequence (q [B, Tq, Hq, d] bf16) over its
        8-bit pages."""
        self._need(q.dim() == 4 and q.shape[1] >= 1, "q must be [B, Tq, Hq, head_dim]")
        return self._attention_fp8(q, q.shape[1], k_pool, v_pool, k_scales, v_scales, block_table, seq_lens,
                                   num_kv_heads, page_size, num_blocks, sm_scale, splits, workspace, out, stream)

    def get_status(self, stream=None) -> int:
        return native.tq_get_status(self.handle, _stream(stream))

    def export_params(self):
        import numpy as np
        d, L = self.head_dim, 1 << self.k_bits
        Pi = np.zeros((d, d), np.float32)
        S = np.zeros((d, d), np.float32)
        c = np.zeros(L, np.float32)
        t = np.zeros(L - 1, np.float32)
        native.tq_export_params(self.handle, Pi.ctypes.data, S.ctypes.data, c.ctypes.data, t.ctypes.data)
        return {"Pi": Pi, "S": S, "centroids": c, "thresholds": t}
