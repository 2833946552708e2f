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


# The current stream's handle; the plain call builds a Stream object each time (1.1 against 0.1 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


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
    # The calls below are made once per layer and token, so their checks are few and plain: what the library cannot
    # see (types, contiguity, sizes, devices) is checked here, everything else by the library.
    def _on(self, stream):
        """Context for a call whose stream or device is not the current one: both made current, so that what the
        call allocates belongs to its stream."""
        if getattr(stream, "device", None) is not None and torch.device(stream.device).index != self.device:
            raise ValueError(f"stream must be one of cuda:{self.device}, the device of this Codec; got one of {stream.device}")
        stack = contextlib.ExitStack()
        stack.enter_context(torch.cuda.device(self.device))
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=self.device)
            stack.enter_context(torch.cuda.stream(stream))
        return stack

    def _elsewhere(self, stream) -> bool:
        return stream is not None or torch.cuda.current_device() != self.device

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

    def _flat(self, t, dtype, numel: int, what: str) -> int:
        """The address of a contiguous tensor of this type and size on the handle's device."""
        if t.dtype is not dtype or t.numel() != numel or not t.is_contiguous() or t.get_device() != self.device:
            raise ValueError(f"{what} must be contiguous {dtype} with {numel} elements on cuda:{self.device}, the device "
                             f"of this Codec; got {t.dtype} {tuple(t.shape)} on {t.device}")
        return t.data_ptr()

    def _rows(self, x, T: int, heads: int, what: str):
        """Address and token stride of bf16 rows x [T, heads, head_dim], the heads of a token side by side."""
        d = self.head_dim
        if x.dtype is not torch.bfloat16 or x.shape != (T, heads, d) or x.get_device() != self.device:
            raise ValueError(f"{what} must be bf16 [{T}, {heads}, {d}] on cuda:{self.device}; got {x.dtype} "
                             f"{tuple(x.shape)} on {x.device}")
        st, sh, sd = x.stride()
        if T > 0 and (sd != 1 or (heads > 1 and sh != d)):
            raise ValueError(f"{what}: the heads of a token must be contiguous")
        return x.data_ptr(), st if T > 1 else heads * d

    def _append(self, call, dtype, k, v, slot_mapping, pools, scales, page_size, num_blocks, q, q_out, positions, rope,
                interleaved, stream):
        if self._elsewhere(stream):
            with self._on(stream):
                return self._append(call, dtype, k, v, slot_mapping, pools, scales, page_size, num_blocks, q, q_out,
                                    positions, rope, interleaved, None)
        if k.dim() != 3:
            raise ValueError("k must be [T, num_kv_heads, head_dim]")
        T, H, _ = k.shape
        kp, ks = self._rows(k, T, H, "k")
        vp, vs = self._rows(v, T, H, "v")
        sp = self._flat(slot_mapping, torch.int64, T, "slot_mapping")
        qp = qs = Hq = qo = rp = rows = rot = pp = 0
        if rope is not None:
            if rope.dim() != 2 or positions is None:
                raise ValueError("rope must be fp32 [rows, rot_dim], and goes with positions")
            rows, rot = rope.shape
            rp = self._flat(rope, torch.float32, rows * rot, "rope")
            pp = self._flat(positions, torch.int64, T, "positions")
        cells = num_blocks * H * page_size * self.head_dim
        ptrs = [self._flat(p, dtype, cells, "a pool [num_blocks, num_kv_heads, page_size, head_dim]") for p in pools]
        ptrs += [self._flat(s, torch.float32, num_blocks * H, "scales [num_blocks, num_kv_heads]") for s in scales]
        if q is not None:
            if q.dim() != 3:
                raise ValueError("q must be [T, num_q_heads, head_dim]")
            Hq = q.shape[1]
            qp, qs = self._rows(q, T, Hq, "q")
            if q_out is None:  # zeros: rows of skipped tokens are not written
                q_out = torch.zeros(q.shape, dtype=torch.bfloat16, device=q.device)
            qo = self._flat(q_out, torch.bfloat16, T * Hq * self.head_dim, "q_out")
        elif q_out is not None:
            raise ValueError("q_out without q")
        call(self.handle, qp, kp, vp, T, Hq, H, qs, ks, vs, pp, rp, rows, rot,
             native.TQ_ROPE_INTERLEAVED if interleaved else native.TQ_ROPE_HALF, sp, *ptrs, page_size, num_blocks, qo,
             _raw_stream(self.device))
        return q_out

    def append_kv_bf16(self, k, v, slot_mapping, k_pool, v_pool, page_size: int, num_blocks: int, q=None, q_out=None,
                       positions=None, rope=None, interleaved: bool = False, stream=None):
        """Put keys (rotated by position where a rope table is given) and values into the bf16 pools.

        k, v: [T, Hkv, d] bf16, tokens strided; q: [T, Hq, d], rotated into q_out, which is returned (None without q).
        rope: fp32 [rows, rot_dim] as rope_table makes it; positions: int64 [T]."""
        return self._append(native.tq_append_kv_bf16, torch.bfloat16, k, v, slot_mapping, (k_pool, v_pool), (), page_size,
                            num_blocks, q, q_out, positions, rope, interleaved, stream)

    def append_kv_fp8(self, k, v, slot_mapping, k_pool, v_pool, k_scales, v_scales, page_size: int, num_blocks: int,
                      q=None, q_out=None, positions=None, rope=None, interleaved: bool = False, stream=None):
        """append_kv_bf16 into e4m3 pools with one scale per (page, kv head)."""
        return self._append(native.tq_append_kv_fp8, torch.float8_e4m3fn, k, v, slot_mapping, (k_pool, v_pool),
                            (k_scales, v_scales), page_size, num_blocks, q, q_out, positions, rope, interleaved, stream)

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
        if self._elsewhere(stream):
            with self._on(stream):
                return self._attention_fp8(q, tq, k_pool, v_pool, k_scales, v_scales, block_table, seq_lens, num_kv_heads,
                                           page_size, num_blocks, sm_scale, splits, workspace, out, None)
        B, Hq, d = q.shape[0], q.shape[-2], self.head_dim
        if q.shape[-1] != d or block_table.dim() != 2:
            raise ValueError(f"q must have head dim {d}, block_table be [B, max_blocks]")
        maxb = block_table.shape[1]
        cells = num_blocks * num_kv_heads
        f8, f32, i32 = torch.float8_e4m3fn, torch.float32, torch.int32
        qp = self._flat(q, torch.bfloat16, B * max(tq, 1) * Hq * d, "q")
        args = (self._flat(k_pool, f8, cells * page_size * d, "k_pool"), self._flat(v_pool, f8, cells * page_size * d, "v_pool"),
                self._flat(k_scales, f32, cells, "k_scales"), self._flat(v_scales, f32, cells, "v_scales"),
                self._flat(block_table, i32, B * maxb, "block_table"), self._flat(seq_lens, i32, B, "seq_lens"))
        if splits == 0:
            splits = self.decode_splits_fp8(B, num_kv_heads, maxb, page_size) if tq == 0 else \
                self.prefill_splits_fp8(B, tq, Hq, num_kv_heads, maxb, page_size)
        if workspace is None:
            workspace = self.workspace_fp8(B * max(tq, 1), Hq, splits)
        if workspace.get_device() != self.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on cuda:{self.device}, the device of this Codec")
        if out is None:
            out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        op = self._flat(out, torch.bfloat16, q.numel(), "out")
        rest = (Hq, num_kv_heads, page_size, maxb, num_blocks, float(sm_scale), splits, workspace.data_ptr(),
                workspace.numel() * workspace.element_size(), op, _raw_stream(self.device))
        if tq == 0:
            native.tq_decode_attention_fp8(self.handle, qp, *args, B, *rest)
        else:
            native.tq_prefill_attention_fp8(self.handle, qp, *args, B, tq, *rest)
        return out

    def decode_attention_fp8(self, q, k_pool, v_pool, k_scales, v_scales, block_table, seq_lens, num_kv_heads: int,
                             page_size: int, num_blocks: int, sm_scale: float, splits: int = 0, workspace=None,
                             out=None, stream=None):
        """Attention of one query token per sequence (q [B, Hq, d] bf16) over its 8-bit pages."""
        if q.dim() != 3:
            raise ValueError("q must be [B, Hq, head_dim]")
        return self._attention_fp8(q, 0, k_pool, v_pool, k_scales, v_scales, block_table, seq_lens, num_kv_heads,
                                   page_size, num_blocks, sm_scale, splits, workspace, out, stream)

    def prefill_attention_fp8(self, q, k_pool, v_pool, k_scales, v_scales, block_table, seq_lens, num_kv_heads: int,
                              page_size: int, num_blocks: int, sm_scale: float, splits: int = 0, workspace=None,
                              out=None, stream=None):
        """Causal attention of the last q.shape[1] positions of every sequence (q [B, Tq, Hq, d] bf16) over its
        8-bit pages."""
        if q.dim() != 4 or q.shape[1] < 1:
            raise ValueError("q must be [B, Tq, Hq, head_dim]")
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
