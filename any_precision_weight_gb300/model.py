"""Loading quantised MoE blocks into a PagedMoE page table, and expert layers with
8-bit floating point weights.

Marshalling only: the packing is pw_pack (C++), the registration is
pw_block_register; this module moves arrays into pinned host memory and
hands the pointers over.
"""
from __future__ import annotations

from typing import NamedTuple

import numpy as np

from . import (KIND_DOWN, KIND_GATE_UP, PagedMoE, _torch, f8_blocks, pw_combine, pw_grouped_linear_f8, pw_lut_bytes,
               pw_pack, pw_quant_f8, pw_quant_f8_blocks, pw_route, pw_silu_quant_f8, pw_tile_planes, rows_f8)


class HostStore:
    """Pinned host backing store carved out of a few large pinned chunks.

    One pinned allocation per block rounds every block up to a power of two
    (about 1.5x the bytes for these shapes) and leaves thousands of small
    pinned regions; chunks of ``chunk_bytes`` hold many blocks each, every
    slice starting on a 256-byte boundary.
    """

    def __init__(self, chunk_bytes: int = 1 << 30):
        self.chunk_bytes = chunk_bytes
        self._chunks = []
        self._cur = None
        self._off = 0

    def alloc(self, nbytes: int):
        """A pinned uint8 CPU tensor of nbytes (a view into a chunk)."""
        import torch
        n = (nbytes + 255) // 256 * 256
        if self._cur is None or self._off + n > self._cur.numel():
            self._cur = torch.empty(max(self.chunk_bytes, n), dtype=torch.uint8, pin_memory=True)
            self._chunks.append(self._cur)
            self._off = 0
        t = self._cur[self._off:self._off + nbytes]
        self._off += n
        return t

    def nbytes(self) -> int:
        return sum(c.numel() for c in self._chunks)


def pack_pinned(P: np.ndarray, parent_lut: np.ndarray, n_bits: int = 8, b_min: int = 3,
                store: HostStore | None = None):
    """pw_pack into pinned torch CPU tensors (planes as int32 in the device page
    layout of pw_tile_planes, tables as int16), from ``store`` if given, else one
    pinned allocation each."""
    import torch
    R, K = P.shape
    pb = n_bits * R * (K // 32) * 4
    lb = pw_lut_bytes(R, b_min, n_bits)
    if store is None:
        planes = torch.empty((n_bits, R, K // 32), dtype=torch.int32, pin_memory=True)
        luts = torch.empty(lb // 2, dtype=torch.int16, pin_memory=True)
    else:
        planes = store.alloc(pb).view(torch.int32).view(n_bits, R, K // 32)
        luts = store.alloc(lb).view(torch.int16)
    flat, _ = pw_pack(P, parent_lut, n_bits, b_min, luts_out=luts.numpy().view(np.uint16))
    pw_tile_planes(flat, out=planes.numpy().view(np.uint32).reshape(-1))
    return planes, luts


def load_expert_layer(moe: PagedMoE, layer: int, blocks, bits, n_bits: int = 8, b_min: int = 3,
                      alloc_planes=None, stream=None, store: HostStore | None = None,
                      per_plane: bool = False):
    """Registers every block of one layer.

    blocks(e, kind) -> (P uint8 [R][K], parent_lut fp16 [R][2^n]);
    bits[e][kind] -> committed bitwidth; alloc_planes(e, kind) -> device pages
    to allocate (default: all n planes); store -> where the pinned host copies
    live (default: one pinned allocation per array).
    """
    for e in range(moe.E):
        for kind in (KIND_GATE_UP, KIND_DOWN):
            P, par = blocks(e, kind)
            planes, luts = pack_pinned(P, par, n_bits, b_min, store=store)
            na = None if alloc_planes is None else alloc_planes(e, kind)
            moe.register(layer, e, kind, planes, luts, int(bits[e][kind]), n_bits=n_bits,
                         b_min=b_min, alloc_planes=na, stream=stream, per_plane=per_plane)


class F8Stages(NamedTuple):
    """What the stages of an F8Experts forward wrote, rows in expert order."""
    routing: object
    q: object           # tokens as e4m3
    scale: object
    up: object          # gate and up rows' product
    act: object         # silu(gate) * up as e4m3
    act_scale: object
    y: object           # down rows' product


class F8Experts:
    """An expert layer whose weights are e4m3 with a scale for each block of 128 x
    128, as fp8 checkpoints hold them: the counterpart of a PagedMoE layer.

    gate_up [E][2 I][H] (gate rows, then up rows) and down [E][H][I]: e4m3 with their
    scales [E][blocks of rows][blocks of columns] float32 and rows on 16-byte
    boundaries, or 16- or 32-bit weights, which are then quantised here.  Scales of gate
    and up that were made apart fit only where I is a multiple of 128: the blocks of 128
    rows are counted through the joined rows.
    """

    def __init__(self, gate_up, down, gate_up_scale=None, down_scale=None):
        self.E, two_i, self.H = gate_up.shape
        self.I = two_i // 2
        if two_i % 2 or tuple(down.shape) != (self.E, self.H, self.I):
            raise ValueError(f"weights [E][2 I][H] and [E][H][I] are needed, got {tuple(gate_up.shape)} and {tuple(down.shape)}")
        self.gate_up, self.gate_up_scale = self._weights(gate_up, gate_up_scale)
        self.down, self.down_scale = self._weights(down, down_scale)

    @staticmethod
    def _weights(w, scale):
        torch = _torch()
        if w.dtype is torch.float8_e4m3fn:
            if scale is None:
                raise ValueError("e4m3 weights need their scales")
            return w, scale
        E, N, K = w.shape
        q = rows_f8(E, N, K, device=w.device)
        scale = torch.empty(E, f8_blocks(N), f8_blocks(K), dtype=torch.float32, device=w.device)
        for e in range(E):
            pw_quant_f8_blocks(w[e], q=q[e], scale=scale[e])
        return q, scale

    def forward(self, x, logits, top_k: int, renorm: bool, residual=None, out=None, stream=None, trace: bool = False):
        """residual + the weighted sum of the top_k experts of every token: x [T][H] of
        16 or 32 bits, logits [T][E] float32.  Six launches (seven for a large batch's
        routing) on the stream, which nothing waits for; can be captured into a CUDA
        graph.  trace: returns (out, F8Stages)."""
        r = pw_route(logits, top_k, renorm, stream=stream)
        q, s = pw_quant_f8(x, rows=r.perm, per=top_k, stream=stream)
        up = pw_grouped_linear_f8(q, s, self.gate_up, self.gate_up_scale, r.offsets, out_dtype=x.dtype, stream=stream)
        a, sa = pw_silu_quant_f8(up, stream=stream)
        y = pw_grouped_linear_f8(a, sa, self.down, self.down_scale, r.offsets, out_dtype=x.dtype, stream=stream)
        out = pw_combine(y, r.weight, r.inv, residual=residual, out=out, out_dtype=x.dtype, stream=stream)
        return (out, F8Stages(r, q, s, up, a, sa, y)) if trace else out
