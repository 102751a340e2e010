"""Thin Python binding of libpw.so, the fused mixed-precision APL MoE layer
for GB300 (sm_103a).

The functions keep the C ABI's names (pw_pack, pw_set_commit, pw_reload_async,
pw_moe_forward, ...) and only marshal arguments: torch tensors become raw
pointers, the current torch stream becomes the CUDA stream.  Every step of the
layer runs in the library's own kernels; there is no fallback path, and every
entry point raises if the library has not been built.

PyTorch supplies device memory (plane pages, tables, descriptors, workspace)
and streams; the library allocates none of its own.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpw.so")
CHECK_LIB_PATH = os.path.join(HERE, "libpw_check.so")

PW_OK = 0
PW_EINVAL = -1
PW_ECUDA = -2
PW_ENOTRESIDENT = -3
PW_ERELOAD = -4
PW_ETIMEOUT = -5
PW_ENOMEM = -6
PW_EDEVICE = -7
PW_STATUS_NAN_LOGIT = 1
PW_STATUS_TIMEOUT = 2
PW_STATUS_BAD_DESC = 4
PW_STATUS_BOUNDS = 8
PW_WS_H, PW_WS_Y = 0, 1
PW_PLANE_HOST, PW_PLANE_HOST_PAGED, PW_PLANE_MOVING, PW_PLANE_DEVICE = 0, 1, 2, 3
KIND_GATE_UP = 0
KIND_DOWN = 1
MAX_BITS = 8
PW_F16, PW_BF16, PW_F32 = 0, 1, 2
MAX_K_I8 = 131071
MAX_TOP = 32
MAX_GROUPS = 512
F8_BLOCK = 128   # columns, and rows of weights, that share a scale

_lib = None

_sz = ctypes.c_size_t
_vp = ctypes.c_void_p
_i = ctypes.c_int
_i64 = ctypes.c_int64
_pi = ctypes.POINTER(ctypes.c_int)

_SIGS = {
    "pw_last_error": (ctypes.c_char_p, []),
    "pw_plane_bytes": (_sz, [_i, _i]),
    "pw_lut_bytes": (_sz, [_i, _i, _i]),
    "pw_lut_offset": (_sz, [_i, _i, _i]),
    "pw_pack": (_i, [_vp, _i, _i, _i, _vp, _i, _vp, _vp]),
    "pw_tile_planes": (_i, [_vp, _i, _i, _i, _vp]),
    "pw_desc_bytes": (_sz, [_i, _i]),
    "pw_table_create": (_i, [ctypes.POINTER(_vp), _i, _i, _i, _i, _vp, _sz, _vp]),
    "pw_block_register": (_i, [_vp, _i, _i, _i, _i, _i, _vp, _vp, ctypes.POINTER(_vp), _vp, _i, _vp]),
    "pw_set_commit": (_i, [_vp, _i, _i, _i, _i, _vp]),
    "pw_reload_async": (_i, [_vp, _i, _i, _i, _i, _vp]),
    "pw_reload_query": (_i, [_vp, _i, _i, _i]),
    "pw_reload_many": (_i, [_vp, _i, _pi, _pi, _pi, _pi, _vp, _pi]),
    "pw_set_commit_many": (_i, [_vp, _i, _pi, _pi, _pi, _pi, _vp]),
    "pw_mover_start": (_i, [_vp, _vp, _sz]),
    "pw_mover_submit": (_i, [_vp, _i, _pi, _pi, _pi, _pi]),
    "pw_commit_arrived": (_i, [_vp, _vp, _pi, _pi]),
    "pw_block_state": (_i, [_vp, _i, _i, _i, _pi, _pi, _pi]),
    "pw_table_destroy": (_i, [_vp]),
    "pw_debug_fail_next_reload": (_i, [_vp]),
    "pw_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "pw_workspace_offset": (_sz, [_i, _i, _i, _i, _i, _i]),
    "pw_moe_forward": (_i, [_vp, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "pw_moe_forward_host": (_i, [_vp, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _sz, _vp]),
    "pw_workspace_status": (_i, [_vp, _vp, _pi]),
    "pw_moe_forward_noalloc": (_i, [_vp, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _vp]),
    "pw_noalloc_status": (_i, [_vp, _pi]),
    "pw_profile_attach": (_i, [ctypes.POINTER(_vp), _i]),
    "pw_stats_attach": (_i, [_vp, _vp, ctypes.c_float]),
    "pw_plan_bits": (_i, [_i, _vp, _vp, _vp, _vp, _vp, _i, ctypes.c_double, _i, _i, _i, ctypes.c_double,
                          _vp, ctypes.POINTER(ctypes.c_int64)]),
    "pw_plan_apply": (_i, [_vp, _vp, _vp, _pi, _pi]),
    "pw_block_release": (_i, [_vp, _i, _i, _i, _i, ctypes.POINTER(_vp)]),
    "pw_block_attach_pages": (_i, [_vp, _i, _i, _i, ctypes.POINTER(_vp)]),
    "pw_plane_states": (_i, [_vp, _i, _i, _i, _pi]),
    "pw_rms_norm": (_i, [_vp, _i64, _vp, _i64, _vp, ctypes.c_float, _i, _i, _i, _vp, _i64, _vp, _i64, _vp, _i64,
                         _vp, _vp]),
    "pw_quant_i8": (_i, [_vp, _i64, _i, _i, _i, _vp, _i64, _vp, _vp]),
    "pw_linear_i8": (_i, [_vp, _i64, _vp, _vp, _i64, _vp, _vp, _i, _i, _i, _i, _vp, _i64, _vp, _sz,
                          _vp]),
    "pw_linear_i8_workspace_bytes": (_sz, [_i, _i]),
    "pw_linear_i8_status": (_i, [_vp, _pi]),
    "pw_debug_linear_timeout": (_i, [_vp]),
    "pw_logprobs": (_i, [_vp, _i64, _i, _i, _i, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
    "pw_route": (_i, [_vp, _i64, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
    "pw_quant_f8": (_i, [_vp, _i64, _i64, _vp, _i, _i, _i, _i, _vp, _i64, _vp, _i64, _vp]),
    "pw_silu_quant_f8": (_i, [_vp, _i64, _i, _i, _i, _vp, _i64, _vp, _i64, _vp]),
    "pw_quant_f8_blocks": (_i, [_vp, _i64, _i, _i, _i, _vp, _i64, _vp, _i64, _vp]),
    "pw_linear_f8": (_i, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i, _i, _i, _i, _vp, _i64, _vp]),
    "pw_grouped_linear_f8": (_i, [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i, _i, _i, _i,
                                  _i, _vp, _i64, _vp]),
    "pw_linear_f8_status": (_i, [_vp, _pi]),
    "pw_debug_linear_f8_timeout": (_i, [_vp]),
    "pw_debug_linear_f8": (_i, [_i, _i, _i, _i, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i, _i,
                                _i, _i, _i, _vp, _i64, _vp]),
    "pw_combine": (_i, [_vp, _i64, _i64, _i, _vp, _vp, _vp, _i64, _i, _i, _i, _i, _vp, _i64, _vp]),
}


class PWError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{msg} (status {code})")
        self.code = code


def lib():
    """Loads libpw.so (once).  Raises if it has not been built.  With the
    environment variable PW_CHECK=1, loads libpw_check.so instead: the same
    library with device-side bounds checks that set PW_STATUS_BOUNDS."""
    global _lib
    if _lib is None:
        path = CHECK_LIB_PATH if os.environ.get("PW_CHECK") == "1" else LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it first "
                               "(python -m any_precision_weight_gb300.build)")
        L = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def exported_symbols():
    return sorted(_SIGS)


def _check(rc: int, what: str) -> int:
    if rc < 0:
        raise PWError(rc, f"{what}: {lib().pw_last_error().decode()}")
    return rc


def _ptr(t):
    """Address of a torch tensor or numpy array (None stays NULL)."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _empty(torch, stream, shape, dtype, device):
    """Uninitialised memory of the stream that a call writes it on: a block of
    another stream's pool may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


# ----------------------------------------------------------------------------- format

def pw_plane_bytes(R: int, K: int) -> int:
    return lib().pw_plane_bytes(R, K)


def pw_lut_bytes(R: int, b_min: int, n_bits: int) -> int:
    return lib().pw_lut_bytes(R, b_min, n_bits)


def pw_lut_offset(R: int, b_min: int, b: int) -> int:
    return lib().pw_lut_offset(R, b_min, b)


def pw_pack(idx: np.ndarray, parent_lut: np.ndarray, n_bits: int = 8, b_min: int = 3,
            planes_out=None, luts_out=None):
    """Packs uint8 parent indices [R][K] and the fp16 parent table [R][2^n].

    Returns (planes uint32 [n][R][K/32], luts uint16 flat) as numpy arrays, or
    fills the given host buffers (numpy arrays over any host memory).
    """
    idx = np.ascontiguousarray(idx, dtype=np.uint8)
    par = np.ascontiguousarray(parent_lut, dtype=np.float16).view(np.uint16)
    R, K = idx.shape
    if planes_out is None:
        planes_out = np.empty((n_bits, R, K // 32), dtype=np.uint32)
    if luts_out is None:
        luts_out = np.empty(pw_lut_bytes(R, b_min, n_bits) // 2, dtype=np.uint16)
    _check(lib().pw_pack(_ptr(idx), R, K, n_bits, _ptr(par), b_min, _ptr(planes_out),
                         _ptr(luts_out)), "pw_pack")
    return planes_out, luts_out


def pw_tile_planes(planes: np.ndarray, out=None):
    """Reorders pw_pack planes uint32 [n][R][K/32] into the device page layout
    (returned as a flat uint32 array of the same size, or written into ``out``)."""
    planes = np.ascontiguousarray(planes, dtype=np.uint32)
    n, R, W = planes.shape
    if out is None:
        out = np.empty(planes.size, dtype=np.uint32)
    _check(lib().pw_tile_planes(_ptr(planes), n, R, W * 32, _ptr(out)), "pw_tile_planes")
    return out


def pw_profile_attach(events):
    """Next pw_moe_forward on this thread records these 5 torch.cuda.Events at its
    kernel boundaries (before routing, after routing, gate_up, down, combine);
    None entries are not recorded.  The decode path is one kernel: it records
    events[0] before it and events[1..4] after it."""
    if not events:
        return lib().pw_profile_attach(None, 0)
    arr = (_vp * len(events))(*[e.cuda_event if e is not None else None for e in events])
    return _check(lib().pw_profile_attach(arr, len(events)), "pw_profile_attach")


# ----------------------------------------------------------------------------- page table

def pw_plan_bits(R, K, sens, mass, n_experts, hot_mass, hot_floor, target_bytes, resid=None,
                 b_min: int = 3, n_bits: int = MAX_BITS):
    """The native planner on host arrays (one entry per block).  Returns
    (bits int32 array, resident bytes of the plan)."""
    R = np.ascontiguousarray(R, dtype=np.int32)
    K = np.ascontiguousarray(K, dtype=np.int32)
    sens = np.ascontiguousarray(sens, dtype=np.float64)
    mass = np.ascontiguousarray(mass, dtype=np.float64)
    rs = None if resid is None else np.ascontiguousarray(resid, dtype=np.float64)
    out = np.empty(len(R), dtype=np.int32)
    res = ctypes.c_int64()
    _check(lib().pw_plan_bits(len(R), _ptr(R), _ptr(K), _ptr(sens), _ptr(rs), _ptr(mass), int(n_experts),
                              float(hot_mass), int(hot_floor), int(b_min), int(n_bits), float(target_bytes),
                              _ptr(out), ctypes.byref(res)), "pw_plan_bits")
    return out, res.value


class PagedMoE:
    """Owns the device memory of one model's MoE blocks and the C page table.

    Plane pages, tables and descriptors are torch CUDA tensors; host backing
    copies are pinned torch CPU tensors.  Only the pages a block may use
    (``alloc_planes``) are allocated on the device.
    """

    def __init__(self, n_layers: int, n_experts: int, H: int, I: int, device="cuda", stream=None,
                 guard: int = 0):
        """guard > 0: every device buffer this object allocates (descriptors,
        plane pages, tables, workspaces) gets canary regions of that many bytes
        on both sides (``guard.GuardSet``), checked by ``corrupted_guards``."""
        import torch
        from .guard import GuardSet
        self.L, self.E, self.H, self.I = n_layers, n_experts, H, I
        self.device = torch.device(device)
        self.guards = GuardSet(guard) if guard > 0 else None
        nb = lib().pw_desc_bytes(n_layers, n_experts)
        self._desc = self._alloc(nb + 128, "descriptors")
        self._desc.zero_()
        base = self._desc.data_ptr()
        self._desc_ptr = base + ((-base) % 128)
        h = _vp()
        _check(lib().pw_table_create(ctypes.byref(h), n_layers, n_experts, H, I, self._desc_ptr, nb,
                                     _stream(stream)), "pw_table_create")
        self._t = h
        self._keep = {}

    def _alloc(self, nbytes: int, name: str, stream=None):
        """Device memory of the given stream, or of the current one."""
        import torch
        if stream is not None:
            with torch.cuda.stream(stream):
                return self._alloc(nbytes, name)
        if self.guards is None:
            return torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        return self.guards.alloc(nbytes, self.device, name)

    def corrupted_guards(self) -> list:
        """Guard regions changed since allocation: [(buffer, side, offset)]."""
        return [] if self.guards is None else self.guards.corrupted()

    def rows_cols(self, kind: int):
        return (2 * self.I, self.H) if kind == KIND_GATE_UP else (self.H, self.I)

    def register(self, layer: int, expert: int, kind: int, planes_host, luts_host, q_init: int,
                 n_bits: int = 8, b_min: int = 3, alloc_planes: int | None = None, stream=None,
                 per_plane: bool = False):
        """planes_host / luts_host: pinned torch CPU tensors (or numpy arrays) in
        pw_pack layout; kept alive by this object.  per_plane: one device
        tensor per plane (so released planes free their memory) instead of one
        tensor for all of the block's pages."""
        import torch
        R, K = self.rows_cols(kind)
        pb = pw_plane_bytes(R, K)
        na = n_bits if alloc_planes is None else max(q_init, min(alloc_planes, n_bits))
        tag = f"{layer}/{expert}/{kind}"
        luts = self._alloc(pw_lut_bytes(R, b_min, n_bits), f"tables {tag}")
        if per_plane:
            pages = [self._alloc(pb, f"plane {p} {tag}") if p < na else None for p in range(n_bits)]
            ptrs = (_vp * n_bits)(*[pg.data_ptr() if pg is not None else None for pg in pages])
        else:
            pages = self._alloc(na * pb, f"planes {tag}")
            ptrs = (_vp * n_bits)(*[pages.data_ptr() + p * pb if p < na else None for p in range(n_bits)])
        _check(lib().pw_block_register(self._t, layer, expert, kind, n_bits, b_min, _ptr(planes_host),
                                       _ptr(luts_host), ptrs, luts.data_ptr(), q_init, _stream(stream)),
               "pw_block_register")
        self._keep[(layer, expert, kind)] = (pages, luts, planes_host, luts_host)

    def pages(self, layer, expert, kind):
        """(device plane pages tensor, device table tensor) of one block."""
        return self._keep[(layer, expert, kind)][:2]

    def device_bytes(self) -> int:
        def nb(pages):
            if isinstance(pages, list):
                return sum(p.numel() for p in pages if p is not None)
            return pages.numel()
        return sum(nb(v[0]) + v[1].numel() for v in self._keep.values())

    def pw_block_release(self, layer, expert, kind, keep, stream=None):
        """Offloads planes [keep, n) of a block.  Per-plane blocks drop their
        page tensors once the stream has passed every earlier forward.
        Returns the released device addresses (None where none)."""
        import torch
        out = (_vp * MAX_BITS)()
        _check(lib().pw_block_release(self._t, layer, expert, kind, keep, out), "pw_block_release")
        rel = [out[p] for p in range(MAX_BITS)]
        pages = self._keep[(layer, expert, kind)][0]
        if isinstance(pages, list) and any(rel):
            (stream or torch.cuda.current_stream()).synchronize()
            for p in range(MAX_BITS):
                if rel[p] and p < len(pages):
                    pages[p] = None
        return rel

    def pw_block_attach_pages(self, layer, expert, kind):
        """Gives a per-plane block fresh device pages for every plane without one."""
        import torch
        pages = self._keep[(layer, expert, kind)][0]
        assert isinstance(pages, list), "attach_pages needs a block registered with per_plane=True"
        R, K = self.rows_cols(kind)
        pb = pw_plane_bytes(R, K)
        new = [None] * MAX_BITS
        for p in range(len(pages)):
            if pages[p] is None:
                new[p] = self._alloc(pb, f"plane {p} {layer}/{expert}/{kind} (attached)")
        ptrs = (_vp * MAX_BITS)(*[t.data_ptr() if t is not None else None for t in new])
        _check(lib().pw_block_attach_pages(self._t, layer, expert, kind, ptrs), "pw_block_attach_pages")
        for p in range(len(pages)):
            if new[p] is not None:
                pages[p] = new[p]

    def pw_plane_states(self, layer, expert, kind):
        st = (_i * MAX_BITS)()
        _check(lib().pw_plane_states(self._t, layer, expert, kind, st), "pw_plane_states")
        return [st[p] for p in range(MAX_BITS)]

    def pw_set_commit(self, layer, expert, kind, q, stream=None):
        return _check(lib().pw_set_commit(self._t, layer, expert, kind, q, _stream(stream)),
                      "pw_set_commit")

    def pw_reload_async(self, layer, expert, kind, q_target, stream=None):
        return _check(lib().pw_reload_async(self._t, layer, expert, kind, q_target, _stream(stream)),
                      "pw_reload_async")

    @staticmethod
    def _columns(items):
        """[(layer, expert, kind, q), ...] -> four ctypes int arrays."""
        n = len(items)
        cols = [(ctypes.c_int * n)(*[int(it[j]) for it in items]) for j in range(4)]
        return n, cols

    def pw_reload_many(self, items, stream=None):
        """items: [(layer, expert, kind, q_target)].  Returns the number enqueued;
        raises PWError on the first failing block."""
        n, (l, e, k, q) = self._columns(items)
        done = _i()
        rc = lib().pw_reload_many(self._t, n, l, e, k, q, _stream(stream), ctypes.byref(done))
        _check(rc, "pw_reload_many")
        return done.value

    def pw_set_commit_many(self, items, stream=None):
        """items: [(layer, expert, kind, q)], committed at one stream boundary."""
        n, (l, e, k, q) = self._columns(items)
        return _check(lib().pw_set_commit_many(self._t, n, l, e, k, q, _stream(stream)),
                      "pw_set_commit_many")

    def pw_mover_start(self, stream, max_inflight_bytes: int = 64 << 20):
        """Starts the table's reload mover thread on the given copy stream."""
        return _check(lib().pw_mover_start(self._t, _stream(stream), max_inflight_bytes),
                      "pw_mover_start")

    def pw_mover_submit(self, items):
        """items: [(layer, expert, kind, q_target)], reloaded in order and
        committed by pw_commit_arrived once landed."""
        n, (l, e, k, q) = self._columns(items)
        return _check(lib().pw_mover_submit(self._t, n, l, e, k, q), "pw_mover_submit")

    def pw_commit_arrived(self, stream=None):
        """Commits every landed mover reload; returns (committed, outstanding)."""
        c, o = _i(), _i()
        _check(lib().pw_commit_arrived(self._t, _stream(stream), ctypes.byref(c), ctypes.byref(o)),
               "pw_commit_arrived")
        return c.value, o.value

    def pw_stats_attach(self, stats=None, alpha: float = 0.05):
        """Attaches a float32 CUDA tensor [L][E] of routing-mass moving averages
        (updated by every forward), or detaches with None."""
        if stats is not None:
            import torch
            assert stats.dtype == torch.float32 and stats.is_contiguous()
            assert stats.numel() == self.L * self.E
        self._stats = stats
        return _check(lib().pw_stats_attach(self._t, _ptr(stats), float(alpha)), "pw_stats_attach")

    def pw_plan_apply(self, desired, stream=None):
        """desired: int array [L][E][2] (0 = leave alone).  Returns (committed now,
        handed to the mover)."""
        d = np.ascontiguousarray(desired, dtype=np.int32).reshape(-1)
        assert d.size == self.L * self.E * 2
        a, b = _i(), _i()
        _check(lib().pw_plan_apply(self._t, _ptr(d), _stream(stream), ctypes.byref(a), ctypes.byref(b)),
               "pw_plan_apply")
        return a.value, b.value

    def pw_reload_query(self, layer, expert, kind) -> int:
        return _check(lib().pw_reload_query(self._t, layer, expert, kind), "pw_reload_query")

    def pw_block_state(self, layer, expert, kind):
        q, res, tgt = _i(), _i(), _i()
        _check(lib().pw_block_state(self._t, layer, expert, kind, ctypes.byref(q), ctypes.byref(res),
                                    ctypes.byref(tgt)), "pw_block_state")
        return q.value, res.value, tgt.value

    def pw_debug_fail_next_reload(self):
        return _check(lib().pw_debug_fail_next_reload(self._t), "pw_debug_fail_next_reload")

    def workspace_h(self, ws, T: int, top_k: int):
        """h (fp16 [T*top_k][I], permuted pair order) left in `ws` by the last forward."""
        import torch
        off = lib().pw_workspace_offset(T, self.E, top_k, self.H, self.I, PW_WS_H)
        n = T * top_k * self.I * 2
        return ws[off:off + n].view(torch.float16).view(T * top_k, self.I)

    def workspace_y(self, ws, T: int, top_k: int):
        """y (fp32 [T*top_k][H], permuted pair order) left in `ws` by the last forward."""
        import torch
        off = lib().pw_workspace_offset(T, self.E, top_k, self.H, self.I, PW_WS_Y)
        n = T * top_k * self.H * 4
        return ws[off:off + n].view(torch.float32).view(T * top_k, self.H)

    def workspace(self, T: int, top_k: int, stream=None):
        nb = lib().pw_workspace_bytes(T, self.E, top_k, self.H, self.I)
        return self._alloc(max(nb, 256), f"workspace T={T}", stream)

    def pw_moe_forward(self, layer, x, logits, top_k, renorm, residual=None, out=None, ws=None,
                       routing=False, stream=None):
        """x [T][H] fp16 and logits [T][E] fp32 CUDA tensors.  Returns out, or
        (out, topk_idx, topk_w, offsets, perm) with routing=True."""
        import torch
        T = x.shape[0]
        assert x.dtype == torch.float16 and logits.dtype == torch.float32
        assert x.is_contiguous() and logits.is_contiguous()
        if out is None:
            out = _empty(torch, stream, x.shape, x.dtype, x.device)
        if ws is None:
            ws = self.workspace(T, top_k, stream)
        ri = rw = ro = rp = None
        if routing:
            ri = _empty(torch, stream, (T, top_k), torch.int32, x.device)
            rw = _empty(torch, stream, (T, top_k), torch.float32, x.device)
            ro = _empty(torch, stream, (self.E + 1,), torch.int32, x.device)
            rp = _empty(torch, stream, (T * top_k,), torch.int32, x.device)
        _check(lib().pw_moe_forward(self._t, layer, _ptr(x), _ptr(logits), T, top_k, int(renorm),
                                    _ptr(residual), _ptr(out), _ptr(ri), _ptr(rw), _ptr(ro), _ptr(rp),
                                    _ptr(ws), ws.numel(), _stream(stream)), "pw_moe_forward")
        return (out, ri, rw, ro, rp) if routing else out

    def pw_moe_forward_host(self, layer, x_host, logits_host, top_k, renorm, out_host,
                            residual_host=None, ws=None, stream=None):
        """Host (pinned) inputs and output; synchronises the stream."""
        T = x_host.shape[0]
        if ws is None:
            ws = self.workspace(T, top_k, stream)
        _check(lib().pw_moe_forward_host(self._t, layer, _ptr(x_host), _ptr(logits_host), T, top_k,
                                         int(renorm), _ptr(residual_host), _ptr(out_host), _ptr(ws),
                                         ws.numel(), _stream(stream)), "pw_moe_forward_host")
        return out_host

    def pw_moe_forward_noalloc(self, layer, x, logits, top_k, renorm, residual=None, out=None,
                               stream=None):
        """pw_moe_forward without a caller workspace: the library's fixed 8 MiB
        device scratch is used instead (for callers that cannot allocate).
        Calls that overlap on the GPU race on that scratch."""
        import torch
        assert x.dtype == torch.float16 and logits.dtype == torch.float32
        if out is None:
            out = _empty(torch, stream, x.shape, x.dtype, x.device)
        _check(lib().pw_moe_forward_noalloc(self._t, layer, _ptr(x), _ptr(logits), x.shape[0], top_k,
                                            int(renorm), _ptr(residual), _ptr(out), _stream(stream)),
               "pw_moe_forward_noalloc")
        return out

    @staticmethod
    def workspace_status(ws, stream=None) -> int:
        st = _i()
        _check(lib().pw_workspace_status(_ptr(ws), _stream(stream), ctypes.byref(st)),
               "pw_workspace_status")
        return st.value

    @staticmethod
    def noalloc_status(stream=None) -> int:
        """Status bits of the last pw_moe_forward_noalloc ordered before `stream`'s work."""
        st = _i()
        _check(lib().pw_noalloc_status(_stream(stream), ctypes.byref(st)), "pw_noalloc_status")
        return st.value

    def close(self):
        if getattr(self, "_t", None):
            lib().pw_table_destroy(self._t)
            self._t = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ----------------------------------------------------------------------------- operators around the layer

# Each call runs on `stream` (default: the current one) of the current device, which
# holds every operand; anything else is refused before a launch.  Outputs and workspaces
# that it makes itself are that stream's memory; one that is used on another
# stream than its own has to be ordered, and recorded, by the caller.

_torch_mod = None
_codes = {}
_devices = 1   # GPUs of the process, once torch is known


def _torch():
    """torch, imported at the first call that needs it (and the C ABI's codes
    of its element types)."""
    global _torch_mod, _devices
    if _torch_mod is None:
        import torch
        _devices = torch.cuda.device_count()
        _codes.update({torch.float16: PW_F16, torch.bfloat16: PW_BF16, torch.float32: PW_F32})
        _torch_mod = torch
    return _torch_mod


def _code(dtype) -> int:
    """The C ABI's code of a torch element type."""
    try:
        return _codes[dtype]
    except KeyError:
        raise TypeError(f"{dtype}: float16, bfloat16 or float32 is needed") from None


def _place(torch, t, name: str, stream):
    """(device index, raw stream) of a call whose first operand is t: on the current
    device, where the library launches, and the given stream or the current one
    (looked up without building a Stream object, which costs more than a launch).
    None for the index where there is one GPU: every CUDA tensor is on it, and to
    ask each for its index costs 0.4 us a call."""
    if not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is needed, got one on {t.device}")
    dev = None
    if _devices > 1:
        dev, now = t.get_device(), torch._C._cuda_getDevice()
        if dev != now:
            raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{now}")
        if stream is not None and stream.device_index != dev:
            raise ValueError(f"{name}: on {t.device}, but the stream is one of cuda:{stream.device_index}")
    return dev, torch._C._cuda_getCurrentRawStream(dev or 0) if stream is None else stream.cuda_stream


def _away(t, dev) -> bool:
    """Whether t is not on the call's device (dev None: the only GPU)."""
    return not t.is_cuda or (dev is not None and t.get_device() != dev)


def _rows(t, name: str, dtype, shape, dev):
    """Row stride of a matrix on the call's device whose rows are consecutive elements."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {dtype} is needed, got {t.dtype}")
    if t.shape != shape or not t.is_cuda or (dev is not None and t.get_device() != dev):
        raise ValueError(f"{name}: a matrix of shape {tuple(shape)} on the call's GPU is needed, "
                         f"got {tuple(t.shape)} on {t.device}")
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the elements of a row must be consecutive")
    # a row alone has no stride of its own
    return ld if shape[0] > 1 else (shape[1] + 15) // 16 * 16


def _matrix(t, name: str):
    """(rows, columns) of a matrix."""
    if t.dim() != 2:
        raise ValueError(f"{name}: a matrix is needed, got {t.dim()} dimensions")
    return t.shape


def _vec(t, name: str, dtype, n: int, dev):
    if (t.dtype is not dtype or not t.is_cuda or t.shape != (n,) or not t.is_contiguous()
            or (dev is not None and t.get_device() != dev)):
        raise ValueError(f"{name}: a contiguous vector of {n} {dtype} on the call's GPU is needed")
    return t.data_ptr()


def rows_i8(T: int, K: int, device="cuda", stream=None):
    """An uninitialised int8 matrix [T][K] whose rows start on 16-byte
    boundaries, as pw_linear_i8 wants them (a view of a padded one), in memory
    of the given stream or the current one."""
    torch = _torch()
    return _empty(torch, stream, (T, (K + 15) // 16 * 16), torch.int8, device)[:, :K]


def _norm(torch, dev, raw, what, x, shape, weight, eps, residual, sum_out, y, q, scale):
    dt = x.dtype
    pr = ps = py = pq = pc = None
    lr = ls = ly = lq = 0
    lx = _rows(x, "x", dt, shape, dev)
    if residual is not None:
        lr, pr = _rows(residual, "residual", dt, shape, dev), residual.data_ptr()
    if sum_out is not None:
        ls, ps = _rows(sum_out, "sum_out", dt, shape, dev), sum_out.data_ptr()
    if y is not None:
        ly, py = _rows(y, "out", dt, shape, dev), y.data_ptr()
    if q is not None:
        lq, pq = _rows(q, "q", torch.int8, shape, dev), q.data_ptr()
        pc = _vec(scale, "scale", torch.float32, shape[0], dev)
    _check(lib().pw_rms_norm(x.data_ptr(), lx, pr, lr, _vec(weight, "weight", dt, shape[1], dev), eps, shape[0],
                             shape[1], _code(dt), ps, ls, py, ly, pq, lq, pc, raw), what)


def pw_rms_norm(x, weight, eps: float = 1e-6, residual=None, out=None, sum_out=None, stream=None):
    """Root-mean-square norm of the rows of x (+ residual).  Returns out, or
    (out, sum_out) with a residual; sum_out (the new residual stream) may be
    the residual itself."""
    torch = _torch()
    shape, (dev, raw) = _matrix(x, "x"), _place(torch, x, "x", stream)
    if out is None:
        out = _empty(torch, stream, shape, x.dtype, x.device)
    if residual is not None and sum_out is None:
        sum_out = _empty(torch, stream, shape, x.dtype, x.device)
    _norm(torch, dev, raw, "pw_rms_norm", x, shape, weight, eps, residual, sum_out, out, None, None)
    return out if residual is None else (out, sum_out)


def pw_rms_norm_i8(x, weight, eps: float = 1e-6, residual=None, q=None, scale=None, out=None, sum_out=None,
                   stream=None):
    """pw_rms_norm with an int8 output and a scale per row: the input of
    pw_linear_i8.  ``out`` also receives the unquantised norm if given.
    Returns (q, scale), or (q, scale, sum_out) with a residual."""
    torch = _torch()
    shape, (dev, raw) = _matrix(x, "x"), _place(torch, x, "x", stream)
    if q is None:
        q = rows_i8(*shape, x.device, stream)
    if scale is None:
        scale = _empty(torch, stream, (shape[0],), torch.float32, x.device)
    if residual is not None and sum_out is None:
        sum_out = _empty(torch, stream, shape, x.dtype, x.device)
    _norm(torch, dev, raw, "pw_rms_norm_i8", x, shape, weight, eps, residual, sum_out, out, q, scale)
    return (q, scale) if residual is None else (q, scale, sum_out)


def pw_quant_i8(x, q=None, scale=None, stream=None):
    """(q, scale): the rows of x as int8 with one scale per row."""
    torch = _torch()
    shape, (dev, raw) = _matrix(x, "x"), _place(torch, x, "x", stream)
    T, K = shape
    if q is None:
        q = rows_i8(T, K, x.device, stream)
    if scale is None:
        scale = _empty(torch, stream, (T,), torch.float32, x.device)
    _check(lib().pw_quant_i8(x.data_ptr(), _rows(x, "x", x.dtype, shape, dev), T, K, _code(x.dtype), q.data_ptr(),
                             _rows(q, "q", torch.int8, shape, dev), _vec(scale, "scale", torch.float32, T, dev),
                             raw), "pw_quant_i8")
    return q, scale


def pw_linear_i8(x, x_scale, w, w_scale, bias=None, out=None, out_dtype=None, ws=None, stream=None):
    """out [T][N] = (x . w^T) * x_scale[t] * w_scale[n] + bias[n], x [T][K] and
    w [N][K] int8 with 16-byte aligned rows (rows_i8), the sum exact.  out has
    type out_dtype (default float16) where it is not given.  ws: a uint8
    workspace of pw_linear_i8_workspace_bytes(T, K) bytes (allocated here where
    it is needed and not given)."""
    torch = _torch()
    T, K = _matrix(x, "x")
    N, (dev, raw) = _matrix(w, "w")[0], _place(torch, x, "x", stream)
    if out is None:
        out = _empty(torch, stream, (T, N), out_dtype or torch.float16, x.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"pw_linear_i8: out is {out.dtype}, not {out_dtype}")
    dt, f32, i8 = out.dtype, torch.float32, torch.int8
    L = lib()
    if ws is None:
        need = L.pw_linear_i8_workspace_bytes(T, K)
        if need:
            ws = _empty(torch, stream, (need,), torch.uint8, x.device)
    elif ws.dtype is not torch.uint8 or not ws.is_contiguous() or _away(ws, dev):
        raise ValueError(f"ws: a contiguous uint8 tensor on the call's GPU is needed, got {ws.dtype} on {ws.device}")
    _check(L.pw_linear_i8(x.data_ptr(), _rows(x, "x", i8, (T, K), dev), _vec(x_scale, "x_scale", f32, T, dev),
                          w.data_ptr(), _rows(w, "w", i8, (N, K), dev), _vec(w_scale, "w_scale", f32, N, dev),
                          None if bias is None else _vec(bias, "bias", dt, N, dev), T, N, K, _code(dt),
                          out.data_ptr(), _rows(out, "out", dt, (T, N), dev), None if ws is None else ws.data_ptr(),
                          0 if ws is None else ws.numel(), raw), "pw_linear_i8")
    return out


def pw_linear_i8_workspace_bytes(T: int, K: int) -> int:
    return lib().pw_linear_i8_workspace_bytes(T, K)


def pw_linear_i8_status(stream=None) -> int:
    """Status bits that pw_linear_i8 calls have raised since the previous status call,
    those ordered before `stream`'s work included."""
    st = _i()
    _check(lib().pw_linear_i8_status(_stream(stream), ctypes.byref(st)), "pw_linear_i8_status")
    return st.value


def pw_debug_linear_timeout(stream=None):
    return _check(lib().pw_debug_linear_timeout(_stream(stream)), "pw_debug_linear_timeout")


class LogProbs(NamedTuple):
    """What pw_logprobs returns; logprob and rank are None without ids,
    top_ids and top_logprobs are [T][0] without alternatives."""
    logprob: object
    rank: object
    entropy: object
    top_ids: object
    top_logprobs: object


def pw_logprobs(logits, ids=None, top: int = 0, out=None, stream=None):
    """Log probability and rank of the given tokens, entropy and the ``top``
    likeliest alternatives of every row of logits.  ids: int32 or int64 [T], or
    None.  out: a LogProbs (or tuple) of tensors to write into; its entries may
    be None for what is not wanted."""
    torch = _torch()
    (T, V), (dev, raw) = _matrix(logits, "logits"), _place(torch, logits, "logits", stream)
    f32, i32 = torch.float32, torch.int32
    if out is None:
        new = lambda dt, *shape: _empty(torch, stream, shape, dt, logits.device)
        out = (None if ids is None else new(f32, T), None if ids is None else new(i32, T), new(f32, T),
               new(i32, T, top), new(f32, T, top))
    lp, rank, ent, ti, tl = out
    pid, ids64 = None, 0
    if ids is not None:
        ids64 = 1 if ids.dtype is torch.int64 else 0
        pid = _vec(ids, "ids", torch.int64 if ids64 else i32, T, dev)
    if top:
        for name, t, dt in (("top_ids", ti, i32), ("top_logprobs", tl, f32)):
            if t is None or t.shape != (T, top) or t.dtype is not dt or not t.is_contiguous() or _away(t, dev):
                raise ValueError(f"{name}: a contiguous matrix [{T}][{top}] of {dt} on the call's GPU is needed")
    _check(lib().pw_logprobs(logits.data_ptr(), _rows(logits, "logits", logits.dtype, (T, V), dev),
                             _code(logits.dtype), T, V, pid, ids64, top,
                             None if lp is None else _vec(lp, "logprob", f32, T, dev),
                             None if rank is None else _vec(rank, "rank", i32, T, dev),
                             None if ent is None else _vec(ent, "entropy", f32, T, dev),
                             ti.data_ptr() if top else None, tl.data_ptr() if top else None,
                             raw), "pw_logprobs")
    return LogProbs(lp, rank, ent, ti, tl)


# ----------------------------------------------------------------------------- expert layers in 8-bit floating point

# The conventions are those of the operators above.  8-bit numbers are
# torch.float8_e4m3fn; scales are float32, one for every 128 columns.

def f8_blocks(n: int) -> int:
    """Scales of n columns (or of n rows of weights)."""
    return (n + F8_BLOCK - 1) // F8_BLOCK


def rows_f8(*shape, device="cuda", stream=None):
    """An uninitialised e4m3 tensor [..][K] whose rows start on 16-byte
    boundaries, as pw_linear_f8 wants them (a view of a padded one), in memory
    of the given stream or the current one."""
    torch = _torch()
    K = shape[-1]
    return _empty(torch, stream, (*shape[:-1], (K + 15) // 16 * 16), torch.float8_e4m3fn, device)[..., :K]


def _stack(t, name: str, dtype, shape, dev):
    """(row stride, stride of the first axis) of [E][rows][columns] on the call's
    device whose rows are consecutive elements."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {dtype} is needed, got {t.dtype}")
    if t.shape != shape or _away(t, dev):
        raise ValueError(f"{name}: a tensor of shape {tuple(shape)} on the call's GPU is needed, "
                         f"got {tuple(t.shape)} on {t.device}")
    group, ld, one = t.stride()
    if one != 1 and shape[2] > 1:
        raise ValueError(f"{name}: the elements of a row must be consecutive")
    # an axis of one has no stride of its own
    return ld if shape[1] > 1 else (shape[2] + 15) // 16 * 16, group if shape[0] > 1 else 0


class Routing(NamedTuple):
    """What pw_route returns."""
    idx: object
    weight: object
    offsets: object
    perm: object
    inv: object


def pw_route(logits, top_k: int, renorm: bool = False, out=None, stream=None):
    """A Routing of logits [T][E] float32: the top_k experts of every token and their
    softmax weights [T][top_k] (renorm: over the chosen ones), offsets [E + 1] of the
    routed pairs in expert order, the pair id t * top_k + j at each place (perm) and
    the place of each pair (inv).  out: a Routing (or tuple) to write into."""
    torch = _torch()
    (T, E), (dev, raw) = _matrix(logits, "logits"), _place(torch, logits, "logits", stream)
    f32, i32, P = torch.float32, torch.int32, T * top_k
    if out is None:
        new = lambda dt, *shape: _empty(torch, stream, shape, dt, logits.device)
        out = (new(i32, T, top_k), new(f32, T, top_k), new(i32, E + 1), new(i32, P), new(i32, P))
    idx, weight, offsets, perm, inv = out
    for name, t, dt in (("idx", idx, i32), ("weight", weight, f32)):
        if t.shape != (T, top_k) or t.dtype is not dt or not t.is_contiguous() or _away(t, dev):
            raise ValueError(f"{name}: a contiguous matrix [{T}][{top_k}] of {dt} on the call's GPU is needed")
    _check(lib().pw_route(logits.data_ptr(), _rows(logits, "logits", f32, (T, E), dev), T, E, top_k, int(renorm),
                      idx.data_ptr(), weight.data_ptr(), _vec(offsets, "offsets", i32, E + 1, dev),
                      _vec(perm, "perm", i32, P, dev), _vec(inv, "inv", i32, P, dev), raw), "pw_route")
    return Routing(idx, weight, offsets, perm, inv)


def _quant_f8(torch, stream, dev, x, T, K, scale_rows, q, scale):
    """(q, its address and row stride, scale, its address and row stride) of a
    quantiser, made where they are not given."""
    shape = (scale_rows, f8_blocks(K))
    if q is None:
        q = rows_f8(T, K, device=x.device, stream=stream)
    if scale is None:
        scale = _empty(torch, stream, shape, torch.float32, x.device)
    return (q, scale, q.data_ptr(), _rows(q, "q", torch.float8_e4m3fn, (T, K), dev), scale.data_ptr(),
            _rows(scale, "scale", torch.float32, shape, dev))


def pw_quant_f8(x, rows=None, per: int = 1, q=None, scale=None, stream=None):
    """(q, scale): the rows of x as e4m3 with a scale for every 128 columns.  rows
    (int32): row t is x[rows[t] // per], so that a Routing's perm with per = top_k
    gives the tokens in expert order."""
    torch = _torch()
    (n, K), (dev, raw) = _matrix(x, "x"), _place(torch, x, "x", stream)
    T, pr = n, None
    if rows is not None:
        T = rows.shape[0]
        pr = _vec(rows, "rows", torch.int32, T, dev)
    q, scale, pq, lq, ps, ls = _quant_f8(torch, stream, dev, x, T, K, T, q, scale)
    _check(lib().pw_quant_f8(x.data_ptr(), _rows(x, "x", x.dtype, (n, K), dev), n, pr, per, T, K, _code(x.dtype), pq, lq,
                             ps, ls, raw), "pw_quant_f8")
    return q, scale


def pw_silu_quant_f8(x, q=None, scale=None, stream=None):
    """(q, scale) of silu(gate) * up, x [T][2 K] with the gate columns first."""
    torch = _torch()
    (T, K2), (dev, raw) = _matrix(x, "x"), _place(torch, x, "x", stream)
    if K2 % 2:
        raise ValueError(f"x: gate and up columns are needed, got {K2}")
    q, scale, pq, lq, ps, ls = _quant_f8(torch, stream, dev, x, T, K2 // 2, T, q, scale)
    _check(lib().pw_silu_quant_f8(x.data_ptr(), _rows(x, "x", x.dtype, (T, K2), dev), T, K2 // 2, _code(x.dtype), pq, lq,
                                  ps, ls, raw), "pw_silu_quant_f8")
    return q, scale


def pw_quant_f8_blocks(w, q=None, scale=None, stream=None):
    """(q, scale): weights [N][K] as e4m3 with a scale for each block of 128 x 128."""
    torch = _torch()
    (N, K), (dev, raw) = _matrix(w, "w"), _place(torch, w, "w", stream)
    q, scale, pq, lq, ps, ls = _quant_f8(torch, stream, dev, w, N, K, f8_blocks(N), q, scale)
    _check(lib().pw_quant_f8_blocks(w.data_ptr(), _rows(w, "w", w.dtype, (N, K), dev), N, K, _code(w.dtype), pq, lq, ps,
                                    ls, raw), "pw_quant_f8_blocks")
    return q, scale


def _f8_out(torch, stream, what, x, shape, out, out_dtype):
    if out is None:
        return _empty(torch, stream, shape, out_dtype or torch.float16, x.device)
    if out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"{what}: out is {out.dtype}, not {out_dtype}")
    return out


def pw_linear_f8(x, x_scale, w, w_scale, bias=None, out=None, out_dtype=None, stream=None):
    """out [T][N] = x . w^T (+ bias), x [T][K] and w [N][K] e4m3 with 16-byte
    aligned rows (rows_f8), x_scale [T][ceil(K / 128)] and w_scale [ceil(N / 128)]
    [ceil(K / 128)], as pw_quant_f8 and pw_quant_f8_blocks write them.  out has type
    out_dtype (default float16) where it is not given."""
    torch = _torch()
    T, K = _matrix(x, "x")
    N, (dev, raw) = _matrix(w, "w")[0], _place(torch, x, "x", stream)
    out = _f8_out(torch, stream, "pw_linear_f8", x, (T, N), out, out_dtype)
    dt, f32, f8, kb = out.dtype, torch.float32, torch.float8_e4m3fn, f8_blocks(K)
    _check(lib().pw_linear_f8(x.data_ptr(), _rows(x, "x", f8, (T, K), dev), x_scale.data_ptr(),
                              _rows(x_scale, "x_scale", f32, (T, kb), dev), w.data_ptr(), _rows(w, "w", f8, (N, K), dev),
                              w_scale.data_ptr(), _rows(w_scale, "w_scale", f32, (f8_blocks(N), kb), dev),
                              None if bias is None else _vec(bias, "bias", dt, N, dev), T, N, K, _code(dt),
                              out.data_ptr(), _rows(out, "out", dt, (T, N), dev), raw), "pw_linear_f8")
    return out


def pw_grouped_linear_f8(x, x_scale, w, w_scale, offsets, bias=None, out=None, out_dtype=None, stream=None):
    """pw_linear_f8 of rows sorted by expert: rows [offsets[e], offsets[e + 1]) of x
    with w[e], w_scale[e] and bias[e]; w [E][N][K], w_scale [E][ceil(N / 128)][ceil(K /
    128)], bias [E][N], offsets [E + 1] int32 on the GPU (pw_route).  Rows outside every
    range are left as they are."""
    torch = _torch()
    T, K = _matrix(x, "x")
    if w.dim() != 3:
        raise ValueError(f"w: weights [E][N][K] are needed, got {w.dim()} dimensions")
    (E, N, _), (dev, raw) = w.shape, _place(torch, x, "x", stream)
    out = _f8_out(torch, stream, "pw_grouped_linear_f8", x, (T, N), out, out_dtype)
    dt, f32, f8, kb = out.dtype, torch.float32, torch.float8_e4m3fn, f8_blocks(K)
    ldw, gw = _stack(w, "w", f8, (E, N, K), dev)
    ldws, gws = _stack(w_scale, "w_scale", f32, (E, f8_blocks(N), kb), dev)
    if bias is not None and (bias.dtype is not dt or bias.shape != (E, N) or not bias.is_contiguous() or _away(bias, dev)):
        raise ValueError(f"bias: a contiguous matrix [{E}][{N}] of {dt} on the call's GPU is needed")
    _check(lib().pw_grouped_linear_f8(x.data_ptr(), _rows(x, "x", f8, (T, K), dev), x_scale.data_ptr(),
                                      _rows(x_scale, "x_scale", f32, (T, kb), dev), w.data_ptr(), ldw, gw,
                                      w_scale.data_ptr(), ldws, gws,
                                      _vec(offsets, "offsets", torch.int32, E + 1, dev),
                                      None if bias is None else bias.data_ptr(), T, E, N, K, _code(dt), out.data_ptr(),
                                      _rows(out, "out", dt, (T, N), dev), raw), "pw_grouped_linear_f8")
    return out


def pw_linear_f8_status(stream=None) -> int:
    """Status bits that pw_linear_f8 and pw_grouped_linear_f8 calls have raised since the
    previous status call, those ordered before `stream`'s work included."""
    st = _i()
    _check(lib().pw_linear_f8_status(_stream(stream), ctypes.byref(st)), "pw_linear_f8_status")
    return st.value


def pw_debug_linear_f8_timeout(stream=None):
    return _check(lib().pw_debug_linear_f8_timeout(_stream(stream)), "pw_debug_linear_f8_timeout")


def pw_debug_linear_f8(way, x, x_scale, w, w_scale, offsets=None, bias=None, out=None, out_dtype=None, stream=None):
    """Test hook: pw_grouped_linear_f8 (w [1][N][K] without offsets: pw_linear_f8) in a
    given way, (CTAs, rows, channels, parts of K) as include/pw.h has them."""
    torch = _torch()
    T, K = _matrix(x, "x")
    (E, N, _), (dev, raw) = w.shape, _place(torch, x, "x", stream)
    out = _f8_out(torch, stream, "pw_debug_linear_f8", x, (T, N), out, out_dtype)
    dt, f32, f8, kb = out.dtype, torch.float32, torch.float8_e4m3fn, f8_blocks(K)
    ldw, gw = _stack(w, "w", f8, (E, N, K), dev)
    ldws, gws = _stack(w_scale, "w_scale", f32, (E, f8_blocks(N), kb), dev)
    _check(lib().pw_debug_linear_f8(*way, x.data_ptr(), _rows(x, "x", f8, (T, K), dev), x_scale.data_ptr(),
                                    _rows(x_scale, "x_scale", f32, (T, kb), dev), w.data_ptr(), ldw, gw,
                                    w_scale.data_ptr(), ldws, gws,
                                    None if offsets is None else _vec(offsets, "offsets", torch.int32, E + 1, dev),
                                    None if bias is None else _vec(bias.view(-1), "bias", dt, E * N, dev), T, E, N, K,
                                    _code(dt), out.data_ptr(), _rows(out, "out", dt, (T, N), dev), raw),
           "pw_debug_linear_f8")
    return out


def pw_combine(y, weight, inv, residual=None, out=None, out_dtype=None, stream=None):
    """out [T][H] = residual + sum_j weight[t][j] * y[inv[t][j]]: y [rows][H] in expert
    order, weight [T][k] and inv ([T * k] or [T][k]) of a Routing.  out has type
    out_dtype (default: the residual's, or y's) where it is not given."""
    torch = _torch()
    R, H = _matrix(y, "y")
    (T, k), (dev, raw) = _matrix(weight, "weight"), _place(torch, y, "y", stream)
    if out_dtype is None and out is None:
        out_dtype = y.dtype if residual is None else residual.dtype
    out = _f8_out(torch, stream, "pw_combine", y, (T, H), out, out_dtype)
    dt, pr, lr = out.dtype, None, 0
    if residual is not None:
        lr, pr = _rows(residual, "residual", dt, (T, H), dev), residual.data_ptr()
    if weight.dtype is not torch.float32 or not weight.is_contiguous() or _away(weight, dev):
        raise ValueError(f"weight: a contiguous float32 matrix [{T}][{k}] on the call's GPU is needed")
    if (inv.dtype is not torch.int32 or (inv.shape != (T * k,) and inv.shape != (T, k)) or not inv.is_contiguous()
            or _away(inv, dev)):
        raise ValueError(f"inv: {T * k} consecutive int32 on the call's GPU are needed")
    _check(lib().pw_combine(y.data_ptr(), _rows(y, "y", y.dtype, (R, H), dev), R, _code(y.dtype), weight.data_ptr(),
                            inv.data_ptr(), pr, lr, T, k, H, _code(dt), out.data_ptr(), _rows(out, "out", dt, (T, H), dev),
                            raw), "pw_combine")
    return out
