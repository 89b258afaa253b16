"""One routed-MoE layer forward as a sequence of library calls on caller-owned buffers.

route + permute (one launch for small T) -> expert FFN -> combine, each a libmoecache.so
entry point; a single token takes moe_decode_token instead where it applies, which does all
of it in one launch.
Device memory comes from torch; this class only allocates the intermediate
buffers once and forwards pointers.
"""
import torch

from . import (MOE_F32, MOE_BF16, MOE_MXFP4, MOE_MXFP8, MOE_PATH_AUTO, moe_route, moe_permute, moe_route_permute,
               moe_permute_workspace_bytes, moe_expert_ffn, moe_expert_ffn_workspace_bytes,
               moe_combine, moe_decode_token, moe_decode_token_workspace_bytes, moe_mxfp8_bytes,
               moe_mxfp8_quantize, moe_rmsnorm, moe_combine_rmsnorm)


def decode_token_supported(T, k, d, f, dtype, w_dtype, y_dtype):
    """Shapes and types moe_decode_token takes (one token, bf16 activations, bf16 or MXFP4
    weights, fp32 expert outputs, x and h within 64 KB of LDS; MXFP4 strips held whole in
    registers: d <= 4096, f <= 2048, k <= 8)."""
    if T != 1 or dtype != MOE_BF16 or y_dtype != MOE_F32:
        return False
    if d > 8192 or f > 8192 or (d + k * f) * 2 > 65536:
        return False
    if w_dtype == MOE_MXFP4:
        return d <= 4096 and f <= 2048 and k <= 8
    return w_dtype == MOE_BF16


def _tdtype(code):
    return torch.float32 if code == MOE_F32 else torch.bfloat16


def _code(t, n):
    """MOE_* code of the element type of a contiguous tensor of n elements (or of no tensor)."""
    if t is None:
        return MOE_BF16
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"fp32 or bf16 tensor expected, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"contiguous tensor of {n} elements expected, got {tuple(t.shape)}, strides {t.stride()}")
    return MOE_F32 if t.dtype == torch.float32 else MOE_BF16


def _check_bytes(t, n):
    """MXFP8 rows: a contiguous uint8 tensor of at least n bytes."""
    if t.dtype != torch.uint8:
        raise TypeError(f"uint8 tensor of MXFP8 rows expected, got {t.dtype}")
    if t.numel() < n or not t.is_contiguous():
        raise ValueError(f"contiguous tensor of at least {n} bytes expected, got {tuple(t.shape)}, strides {t.stride()}")


class MoeLayer:
    def __init__(self, T, E, k, d, f, dtype=MOE_BF16, y_dtype=MOE_F32, device="cuda",
                 w_dtype=None):
        """dtype: activations (and weights unless w_dtype is given, e.g. MOE_MXFP4).  With
        MOE_MXFP8 activations (and MXFP4 weights, the default there) the layer keeps a buffer x8
        of T MXFP8 rows, which norm() or quantize() fills."""
        if w_dtype is None and dtype == MOE_MXFP8:
            w_dtype = MOE_MXFP4
        self.T, self.E, self.k, self.d, self.f = T, E, k, d, f
        self.dtype, self.y_dtype = dtype, y_dtype
        self.w_dtype = dtype if w_dtype is None else w_dtype
        A = T * k
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.ids = torch.empty((T, k), **i32)
        self.w = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.counts = torch.empty(E, **i32)
        self.offsets = torch.empty(E + 1, **i32)
        self.perm = torch.empty(max(A, 1), **i32)
        self.inv = torch.empty(max(A, 1), **i32)
        self.status = torch.zeros(1, **i32)
        self.perm_ws_bytes = moe_permute_workspace_bytes(T, k, E)
        self.perm_ws = torch.empty(self.perm_ws_bytes, dtype=torch.uint8, device=dev)
        self.ffn_ws_bytes = moe_expert_ffn_workspace_bytes(T, k, f, dtype)
        self.ffn_ws = torch.empty(self.ffn_ws_bytes, dtype=torch.uint8, device=dev)
        self.y_perm = torch.empty((max(A, 1), d), dtype=_tdtype(y_dtype), device=dev)
        self.out = torch.empty((T, d), dtype=torch.float32, device=dev)
        if dtype == MOE_MXFP8:
            self.x8 = torch.empty(max(moe_mxfp8_bytes(T, d), 16), dtype=torch.uint8, device=dev)
        self.fusable = decode_token_supported(T, k, d, f, dtype, self.w_dtype, y_dtype)
        if self.fusable:
            # counters of the one-launch path: zero before the first call, zero after each
            self.tok_ws_bytes = moe_decode_token_workspace_bytes(k, f)
            self.tok_ws = torch.zeros(self.tok_ws_bytes, dtype=torch.uint8, device=dev)

    def route(self, logits, stream=None):
        moe_route(logits, self.T, self.E, self.k, self.ids, self.w, stream)

    def permute(self, stream=None):
        moe_permute(self.ids, self.T, self.k, self.E, self.counts, self.offsets, self.perm,
                    self.inv, self.perm_ws, self.perm_ws_bytes, self.status, stream)

    def route_permute(self, logits, stream=None):
        """route() then permute(), in one launch for small T."""
        moe_route_permute(logits, self.T, self.E, self.k, self.ids, self.w, self.counts,
                          self.offsets, self.perm, self.inv, self.perm_ws, self.perm_ws_bytes,
                          self.status, stream)

    def ffn(self, x, arena, entry_stride, expert_slot=None, mask=None, slot_key=None, key_base=0,
            path=MOE_PATH_AUTO, stream=None):
        if self.dtype == MOE_MXFP8 and torch.is_tensor(x):
            _check_bytes(x, moe_mxfp8_bytes(self.T, self.d))
        moe_expert_ffn(x, self.dtype, self.perm, self.offsets, self.T, self.k, self.E, self.d,
                       self.f, expert_slot, arena, entry_stride, self.w_dtype, mask, slot_key,
                       key_base, self.ffn_ws, self.ffn_ws_bytes, self.y_perm, self.y_dtype, path,
                       self.status, stream)

    def quantize(self, x, stream=None):
        """x [T, d] (fp32 or bf16) into the layer's MXFP8 rows."""
        moe_mxfp8_quantize(x, _code(x, self.T * self.d), self.T, self.d, self.x8, stream)
        return self.x8

    def norm(self, x, gamma, eps, delta=None, x_out=None, y=None, stream=None):
        """Residual addition and RMS norm in front of the layer: x (+ delta) to x_out, the
        normalised rows to y and, with MXFP8 activations, to the layer's MXFP8 rows."""
        n = self.T * self.d
        if x_out is not None and _code(x_out, n) != _code(x, n):
            raise TypeError(f"x_out is {x_out.dtype}, x {x.dtype}")
        moe_rmsnorm(x, _code(x, n), delta, _code(delta, n), gamma, _code(gamma, self.d), eps, self.T, self.d,
                    x_out, y, _code(y, n), self.x8 if self.dtype == MOE_MXFP8 else None, stream)

    def combine_norm(self, x, gamma, eps, x_out=None, y=None, x8=None, stream=None):
        """combine(), the residual addition and the next RMS norm in one launch (self.out is not
        written): x + combined rows to x_out, the normalised rows to y and / or, in MXFP8, to x8."""
        n = self.T * self.d
        if x_out is not None and _code(x_out, n) != _code(x, n):
            raise TypeError(f"x_out is {x_out.dtype}, x {x.dtype}")
        if x8 is not None:
            _check_bytes(x8, moe_mxfp8_bytes(self.T, self.d))
        moe_combine_rmsnorm(self.y_perm, self.y_dtype, self.inv, self.w, self.k, x, _code(x, n), gamma,
                            _code(gamma, self.d), eps, self.T, self.d, x_out, y, _code(y, n), x8, stream)

    def combine(self, stream=None):
        moe_combine(self.y_perm, self.y_dtype, self.inv, self.w, self.T, self.k, self.d,
                    self.out, stream)

    def decode_token(self, x, logits, arena, entry_stride, expert_slot=None, slot_key=None,
                     key_base=0, stream=None):
        """The whole layer for one token in one launch (logits None: route with self.ids and
        self.w as they stand).  Leaves counts/offsets/perm/inv untouched."""
        moe_decode_token(logits, x, self.E, self.k, self.d, self.f, expert_slot, arena,
                         entry_stride, self.w_dtype, slot_key, key_base, self.ids, self.w,
                         self.tok_ws, self.tok_ws_bytes, self.out, self.status, stream)
        return self.out

    def forward(self, x, logits, arena, entry_stride, expert_slot=None, path=MOE_PATH_AUTO,
                stream=None, fused=None):
        """fused: None = the one-launch path where it applies (path AUTO), True = require it,
        False = separate launches.  With MXFP8 activations x is an MXFP8 buffer (uint8, e.g.
        self.x8 after norm()) or fp32 / bf16 rows, which are quantised first."""
        if self.dtype == MOE_MXFP8 and x.dtype != torch.uint8:
            x = self.quantize(x, stream)
        if fused is None:
            fused = self.fusable and path == MOE_PATH_AUTO
        if fused:
            return self.decode_token(x, logits, arena, entry_stride, expert_slot, stream=stream)
        self.route_permute(logits, stream)
        self.ffn(x, arena, entry_stride, expert_slot, path=path, stream=stream)
        self.combine(stream)
        return self.out
