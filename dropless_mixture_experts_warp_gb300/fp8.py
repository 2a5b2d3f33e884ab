"""8-bit products with a scale for each block of 128: E4M3 codes, fp32 scales.

    w = weights_of(codes, scales)             # a checkpoint's, or allocate_weights() and quantize_weights()
    a = allocate_rows(R, K)                   # both=True: with the columns' form, for weight_grad()
    quantize(a, x)                            # x [R, K] bf16
    matmul(a, w, out)                         # out [R, N] bf16 = x w^T
    matmul(dy, w, dx, transposed=True)        # dx [R, K] = dy w; w with codes_t
    weight_grad(dy, x, dw)                    # dw [1, N, K] = dy^T x, from the columns' forms

With `offsets` (int32 [E + 1], multiples of 128, as moe_route_topk's row_offsets) each expert multiplies its own
rows.  PyTorch only allocates; the steps run in libmoe.so's kernels (moe_fp8_* of include/moe.h, where the formulas
and forms are).  layer.py runs a whole layer on them (prec="fp8-block").
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import binding as B

BLOCK = 128
E4M3 = torch.float8_e4m3fn


def _up(n):
    return -(-n // BLOCK) * BLOCK


@dataclass
class Rows:
    """A quantised matrix [R, C]: the rows' form, the columns' form (transposed, rows padded to whole blocks), or both."""
    R: int
    C: int
    codes: Optional[torch.Tensor]       # [R, C] E4M3
    scales: Optional[torch.Tensor]      # [ceil(C / 128), R] fp32
    codes_t: Optional[torch.Tensor]     # [C, R up to 128]
    scales_t: Optional[torch.Tensor]    # [ceil(R / 128), C]
    device: torch.device
    status: torch.Tensor                # errors of the products that read it


@dataclass
class Weights:
    """Quantised matrices [E, N, K], one scale for each 128 x 128 block of each."""
    E: int
    N: int
    K: int
    codes: torch.Tensor                 # [E, N, K] E4M3
    scales: torch.Tensor                # [E, ceil(N / 128), ceil(K / 128)] fp32
    codes_t: Optional[torch.Tensor]     # [E, K, N], for matmul(transposed=True)
    device: torch.device


def allocate_rows(R, C, both=False, device="cuda") -> Rows:
    if R < 0 or C <= 0 or C % 16:
        raise ValueError(f"rows of a multiple of 16 values: got {R} x {C}")
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device=device)  # noqa: E731
    codes = e(R, C, dt=E4M3)
    more = (e(C, _up(R), dt=E4M3), e(_up(R) // BLOCK, C)) if both else (None, None)
    return Rows(R, C, codes, e(_up(C) // BLOCK, R), *more, codes.device, torch.zeros(1, dtype=torch.int32, device=device))


def rows_of(codes=None, scales=None, codes_t=None, scales_t=None, R=None) -> Rows:
    """Rows that hold the given tensors.  With the columns' form alone, R is its (padded) length unless given."""
    if (codes is None) != (scales is None) or (codes_t is None) != (scales_t is None) or (codes is None and codes_t is None):
        raise ValueError("codes with their scales: of the rows, of the columns, or both")
    dev = (codes if codes is not None else codes_t).device
    if codes is not None:
        R, C = codes.shape
    else:
        C = codes_t.shape[0]
        R = codes_t.shape[1] if R is None else R
    if C % 16:
        raise ValueError(f"rows of a multiple of 16 values: got {C}")
    B.check_tensor(codes, E4M3, (R, C), dev)
    B.check_tensor(scales, torch.float32, (_up(C) // BLOCK, R), dev)
    B.check_tensor(codes_t, E4M3, (C, _up(R)), dev)
    B.check_tensor(scales_t, torch.float32, (_up(R) // BLOCK, C), dev)
    return Rows(R, C, codes, scales, codes_t, scales_t, dev, torch.zeros(1, dtype=torch.int32, device=dev))


def allocate_weights(E, N, K, both=False, device="cuda") -> Weights:
    if E <= 0 or N <= 0 or K <= 0 or N % 16 or K % 16:
        raise ValueError(f"matrices with sides that are multiples of 16: got {E} x {N} x {K}")
    codes = torch.empty(E, N, K, dtype=E4M3, device=device)
    return Weights(E, N, K, codes, torch.empty(E, _up(N) // BLOCK, _up(K) // BLOCK, device=device),
                   torch.empty(E, K, N, dtype=E4M3, device=device) if both else None, codes.device)


def weights_of(codes, scales, codes_t=None) -> Weights:
    """Weights that hold the given tensors (a checkpoint's codes and block scales)."""
    E, N, K = codes.shape
    if N % 16 or K % 16:
        raise ValueError(f"matrices with sides that are multiples of 16: got {N} x {K}")
    B.check_tensor(codes, E4M3, (E, N, K), codes.device)
    B.check_tensor(scales, torch.float32, (E, _up(N) // BLOCK, _up(K) // BLOCK), codes.device)
    B.check_tensor(codes_t, E4M3, (E, K, N), codes.device)
    return Weights(E, N, K, codes, scales, codes_t, codes.device)


def quantize(a: Rows, x, row_map=None, n_rows=None, stream=None) -> Rows:
    """x bf16 [R, C] -> the forms that a has.  row_map int32 [R]: row r is x[row_map[r]], zeros where that is negative
    (x then has any number of rows).  n_rows int32 [1] on the device: blocks of 128 rows from there on are left."""
    B.check_device(a.device, stream)
    B.check_tensor(x, torch.bfloat16, (a.R, a.C) if row_map is None else (x.shape[0], a.C), a.device)
    B.check_tensor(row_map, torch.int32, (a.R,), a.device)
    B.check_tensor(n_rows, torch.int32, (1,), a.device)
    B.moe_fp8_quantize(x, a.R, a.C, row_map, n_rows, a.codes, a.scales, a.codes_t, a.scales_t, stream)
    return a


def quantize_weights(w: Weights, w16, stream=None) -> Weights:
    """w16 bf16 [E, N, K] -> w's codes, scales and, where it has them, transposed codes."""
    B.check_device(w.device, stream)
    B.check_tensor(w16, torch.bfloat16, (w.E, w.N, w.K), w.device)
    B.moe_fp8_quantize_weights(w16, w.E, w.N, w.K, w.codes, w.codes_t, w.scales, stream)
    return w


def _experts(E, offsets, device):
    if offsets is None and E != 1:
        raise ValueError("offsets say which rows are whose")
    B.check_tensor(offsets, torch.int32, (E + 1,), device)


def matmul(a: Rows, w: Weights, out, offsets=None, transposed=False, stream=None):
    """out bf16 = a times each expert's w^T ([R, N] from a [R, K]), or w (transposed: [R, K] from a [R, N])."""
    B.check_device(a.device, stream)
    if a.codes is None or w.device != a.device or a.C != (w.N if transposed else w.K):
        raise ValueError(f"rows [{a.R}, {a.C}] in the rows' form on {a.device} do not fit weights [{w.E}, {w.N}, {w.K}] on {w.device}")
    if transposed and w.codes_t is None:
        raise ValueError("transposed wants weights with codes_t")
    N = w.K if transposed else w.N
    B.check_tensor(out, torch.bfloat16, (a.R, N), a.device)
    _experts(w.E, offsets, a.device)
    B.moe_fp8_gemm(a.codes, a.scales, a.R, a.C, w.codes_t if transposed else w.codes, w.scales, transposed, N, w.E, offsets, out,
                   a.status, stream)
    return out


def weight_grad(dy: Rows, x: Rows, out, offsets=None, stream=None):
    """out bf16 [E, N, K] = dy^T x over each expert's rows, from dy [R, N] and x [R, K] in the columns' form."""
    B.check_device(dy.device, stream)
    if dy.codes_t is None or x.codes_t is None or _up(dy.R) != _up(x.R) or x.device != dy.device:
        raise ValueError("weight_grad takes two matrices of as many rows in the columns' form, on one device")
    E = out.shape[0]
    B.check_tensor(out, torch.bfloat16, (E, dy.C, x.C), dy.device)
    _experts(E, offsets, dy.device)
    B.moe_fp8_wgrad(dy.codes_t, dy.scales_t, x.codes_t, x.scales_t, _up(dy.R), dy.C, x.C, E, offsets, out, dy.status, stream)
    return out


def check(a: Rows, stream=None):
    """Raise on an error that a product of a found on the device."""
    st = B.moe_check_status(a.status, stream)
    if st != B.MOE_OK:
        raise B.MoeError("device status", st)
