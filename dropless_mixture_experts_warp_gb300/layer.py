"""One dropless MoE layer step through the C ABI: buffers and the call sequence.

PyTorch only allocates device memory and provides the stream; every step runs in
libmoe.so's kernels.  Forward: route -> permute -> grouped MLP -> combine.
Backward: combine_bwd -> grouped MLP backward -> un-permute (combine of dXp) ->
route backward.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import binding as B
from . import fp8

FP8_BLOCK = B.PREC["fp8-block"]

@dataclass
class Buffers:
    dims: B.moe_dims
    rows: int
    topk_idx: torch.Tensor
    topk_w: torch.Tensor
    split_sizes: torch.Tensor
    offsets: torch.Tensor
    row_offsets: torch.Tensor
    xp: torch.Tensor
    row_to_token: torch.Tensor
    token_to_row: torch.Tensor
    w_rows: torch.Tensor
    gu: torch.Tensor
    h: torch.Tensor
    y_rows: torch.Tensor
    y: torch.Tensor
    dy_rows: torch.Tensor
    dgu: torch.Tensor
    dxp: torch.Tensor
    dw_gu: torch.Tensor
    dw_d: torch.Tensor
    dw_rows: torch.Tensor
    dx: torch.Tensor
    d_logits: torch.Tensor
    workspace: torch.Tensor
    status: torch.Tensor
    # shared expert (dims.f_shared > 0), else None
    gu_s: torch.Tensor = None
    h_s: torch.Tensor = None
    y_s: torch.Tensor = None
    dgu_s: torch.Tensor = None
    dx_s: torch.Tensor = None
    dw_gu_s: torch.Tensor = None
    dw_d_s: torch.Tensor = None
    # MXFP8 path (dims.prec == mxfp8): quantised weights and activation scratch
    wq: torch.Tensor = None
    mx_ws: torch.Tensor = None
    wq_s: torch.Tensor = None
    mx_ws_s: torch.Tensor = None
    # blocks of 128 (dims.prec == fp8-block), the row space's and the shared expert's
    q: "Blocks" = None
    q_s: "Blocks" = None


@dataclass
class Blocks:
    """One expert MLP's operands with blocks of 128: weights (use_weights(), quantize_weights()) and activations; for
    training with the columns' forms and the gradients'."""
    gu: fp8.Weights = None     # [E, 2f, d]
    down: fp8.Weights = None   # [E, d, f]
    x: fp8.Rows = None         # [rows, d]
    h: fp8.Rows = None         # [rows, f]
    dy: fp8.Rows = None        # [rows, d]
    dgu: fp8.Rows = None       # [rows, 2f]
    dh: torch.Tensor = None    # [rows, f] bf16
    dw_part: torch.Tensor = None
    given: bool = False        # the weights are the caller's: never written


def dims_of(T, d, f, E, k, f_shared=0, score="softmax", prec="bf16") -> B.moe_dims:
    dims = B.make_dims(T, d, f, E, k, f_shared, score, prec)
    st = B.moe_check_dims(dims)
    if st != B.MOE_OK:
        raise B.MoeError("moe_check_dims", st)
    return dims


def allocate(dims: B.moe_dims, device="cuda", train=True) -> Buffers:
    """train=False: for forward() alone, without the gradients' buffers."""
    T, d, f, E, k = dims.T, dims.d, dims.f, dims.E, dims.k
    rows = B.moe_row_capacity(dims)
    i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
    e = lambda *s, dt=bf: torch.empty(*s, dtype=dt, device=device)  # noqa: E731
    g = e if train else lambda *s, dt=bf: None  # noqa: E731
    blocks = dims.prec == FP8_BLOCK
    plain = (lambda *s, dt=bf: None) if blocks else e  # rows that the blocks' path holds as codes  # noqa: E731
    shared = {}
    if dims.f_shared:
        fs = dims.f_shared
        shared = dict(gu_s=e(T, 2 * fs), h_s=plain(T, fs), y_s=e(T, d), dgu_s=None if blocks else g(T, 2 * fs), dx_s=g(T, d),
                      dw_gu_s=g(2 * fs, d), dw_d_s=g(d, fs))
    if dims.prec in (1, 2):
        shared["wq"] = torch.empty(B.moe_mx_weights_size(dims), dtype=torch.uint8, device=device)
        shared["mx_ws"] = torch.empty(B.moe_mx_workspace_size(dims), dtype=torch.uint8, device=device)
        if dims.f_shared:
            shared["wq_s"] = torch.empty(B.moe_mx_shared_weights_size(dims), dtype=torch.uint8, device=device)
            shared["mx_ws_s"] = torch.empty(max(1, B.moe_mx_shared_workspace_size(dims)), dtype=torch.uint8,
                                            device=device)
    if blocks:
        shared["q"] = _allocate_blocks(rows, d, f, train, True, device)
        if dims.f_shared:
            shared["q_s"] = _allocate_blocks(T, d, dims.f_shared, train, False, device)
    return Buffers(**shared,
        dims=dims, rows=rows,
        topk_idx=e(T, k, dt=i32), topk_w=e(T, k, dt=f32), split_sizes=e(E, dt=i32),
        offsets=e(E + 1, dt=i32), row_offsets=e(E + 1, dt=i32),
        xp=plain(rows, d), row_to_token=e(rows, dt=i32), token_to_row=e(T, k, dt=i32), w_rows=e(rows, dt=f32),
        gu=e(rows, 2 * f), h=plain(rows, f), y_rows=e(rows, d), y=e(T, d),
        dy_rows=None if blocks else g(rows, d), dgu=None if blocks else g(rows, 2 * f), dxp=g(rows, d),
        dw_gu=g(E, 2 * f, d), dw_d=g(E, d, f), dw_rows=g(rows, dt=f32), dx=g(T, d), d_logits=g(T, E, dt=f32),
        workspace=torch.empty(max(1, B.moe_workspace_size(dims)), dtype=torch.uint8, device=device),
        status=torch.zeros(1, dtype=i32, device=device),
    )


def _allocate_blocks(rows, d, f, train, weighted, device) -> Blocks:
    q = Blocks(x=fp8.allocate_rows(rows, d, both=train, device=device), h=fp8.allocate_rows(rows, f, both=train, device=device))
    if train:
        q.dy = fp8.allocate_rows(rows, d, both=True, device=device)
        q.dgu = fp8.allocate_rows(rows, 2 * f, both=True, device=device)
        q.dh = torch.empty(rows, f, dtype=torch.bfloat16, device=device)
        q.dw_part = torch.empty(rows, f // fp8.BLOCK, device=device) if weighted else None
    return q


def use_weights(b: Buffers, gu: fp8.Weights, down: fp8.Weights, gu_s: fp8.Weights = None, down_s: fp8.Weights = None):
    """fp8-block: the layer computes with these weights (a checkpoint's, fp8.weights_of()), in forward(...,
    weights_cached=True); backward() wants their transposed codes too."""
    dm = b.dims
    if dm.prec != FP8_BLOCK:
        raise ValueError("use_weights: the layer is not fp8-block")

    def check(w, E, N, K):
        if w is None or (w.E, w.N, w.K) != (E, N, K) or w.device != b.y.device:
            raise ValueError(f"expected weights [{E}, {N}, {K}] on {b.y.device}, got {w and (w.E, w.N, w.K, w.device)}")

    check(gu, dm.E, 2 * dm.f, dm.d)
    check(down, dm.E, dm.d, dm.f)
    if dm.f_shared:
        check(gu_s, 1, 2 * dm.f_shared, dm.d)
        check(down_s, 1, dm.d, dm.f_shared)
        b.q_s.gu, b.q_s.down, b.q_s.given = gu_s, down_s, True
    b.q.gu, b.q.down, b.q.given = gu, down, True


def quantize_weights(b: Buffers, w_gu, w_d, stream=None, w_gu_s=None, w_d_s=None):
    """MXFP8: the 16-bit master weights -> b.wq (and b.wq_s for the shared expert), codes and
    scales in both contraction orientations.  The weights change once per optimiser step, so a
    step of several micro-batches quantises them once and passes weights_cached=True to every
    forward() of the step.  fp8-block: to b.q's weights (and b.q_s's), allocated at the first call and in
    place of those that use_weights() gave, which stay as they are."""
    dm = b.dims
    if dm.prec == FP8_BLOCK:
        for q, E, f, gu, down in ((b.q, dm.E, dm.f, w_gu, w_d), (b.q_s, 1, dm.f_shared, w_gu_s, w_d_s)):
            if q is None:
                continue
            if gu is None or down is None:
                raise ValueError("quantize_weights: no 16-bit weights (weights_cached=True after use_weights())")
            if q.gu is None or q.given:
                both, dev = q.dy is not None, b.y.device
                q.gu = fp8.allocate_weights(E, 2 * f, dm.d, both=both, device=dev)
                q.down = fp8.allocate_weights(E, dm.d, f, both=both, device=dev)
                q.given = False
            fp8.quantize_weights(q.gu, gu.view(E, 2 * f, dm.d), stream)
            fp8.quantize_weights(q.down, down.view(E, dm.d, f), stream)
        return
    if dm.prec not in (1, 2):
        raise ValueError("quantize_weights: the layer is not in 8 bits")
    B.moe_mx_quantize_weights(dm, w_gu, w_d, b.wq, stream)
    if dm.f_shared:
        B.moe_mx_quantize_shared_weights(dm, w_gu_s, w_d_s, b.wq_s, stream)


def forward(b: Buffers, x, logits, w_gu, w_d, stream=None, w_gu_s=None, w_d_s=None, grouped=None,
            weights_cached=False):
    """grouped: {"n_group", "topk_group", "bias" (device [E] fp32 or None), "routed_scale"} selects the
    group-limited sigmoid router instead of the plain top-k.  weights_cached (MXFP8): b.wq (and
    b.wq_s) already hold this step's quantised weights (quantize_weights()), so they are not
    quantised again."""
    dm = b.dims
    mx8 = dm.prec in (1, 2)   # MXFP8, or FP8 x FP4 (MXFP4 weights)
    blocks = dm.prec == FP8_BLOCK
    if (mx8 or blocks) and not weights_cached:
        quantize_weights(b, w_gu, w_d, stream, w_gu_s, w_d_s)
    if blocks and b.q.gu is None:
        raise ValueError("weights_cached: no weights yet (use_weights() or quantize_weights())")
    shared_out = None
    if dm.f_shared and blocks:
        fp8.quantize(b.q_s.x, x, stream=stream)
        _blocks_forward(b.q_s, dm.f_shared, None, None, b.gu_s, b.y_s, b.status, stream)
        shared_out = b.y_s
    elif dm.f_shared and mx8:
        B.moe_shared_mlp_fwd_mx(dm, x, b.wq_s, b.mx_ws_s, b.gu_s, b.y_s, b.status, stream)
        shared_out = b.y_s
    elif dm.f_shared:
        B.moe_shared_mlp_fwd(dm, x, w_gu_s, w_d_s, b.gu_s, b.h_s, b.y_s, b.status, stream)
        shared_out = b.y_s
    if grouped is not None:
        B.moe_route_topk_grouped(dm, logits, grouped.get("bias"), grouped["n_group"], grouped["topk_group"],
                                 grouped.get("routed_scale", 1.0), b.topk_idx, b.topk_w, b.split_sizes,
                                 b.offsets, b.row_offsets, b.workspace, b.status, stream)
    else:
        B.moe_route_topk(dm, logits, b.topk_idx, b.topk_w, b.split_sizes, b.offsets, b.row_offsets,
                         b.workspace, b.status, stream)
    if blocks:
        B.moe_permute_fp8(dm, x, b.topk_idx, b.topk_w, b.split_sizes, b.row_offsets, b.workspace, b.q.x.codes, b.q.x.scales,
                          b.q.x.codes_t, b.q.x.scales_t, b.row_to_token, b.token_to_row, b.w_rows, b.status, stream)
        _blocks_forward(b.q, dm.f, b.row_offsets, b.w_rows, b.gu, b.y_rows, b.status, stream)
    elif mx8:
        B.moe_permute_mx(dm, x, b.topk_idx, b.topk_w, b.split_sizes, b.row_offsets, b.workspace, b.mx_ws,
                         b.row_to_token, b.token_to_row, b.w_rows, b.status, stream)
        B.moe_grouped_mlp_fwd_mx(dm, b.row_offsets, b.w_rows, b.wq, b.mx_ws, b.gu, b.y_rows, b.status, stream)
    else:
        B.moe_permute(dm, x, b.topk_idx, b.topk_w, b.split_sizes, b.row_offsets, b.workspace, b.xp,
                      b.row_to_token, b.token_to_row, b.w_rows, b.status, stream)
        B.moe_grouped_mlp_fwd(dm, b.xp, b.row_offsets, b.w_rows, w_gu, w_d, b.gu, b.h, b.y_rows, b.status,
                              stream)
    B.moe_combine_fwd(dm, b.y_rows, b.token_to_row, shared_out, b.y, stream)
    return b.y


def _blocks_forward(q: Blocks, f, offsets, w_rows, gu, y, status, stream):
    """q.x's rows through both products, with the SwiGLU quantised between them: gu and y."""
    R, d, E = q.x.R, q.x.C, q.gu.E
    used = None if offsets is None else offsets.data_ptr() + 4 * E       # the rows in use
    B.moe_fp8_gemm(q.x.codes, q.x.scales, R, d, q.gu.codes, q.gu.scales, 0, 2 * f, E, offsets, gu, status, stream)
    B.moe_fp8_swiglu(gu, w_rows, R, f, used, q.h.codes, q.h.scales, stream)
    B.moe_fp8_gemm(q.h.codes, q.h.scales, R, f, q.down.codes, q.down.scales, 0, d, E, offsets, y, status, stream)


def _blocks_backward(q: Blocks, f, offsets, w_rows, gu, dx, dw_gu, dw_d, dw_rows, status, stream):
    """From q.dy (quantised both ways) to the gradients of q.x's rows, the weights and w_rows."""
    R, d, E = q.x.R, q.x.C, q.gu.E
    used = None if offsets is None else offsets.data_ptr() + 4 * E
    B.moe_fp8_gemm(q.dy.codes, q.dy.scales, R, d, q.down.codes_t, q.down.scales, 1, f, E, offsets, q.dh, status, stream)
    B.moe_fp8_swiglu_bwd(gu, q.dh, w_rows, R, f, used, q.dgu.codes, q.dgu.scales, q.dgu.codes_t, q.dgu.scales_t, q.h.codes_t,
                         q.h.scales_t, dw_rows, q.dw_part, stream)
    R_t = q.x.codes_t.shape[1]
    B.moe_fp8_wgrad(q.dy.codes_t, q.dy.scales_t, q.h.codes_t, q.h.scales_t, R_t, d, f, E, offsets, dw_d, status, stream)
    B.moe_fp8_gemm(q.dgu.codes, q.dgu.scales, R, 2 * f, q.gu.codes_t, q.gu.scales, 1, d, E, offsets, dx, status, stream)
    B.moe_fp8_wgrad(q.dgu.codes_t, q.dgu.scales_t, q.x.codes_t, q.x.scales_t, R_t, 2 * f, d, E, offsets, dw_gu, status, stream)


def backward(b: Buffers, dy, logits, w_gu, w_d, stream=None, x=None, w_gu_s=None, w_d_s=None, grouped=None):
    """x (the forward's input) is needed by the shared expert and by the MXFP8 path; grouped as in
    forward()."""
    dm = b.dims
    mx8 = dm.prec in (1, 2)   # MXFP8, or FP8 x FP4 (MXFP4 weights)
    blocks = dm.prec == FP8_BLOCK
    if b.dx is None:
        raise ValueError("backward: the buffers are of allocate(train=False)")
    if blocks and (b.q.gu is None or b.q.gu.codes_t is None or b.q.down.codes_t is None):
        raise ValueError("backward: wants the weights' transposed codes")
    shared_dx = None
    if dm.f_shared and blocks:
        fp8.quantize(b.q_s.dy, dy, stream=stream)
        _blocks_backward(b.q_s, dm.f_shared, None, None, b.gu_s, b.dx_s, b.dw_gu_s, b.dw_d_s, None, b.status, stream)
        shared_dx = b.dx_s
    elif dm.f_shared and mx8:
        B.moe_shared_mlp_bwd_mx(dm, b.wq_s, b.mx_ws_s, b.gu_s, dy, b.dx_s, b.dw_gu_s, b.dw_d_s, b.status,
                                stream)
        shared_dx = b.dx_s
    elif dm.f_shared:
        B.moe_shared_mlp_bwd(dm, x, w_gu_s, w_d_s, b.gu_s, b.h_s, dy, b.dgu_s, b.dx_s, b.dw_gu_s, b.dw_d_s,
                             b.status, stream)
        shared_dx = b.dx_s
    if blocks:
        if dm.T:
            B.moe_fp8_quantize(dy, b.rows, dm.d, b.row_to_token, b.row_offsets.data_ptr() + 4 * dm.E, b.q.dy.codes,
                               b.q.dy.scales, b.q.dy.codes_t, b.q.dy.scales_t, stream)
        _blocks_backward(b.q, dm.f, b.row_offsets, b.w_rows, b.gu, b.dxp, b.dw_gu, b.dw_d, b.dw_rows, b.status, stream)
    elif mx8:
        B.moe_combine_bwd_mx(dm, dy, b.row_to_token, b.split_sizes, b.row_offsets, b.mx_ws, stream)
        B.moe_grouped_mlp_bwd_mx(dm, b.row_offsets, b.w_rows, b.wq, b.mx_ws, b.gu, b.dxp, b.dw_gu, b.dw_d,
                                 b.dw_rows, b.workspace, b.status, stream)
    else:
        B.moe_combine_bwd(dm, dy, b.token_to_row, b.split_sizes, b.row_offsets, b.dy_rows, stream)
        B.moe_grouped_mlp_bwd(dm, b.xp, b.row_offsets, b.w_rows, w_gu, w_d, b.gu, b.h, b.dy_rows, b.dgu,
                              b.dxp, b.dw_gu, b.dw_d, b.dw_rows, b.workspace, b.status, stream)
    B.moe_combine_fwd(dm, b.dxp, b.token_to_row, shared_dx, b.dx, stream)
    if grouped is not None:
        B.moe_route_topk_bwd_scaled(dm, logits, b.topk_idx, b.topk_w, grouped.get("routed_scale", 1.0), b.dw_rows,
                                    b.token_to_row, b.d_logits, stream)
    else:
        B.moe_route_topk_bwd(dm, logits, b.topk_idx, b.topk_w, b.dw_rows, b.token_to_row, b.d_logits, stream)
    return b.dx


def check(b: Buffers, stream=None):
    st = B.moe_check_status(b.status, stream)
    if st != B.MOE_OK:
        raise B.MoeError("device status", st)
