"""One MoE feed-forward layer on one GPU, sequenced over the C ABI.

``MoELayer`` owns the device buffers of one layer shape and issues the ABI
calls in the order of the method (route -> permute -> grouped GEMM forward ->
combine, then the backward twins), all on one stream with no host
synchronisation.  It does no arithmetic of its own: every step runs in the
HIP library.  Buffers come from torch's caching allocator.

The backward of the layer with the routing held fixed:
    dy_perm = permute(dout, row_scale = topk_w)     (combine backward)
    dgu, dx_perm, dw13, dw2 = grouped_gemm_bwd(...)
    dx = unpermute_combine(dx_perm, weights = None) (permute backward)

With MXFP4 the forward runs in 4 bits and the backward is the bf16 one on the
decoded rows and weights, with the quantisers taken as the identity.  dw2 =
dy^T h is made from the h the forward saved, in bf16, and not from the 4-bit
copy that the down product multiplied by: that costs no further pass over h
and is nearer to the layer without quantisers (with Gaussian operands 23% off
its dw2 in norm, against 28%; the two lie 15% apart).  decode_h=True makes
dw2 from the 4-bit copy: the gradient of the forward that ran.
"""
import ctypes

import torch

from . import (MOE_ACT_RELU, MOE_ACT_SILU, MOE_BF16, MOE_F32, MOE_GEMM_DGRAD_DOWN, MOE_GEMM_DGRAD_GATE_UP,
               MOE_GEMM_WGRAD, MOE_INT4, MOE_MXFP4, MOE_MXFP8,
               _array, _launch, _nbytes, _p,
               gemm_tensors, glu, moe_balance_loss, moe_balance_loss_bwd, moe_balance_workspace_bytes,
               moe_combine_dropout, moe_dequantize_mxfp4, moe_dropout, moe_gate_grad, moe_gemm_workspace_bytes,
               moe_grouped_gemm_op, moe_grouped_glu_bwd, moe_grouped_glu_fwd, moe_grouped_glu_op, moe_int4_ffn,
               moe_int4_workspace_bytes, moe_quantize_int4, moe_quantize_mxfp4, moe_quantize_mxfp8,
               moe_route_workspace_bytes, moe_router_logits)

_ACT = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16, MOE_MXFP8: torch.bfloat16,
        MOE_MXFP4: torch.bfloat16, MOE_INT4: torch.bfloat16}


def int4_sizes_ok(T, E, d, f, k):
    """Whether moe_int4_ffn takes T tokens of k slots (shared experts counted in E and k)."""
    return (0 <= T and 1 <= k <= 8 and 1 <= E <= 1024 and 1 <= d <= 1 << 20 and 1 <= f <= 1 << 20 and T * k < 1 << 31 and
            T * d < 1 << 30 and T * k * f < 1 << 30 and d * f < 1 << 31)


class MoELayer:
    """n_shared > 0 adds that many shared experts (ungated, every token, weight
    1) as extra groups E .. E+n_shared-1 of the same grouped GEMM: weights are
    then [E + n_shared, ...] with the shared experts last, and the buffers hold
    the routed rows followed by n_shared * T shared rows.  save=False (MXFP4
    only) keeps no activations for a backward, as serving wants it.
    decode_h=True (MXFP4 only): dw2 from the 4-bit h.

    act and limit: the gate of the experts' blocks, MOE_ACT_*, and the limit on
    what goes into it (0: none); other ones than silu without a limit with
    fp32, bf16 and INT4.  h_dropout: dropout of the experts' h (fp32, bf16);
    out_dropout: of the layer's output, before the residual that forward may be
    given.  Masks follow from rng, int64 [2, 2] on the device: (seed, step) of the
    two, written in place if at all.  Each forward advances both steps, by a kernel
    of its own, so that a replayed graph draws new masks; forward(same_mask=True)
    does not, to recompute activations.  Layers that train together need different
    seeds: without one (None) a layer draws its own from torch's default generator,
    so that torch.manual_seed repeats a run.  Ranks with one seed drop the same
    places of their own tokens.
    With training set to False nothing is dropped (set it before a forward and
    leave it until its backward).

    dtype=MOE_INT4 serves experts held in 4-bit integers with a scale for each
    `group` elements, with zero points if zeros is true: forward only, unpadded,
    activations in bf16."""

    def __init__(self, T, d, E, f, k, dtype=MOE_BF16, capacity=0, device="cuda", n_shared=0, save=True,
                 decode_h=False, act=MOE_ACT_SILU, limit=0.0, h_dropout=0.0, out_dropout=0.0, seed=None, group=128,
                 zeros=False):
        if dtype == MOE_INT4:
            save = False
            if capacity:
                raise ValueError("an INT4 layer has no padded layout")
            if group not in (32, 64, 128) or d % group or f % group:
                raise ValueError(f"INT4: groups of 32, 64 or 128 that divide d = {d} and f = {f}, got {group}")
            if not int4_sizes_ok(T, E + n_shared, d, f, k + n_shared):
                raise ValueError(f"INT4: T = {T}, d = {d}, f = {f}, {k + n_shared} slots of {E + n_shared} experts are past "
                                 "what moe_int4_ffn takes: T * d and T * k * f below 2^30, d * f below 2^31, d and f at "
                                 "most 2^20, 8 slots, 1024 experts")
            if out_dropout:
                raise ValueError("out_dropout: an INT4 layer serves, it has no dropout")
        # (as the calls see them, in fp32)
        L = ctypes.c_float(limit).value
        if not (MOE_ACT_SILU <= act <= MOE_ACT_RELU and 0 <= L < float("inf") and (L > 0) == (limit > 0)):
            raise ValueError(f"act = {act}, limit = {limit}: expected a MOE_ACT_* and a limit >= 0 (0: none)")
        for name, p in (("h_dropout", h_dropout), ("out_dropout", out_dropout)):
            if not 0 <= ctypes.c_float(p).value < 1:
                raise ValueError(f"{name}: expected 0 <= p < 1, got {p}")
        other_gate = act != MOE_ACT_SILU or limit > 0
        if other_gate and dtype not in (MOE_F32, MOE_BF16, MOE_INT4):
            raise ValueError("the MXFP8 and MXFP4 products have the silu gate without a limit")
        if h_dropout and dtype not in (MOE_F32, MOE_BF16):
            raise ValueError("h_dropout: fp32 and bf16 layers only")
        if not save and dtype not in (MOE_MXFP4, MOE_INT4):
            raise ValueError("save=False: only the MXFP4 forward runs without its saved activations")
        if decode_h and (dtype != MOE_MXFP4 or not save):
            raise ValueError("decode_h=True: only an MXFP4 layer with saved activations has an h in 4 bits to decode")
        self.save, self.decode_h = save, decode_h
        self.act, self.limit, self.h_dropout, self.out_dropout = act, limit, h_dropout, out_dropout
        self.group, self.zeros = group, zeros
        self.training = True
        self._glu = None
        self.rng = self._rng_step = None
        if h_dropout or out_dropout:
            if seed is None:
                seed = int(torch.randint(1 << 62, (), device="cpu"))
            # the two masks of one step are 2^62 steps apart
            self.rng = torch.tensor([[seed, 0], [seed, 1 << 62]], dtype=torch.int64, device=device)
            self._rng_step = self.rng[:, 1]
        if other_gate or h_dropout:
            rng = self.rng[0] if h_dropout else None
            self._glu = {t: glu(act, limit, h_dropout if t else 0.0, rng) for t in (False, True)}
        self.T, self.d, self.E, self.f, self.k = T, d, E, f, k
        self.dtype, self.capacity, self.device = dtype, capacity, device
        self.S = n_shared
        self.K = k + n_shared                  # slots per token (routed, then shared)
        self.G = E + n_shared                  # GEMM groups
        self.R = E * capacity if capacity > 0 else T * k   # routed rows
        self.n_rows = self.R + n_shared * T
        R = self.n_rows
        act_dtype = _ACT[dtype]
        i32 = dict(dtype=torch.int32, device=device)
        self.topk_idx = torch.empty(T, k, **i32)
        self.topk_w = torch.empty(T, k, dtype=torch.float32, device=device)
        self.counts = torch.empty(E, **i32)
        self.offsets = torch.empty(E + 1, **i32)
        self.dst_row = torch.empty(T * k, **i32)
        self.src_slot = torch.empty(self.R, **i32)
        if n_shared:
            K, G = self.K, self.G
            self.s_idx = torch.empty(T, K, **i32)
            self.s_w = torch.empty(T, K, dtype=torch.float32, device=device)
            self.s_counts = torch.empty(G, **i32)
            self.s_off = torch.empty(G + 1, **i32)
            self.s_dst = torch.empty(T * K, **i32)
            self.s_src = torch.empty(R, **i32)
        else:
            self.s_idx, self.s_w, self.s_dst, self.s_src = self.topk_idx, self.topk_w, self.dst_row, self.src_slot
            self.s_counts, self.s_off = self.counts, self.offsets
        self.s_fill = self.s_src if capacity > 0 else None   # where a permute finds the empty rows
        # group offsets and capacity the grouped GEMM takes (shared groups: explicit offsets)
        self.g_cap = 0 if n_shared else capacity
        self.dev_err = torch.zeros(1, **i32)
        self.route_ws = torch.empty(moe_route_workspace_bytes(T, E, k), dtype=torch.uint8,
                                    device=device)
        if dtype == MOE_INT4:
            self._glu = glu(act, limit)
            self.w13_4 = self.w2_4 = None
            self.out = torch.empty(T, d, dtype=act_dtype, device=device)
            self._dev = self.out.get_device()
            self.int4_ws = torch.empty(moe_int4_workspace_bytes(R, d, f), dtype=torch.uint8, device=device)
            self._bwd_alloc = False
            return
        if dtype == MOE_MXFP8:
            self.x_perm = torch.empty(R, d, dtype=torch.uint8, device=device)
            self.x_perm_scales = torch.empty(R, d // 32, dtype=torch.uint8, device=device)
        elif dtype == MOE_MXFP4:
            self.x_perm = torch.empty(R, d // 2, dtype=torch.uint8, device=device)
            self.x_perm_scales = torch.empty(R, d // 32, dtype=torch.uint8, device=device)
        else:
            self.x_perm = torch.empty(R, d, dtype=act_dtype, device=device)
            self.x_perm_scales = None
        self.gu = torch.empty(R, 2 * f, dtype=act_dtype, device=device) if save else None
        self.h = torch.empty(R, f, dtype=act_dtype, device=device) if save else None
        self.y_perm = torch.empty(R, d, dtype=act_dtype, device=device)
        self.out = torch.empty(T, d, dtype=act_dtype, device=device)
        self._dev = self.out.get_device()
        self.gemm_ws = None
        wsb = moe_gemm_workspace_bytes(dtype, self.G, R, d, f)
        if wsb:
            self.gemm_ws = torch.empty(wsb, dtype=torch.uint8, device=device)
        self._bwd_alloc = False

    def _alloc_bwd(self):
        if self._bwd_alloc:
            return
        if not self.save:
            raise RuntimeError("an INT4 layer has no backward" if self.dtype == MOE_INT4 else
                               "a layer made with save=False has no backward")
        R, d, f, E = self.n_rows, self.d, self.f, self.G
        act = _ACT[self.dtype]
        dev = self.device
        self.dy_perm = torch.empty(R, d, dtype=act, device=dev)
        self.dgu = torch.empty(R, 2 * f, dtype=act, device=dev)
        self.dx_perm = torch.empty(R, d, dtype=act, device=dev)
        self.dx = torch.empty(self.T, d, dtype=act, device=dev)
        self.dw13 = torch.empty(E, 2 * f, d, dtype=act, device=dev)
        self.dw2 = torch.empty(E, d, f, dtype=act, device=dev)
        if self.dtype == MOE_MXFP4:   # the decoded operands of the bf16 backward, and its workspace
            self.x_perm_d = torch.empty(R, d, dtype=act, device=dev)
            self.h_d = self.h
            if self.decode_h:
                self.h_d = torch.empty(R, f, dtype=act, device=dev)
                self.h_q = torch.empty(R, f // 2, dtype=torch.uint8, device=dev)
                self.h_s = torch.empty(R, f // 32, dtype=torch.uint8, device=dev)
            self.w13_d = torch.empty(E, 2 * f, d, dtype=act, device=dev)
            self.w2_d = torch.empty(E, d, f, dtype=act, device=dev)
            if self.w13 is not None:
                self._decode_weights()
            self.bwd_ws = torch.empty(moe_gemm_workspace_bytes(MOE_BF16, E, R, d, f), dtype=torch.uint8,
                                      device=dev)
        self._bwd_alloc = True

    def _decode_weights(self):
        E, f, d = self.G, self.f, self.d
        moe_dequantize_mxfp4(self.w13_q.view(E * 2 * f, -1), self.w13_s.view(E * 2 * f, -1),
                             self.w13_d.view(E * 2 * f, d))
        moe_dequantize_mxfp4(self.w2_q.view(E * d, -1), self.w2_s.view(E * d, -1), self.w2_d.view(E * d, f))

    # -------------------------------------------------------------- weights
    def _check_held(self, name, w, n, dtype, dense=True):
        # the kernels read n elements at w's address, whatever its shape
        if w.dtype is not dtype or w.numel() != n or w.device != self.out.device or (dense and not w.is_contiguous()):
            raise ValueError(f"{name}: expected a {'contiguous ' if dense else ''}{dtype} tensor of {n} elements on "
                             f"{self.out.device}, got {w.dtype} {tuple(w.shape)} with strides {w.stride()} on {w.device}")

    def set_weights(self, w13, w2):
        """Weights [E, 2f, d] and [E, d, f] (MOE_F32: fp32, otherwise bf16) on the
        layer's device; refused ones leave the layer with those it had.  For MXFP8
        the forward and backward MXFP8 caches are made here (once per optimizer
        step), for MXFP4 and INT4 the codes of both; an INT4 layer does not keep the
        bf16 weights.  Each call makes new caches and lets go of the last ones, so a
        graph that was captured with those is not replayed afterwards: weights that
        change under a graph go through requantize_weights, which works in place."""
        E, f, d = self.G, self.f, self.d
        # (the quantisers are given a dense copy of weights that are not)
        dense = self.dtype in (MOE_F32, MOE_BF16)
        self._check_held("w13", w13, E * 2 * f * d, _ACT[self.dtype], dense)
        self._check_held("w2", w2, E * d * f, _ACT[self.dtype], dense)
        if self.dtype == MOE_MXFP4:
            u8 = dict(dtype=torch.uint8, device=self.device)
            codes = (torch.empty(E, 2 * f, d // 2, **u8), torch.empty(E, 2 * f, d // 32, **u8),
                     torch.empty(E, d, f // 2, **u8), torch.empty(E, d, f // 32, **u8))
            self._quantize_mxfp4(w13, w2, *codes)
            self.set_weights_mxfp4(*codes)
            self.w13, self.w2 = w13, w2
            if self._bwd_alloc:
                self._decode_weights()
            return
        if self.dtype == MOE_INT4:
            g = self.group
            made = []
            for N, K in ((2 * f, d), (d, f)):
                u8 = dict(dtype=torch.uint8, device=self.device)
                made.append((torch.empty(E, N, K // 2, **u8),
                             torch.empty(E, N, K // g, dtype=torch.bfloat16, device=self.device),
                             torch.empty(E, N, K // g, **u8) if self.zeros else None))
            self._quantize_int4(w13, w2, *made)
            self.set_weights_int4(*made)
            return
        self.w13, self.w2 = w13, w2
        self._stages = None
        if self.dtype != MOE_MXFP8:
            return
        dev = self.device
        u8 = dict(dtype=torch.uint8, device=dev)
        # forward direction: blocks along the contraction dim of each GEMM
        self.w13_q = torch.empty(E * 2 * f, d, **u8)
        self.w13_s = torch.empty(E * 2 * f, d // 32, **u8)
        self.w2_q = torch.empty(E * d, f, **u8)
        self.w2_s = torch.empty(E * d, f // 32, **u8)
        # backward direction: each expert's matrix transposed, blocks along 2f / d
        # (column-wise quantiser layout: K * (rows + 128 * groups) codes)
        self._g13 = torch.arange(0, E + 1, dtype=torch.int32, device=dev) * (2 * f)
        self._g2 = torch.arange(0, E + 1, dtype=torch.int32, device=dev) * d
        n13 = d * (E * 2 * f + 128 * E)
        n2 = f * (E * d + 128 * E)
        self.w13t_q = torch.empty(n13, **u8)
        self.w13t_s = torch.empty(n13 // 32, **u8)
        self.w2t_q = torch.empty(n2, **u8)
        self.w2t_s = torch.empty(n2 // 32, **u8)
        self.requantize_weights()

    def set_weights_mxfp4(self, w13_q, w13_s, w2_q, w2_s):
        """MXFP4: weights that are held in 4 bits already, codes [E, 2f, d/2] and [E, d, f/2]
        with scales [E, 2f, d/32] and [E, d, f/32] (as moe_quantize_mxfp4 makes them).  The
        layer reads these tensors at each step: they may be quantised anew in place between
        steps, so the backward decodes them each time it runs."""
        if self.dtype != MOE_MXFP4:
            raise ValueError("set_weights_mxfp4 needs an MXFP4 layer")
        n13, n2 = self.G * 2 * self.f * self.d, self.G * self.d * self.f
        for name, w, n in (("w13_q", w13_q, n13 // 2), ("w13_s", w13_s, n13 // 32), ("w2_q", w2_q, n2 // 2),
                           ("w2_s", w2_s, n2 // 32)):
            self._check_held(name, w, n, torch.uint8)
        self.w13_q, self.w13_s, self.w2_q, self.w2_s = w13_q, w13_s, w2_q, w2_s
        self.w13 = self.w2 = None   # these codes have no bf16 weights behind them
        self._stages = None

    def set_weights_int4(self, w13, w2):
        """INT4: weights that are held in 4-bit integers already, each (codes, scales, zeros or
        None) as moe_quantize_int4 makes them: codes [E, 2f, d/2] and [E, d, f/2] uint8, scales
        and zeros [..., K/group].  The layer reads these tensors at each step."""
        if self.dtype != MOE_INT4:
            raise ValueError("set_weights_int4 needs an INT4 layer")
        E, f, d = self.G, self.f, self.d
        for name, w, N, K in (("w13", w13, 2 * f, d), ("w2", w2, d, f)):
            if len(w) != 3 or w[0] is None or w[1] is None:
                raise ValueError(f"{name}: expected (codes, scales, zeros or None)")
            for t, shape, dt in zip(w, ((E, N, K // 2), (E, N, K // self.group), (E, N, K // self.group)),
                                    (torch.uint8, torch.bfloat16, torch.uint8)):
                if t is not None and (tuple(t.shape) != shape or t.dtype is not dt or not t.is_contiguous()
                                      or t.get_device() != self.out.get_device()):
                    raise ValueError(f"{name}: expected a contiguous {dt} tensor of shape {shape} on {self.out.device}, "
                                     f"got {t.dtype} {tuple(t.shape)} on {t.device}")
        self.w13_4, self.w2_4 = tuple(w13), tuple(w2)

    def _quantize_mxfp4(self, w13, w2, w13_q, w13_s, w2_q, w2_s):
        E, f, d = self.G, self.f, self.d
        moe_quantize_mxfp4(w13.reshape(E * 2 * f, d), w13_q.view(E * 2 * f, -1), w13_s.view(E * 2 * f, -1))
        moe_quantize_mxfp4(w2.reshape(E * d, f), w2_q.view(E * d, -1), w2_s.view(E * d, -1))

    def _quantize_int4(self, w13, w2, w13_4, w2_4):
        for w, (codes, scales, zeros) in ((w13, w13_4), (w2, w2_4)):
            rows, K = codes.shape[0] * codes.shape[1], 2 * codes.shape[2]
            moe_quantize_int4(w.reshape(rows, K), self.group, codes.view(rows, -1), scales.view(rows, -1),
                              None if zeros is None else zeros.view(rows, -1))

    def requantize_weights(self, w13=None, w2=None):
        """Rebuild in place what the layer's kernels read, as after an optimizer step.  MXFP8: the four
        weight caches (forward and backward direction of w13 and w2) from the bf16 weights.  MXFP4: the
        codes.  INT4, whose bf16 weights the layer does not keep: the codes, scales and zero points it
        holds (with zero points where it holds some) from the w13 and w2 given here."""
        E, f, d = self.G, self.f, self.d
        if self.dtype not in (MOE_MXFP8, MOE_MXFP4, MOE_INT4):
            raise ValueError("requantize_weights: fp32 and bf16 layers read the weights themselves")
        given = self.dtype == MOE_INT4
        if (w13 is not None) != given or (w2 is not None) != given:
            raise ValueError("requantize_weights takes w13 and w2 for an INT4 layer, and no tensors for the others")
        if given:
            if self.w13_4 is None:
                raise ValueError("requantize_weights: the layer has no weights yet (set_weights)")
            self._check_held("w13", w13, E * 2 * f * d, torch.bfloat16, False)
            self._check_held("w2", w2, E * d * f, torch.bfloat16, False)
            self._quantize_int4(w13, w2, self.w13_4, self.w2_4)
            return
        if self.dtype == MOE_MXFP4:
            if self.w13 is None:
                raise ValueError("requantize_weights: the layer's weights were given in 4 bits")
            self._quantize_mxfp4(self.w13, self.w2, self.w13_q, self.w13_s, self.w2_q, self.w2_s)
            if self._bwd_alloc:
                self._decode_weights()
            return
        moe_quantize_mxfp8(self.w13.reshape(E * 2 * f, d), 0, self.w13_q, self.w13_s)
        moe_quantize_mxfp8(self.w2.reshape(E * d, f), 0, self.w2_q, self.w2_s)
        moe_quantize_mxfp8(self.w13.reshape(E * 2 * f, d), 1, self.w13t_q, self.w13t_s, self._g13, E)
        moe_quantize_mxfp8(self.w2.reshape(E * d, f), 1, self.w2t_q, self.w2t_s, self._g2, E)

    # -------------------------------------------------------------- stages
    def _stage_tensors(self):
        """Operands of the five grouped GEMM stages: (forward-direction set,
        backward-direction set); they differ only in the MXFP8 weight caches."""
        if not self.save:
            t = dict(x_perm=self.x_perm, x_perm_scales=self.x_perm_scales, y_perm=self.y_perm, ws=self.gemm_ws)
            return gemm_tensors(w13=self.w13_q, w13_scales=self.w13_s, w2=self.w2_q, w2_scales=self.w2_s, **t), None
        self._alloc_bwd()
        common = dict(x_perm=self.x_perm, x_perm_scales=self.x_perm_scales, gu=self.gu, h=self.h,
                      y_perm=self.y_perm, dy_perm=self.dy_perm, dgu=self.dgu, dx_perm=self.dx_perm,
                      dw13=self.dw13, dw2=self.dw2, ws=self.gemm_ws)
        if self.dtype == MOE_MXFP4:
            fwd = gemm_tensors(w13=self.w13_q, w13_scales=self.w13_s, w2=self.w2_q, w2_scales=self.w2_s, **common)
            common.update(x_perm=self.x_perm_d, x_perm_scales=None, h=self.h_d, ws=self.bwd_ws)
            return fwd, gemm_tensors(w13=self.w13_d, w2=self.w2_d, **common)
        if self.dtype != MOE_MXFP8:
            t = gemm_tensors(w13=self.w13, w2=self.w2, **common)
            return t, t
        fwd = gemm_tensors(w13=self.w13_q, w13_scales=self.w13_s, w2=self.w2_q,
                           w2_scales=self.w2_s, **common)
        bwd = gemm_tensors(w13=self.w13t_q, w13_scales=self.w13t_s, w2=self.w2t_q,
                           w2_scales=self.w2t_s, **common)
        return fwd, bwd

    def gemm_stage(self, op):
        """Issue one grouped GEMM stage (MOE_GEMM_*) on the layer's buffers (the
        forward and backward calls are these stages in order).  Call
        set_weights first; the tensors are bound on first use."""
        self._no_int4()
        if getattr(self, "_stages", None) is None:
            self._stages = self._stage_tensors()
        bwd = op in (MOE_GEMM_DGRAD_DOWN, MOE_GEMM_DGRAD_GATE_UP)
        dtype = self.dtype
        if dtype == MOE_MXFP4 and (bwd or op == MOE_GEMM_WGRAD):
            self._alloc_bwd()
            if op == MOE_GEMM_WGRAD:
                self._decode_rows()
            elif self.w13 is None:
                self._decode_weights()
            bwd, dtype = True, MOE_BF16
        if self._glu is not None:
            moe_grouped_glu_op(op, dtype, self._glu[self.training], self._stages[1 if bwd else 0], self.s_off,
                               self.g_cap, self.G, self.n_rows, self.d, self.f)
            return
        moe_grouped_gemm_op(op, dtype, self._stages[1 if bwd else 0], self.s_off,
                            self.g_cap, self.G, self.n_rows, self.d, self.f)

    def _decode_rows(self):
        moe_dequantize_mxfp4(self.x_perm, self.x_perm_scales, self.x_perm_d)
        if self.decode_h:
            moe_quantize_mxfp4(self.h, self.h_q, self.h_s)   # the codes the down product read
            moe_dequantize_mxfp4(self.h_q, self.h_s, self.h_d)

    def wgrad_accumulate(self, dw13_f32, dw2_f32):
        """bf16 and MXFP4: the weight-gradient stage adding into fp32 accumulators
        (dw13_f32 += dgu^T x_perm, dw2_f32 += dy_perm^T h, per expert) instead
        of writing the bf16 dw13 / dw2.  Call after backward (it reads dgu)."""
        self._alloc_bwd()
        mx4 = self.dtype == MOE_MXFP4
        if mx4:   # the activation gradients may have come stage by stage, which decodes no rows
            self._decode_rows()
        t = gemm_tensors(x_perm=self.x_perm_d if mx4 else self.x_perm, h=self.h_d if mx4 else self.h,
                         dy_perm=self.dy_perm, dgu=self.dgu, dw13_f32=dw13_f32, dw2_f32=dw2_f32,
                         ws=self.bwd_ws if mx4 else self.gemm_ws)
        moe_grouped_gemm_op(MOE_GEMM_WGRAD, MOE_BF16 if mx4 else self.dtype, t, self.s_off, self.g_cap, self.G,
                            self.n_rows, self.d, self.f)

    # -------------------------------------------------------------- steps
    # The layer's own buffers have the sizes that its calls take, so a step checks what it is given and hands
    # pointers on: a bf16 forward takes 20 us of the host so, and 39 through the calls that check every tensor.
    def _rows_given(self, name, t, dtype, width):
        # the pointer of up to T rows that the caller gives
        if t.dim() != 2 or t.shape[0] > self.T or t.shape[1] != width or t.get_device() != self._dev:
            raise ValueError(f"{name}: expected up to {self.T} rows of {width} on {self.out.device}, got {tuple(t.shape)} on "
                             f"{t.device}")
        return _array(name, t, dtype, 0)

    def _do(self, name, *args):
        if self._dev < 0:
            raise ValueError(f"{name}: the layer is not on a GPU")
        _launch(name, self._dev, None, args)

    def route(self, logits):
        at = self._rows_given("logits", logits, torch.float32, self.E)
        T, idx, w, counts, off = logits.shape[0], _p(self.topk_idx), _p(self.topk_w), _p(self.counts), _p(self.offsets)
        dst, src = _p(self.dst_row), _p(self.src_slot)
        self._do("moe_route_topk", at, T, self.E, self.k, self.capacity, idx, w, counts, off, dst, src, self.R,
                 _p(self.route_ws), self.route_ws.numel(), _p(self.dev_err))
        if self.S:
            self._do("moe_route_add_shared", self.T, self.E, self.k, self.S, self.capacity, idx, w, dst, counts, off, src,
                     self.R, _p(self.s_idx), _p(self.s_w), _p(self.s_counts), _p(self.s_off), _p(self.s_dst),
                     _p(self.s_src))

    def _permute(self, dtype, x, out, scales, row_scale):
        # the rows of x, or of an upstream gradient, to the experts
        act = torch.float32 if dtype == MOE_F32 else torch.bfloat16
        at = self._rows_given("x" if row_scale is None else "dout", x, act, self.d)
        self._do("moe_permute", dtype, at, x.shape[0], self.d, self.K, _p(self.s_dst), _p(self.s_fill), row_scale,
                 self.n_rows, _p(out), _p(scales), _p(self.dev_err))

    def _unpermute(self, y, weights, out):
        self._do("moe_unpermute_combine", MOE_F32 if self.dtype == MOE_F32 else MOE_BF16, _p(y), _p(self.s_dst), weights,
                 self.T, self.K, self.d, self.n_rows, _p(out), _p(self.dev_err))

    def _no_int4(self):
        if self.dtype == MOE_INT4:
            raise ValueError("an INT4 layer has no separate stages: forward is one call")

    def permute(self, x):
        self._no_int4()
        self._permute(self.dtype, x, self.x_perm, self.x_perm_scales, None)

    def gemm_fwd(self):
        self._no_int4()
        if self._glu is not None:
            moe_grouped_glu_fwd(self.dtype, self._glu[self.training], self.x_perm, self.w13, self.w2, self.s_off,
                                self.g_cap, self.gu, self.h, self.y_perm)
        else:
            quantised = self.dtype in (MOE_MXFP8, MOE_MXFP4)
            w13, w2, s13, s2 = ((self.w13_q, self.w2_q, self.w13_s, self.w2_s) if quantised else
                                (self.w13, self.w2, None, None))
            self._do("moe_grouped_gemm_fwd", self.dtype, _p(self.x_perm), _p(self.x_perm_scales), _p(w13), _p(s13), _p(w2),
                     _p(s2), _p(self.s_off), self.g_cap, self.G, self.n_rows, self.d, self.f, _p(self.gu), _p(self.h),
                     _p(self.y_perm), _p(self.gemm_ws), _nbytes(self.gemm_ws))

    def _gemm_bwd(self, dtype, x_perm, scales, h, w13, s13, w2, s2, ws):
        self._do("moe_grouped_gemm_bwd", dtype, _p(self.dy_perm), _p(x_perm), _p(scales), _p(self.gu), _p(h), _p(w13),
                 _p(s13), _p(w2), _p(s2), _p(self.s_off), self.g_cap, self.G, self.n_rows, self.d, self.f, _p(self.dgu),
                 _p(self.dx_perm), _p(self.dw13), _p(self.dw2), _p(ws), _nbytes(ws))

    def _slot_weights(self, weights):
        if weights is None or weights is self.s_w:
            return self.s_w
        assert not self.S, "per-row weights are not combined with shared experts"
        if weights.get_device() != self._dev:
            raise ValueError(f"weights: expected a tensor on {self.out.device}, got one on {weights.device}")
        _array("weights", weights, torch.float32, self.T * self.K)
        return weights

    def _out_drop(self):
        return self.out_dropout if self.training else 0.0

    def combine(self, weights=None, residual=None):
        self._no_int4()
        p = self._out_drop()
        if p or residual is not None:
            moe_combine_dropout(MOE_F32 if self.dtype == MOE_F32 else MOE_BF16, self.y_perm, self.s_dst,
                                self._slot_weights(weights), self.K, p, self.rng[1] if p else None, self.out,
                                residual=residual, dev_err=self.dev_err)
            return
        self._unpermute(self.y_perm, _p(self._slot_weights(weights)), self.out)

    def router_scores(self, x, w_router):
        """Router scores [T, E] fp32 = x . w_router^T (bf16 x and w_router [E, d])."""
        if getattr(self, "logits", None) is None:
            self.logits = torch.empty(self.T, self.E, dtype=torch.float32, device=x.device)
        moe_router_logits(x, w_router, self.logits)
        return self.logits

    def gate_grad(self, dout):
        """dlogits [T, E] fp32: the gradient of <dout, out> through the gate
        weights of the last forward (bf16 activations; call after forward).  dout
        is the gradient of the layer's output, whatever was dropped of it."""
        self._no_int4()
        dout = self._drop_dout(dout)
        if getattr(self, "dlogits", None) is None:
            self.dlogits = torch.empty(self.T, self.E, dtype=torch.float32, device=dout.device)
        moe_gate_grad(dout, self.y_perm, self.topk_idx, self.topk_w, self.dst_row, self.dlogits,
                      dev_err=self.dev_err)
        return self.dlogits

    def _balance_buffers(self, n):
        # Tensors for n sequences, out of the latest set made, which has at least as many.  Sets double in
        # size and are kept with the layer: a captured balance_loss replays into the one it was given.
        if not hasattr(self, "_balance_sets"):
            self._balance_sets = []
            self.balance_losses = torch.empty(2, dtype=torch.float32, device=self.device)
        if not self._balance_sets or self._balance_sets[-1][0] < n:
            m = 1 << (n - 1).bit_length()
            dev = self.device
            self._balance_sets.append((m, torch.empty(m, self.E, dtype=torch.int32, device=dev),
                                       torch.empty(m, self.E, dtype=torch.float32, device=dev),
                                       torch.empty(m + 1, dtype=torch.int32, device=dev),
                                       torch.empty(moe_balance_workspace_bytes(self.T, self.E, m), dtype=torch.uint8,
                                                   device=dev)))
        _, counts, probs, tokens, self.balance_ws = self._balance_sets[-1]
        self.balance_counts, self.balance_probs, self.balance_tokens = counts[:n], probs[:n], tokens[:n + 1]

    def balance_loss(self, logits, balance_coef, z_coef=0.0, seg_off=None, mask=None):
        """losses [2] fp32 on the device: the balance loss and the z loss of the router's
        logits under the last route, over the packed sequences seg_off [n_seg+1] int32
        (None: the batch as one), tokens with mask [T] uint8 = 0 left out.  The counts
        and mean probabilities per sequence stay in balance_counts, balance_probs until
        the next call."""
        self._balance_buffers(1 if seg_off is None else seg_off.numel() - 1)
        moe_balance_loss(logits, self.topk_idx, balance_coef, z_coef, self.balance_losses, self.balance_counts,
                         self.balance_probs, None, self.balance_tokens, self.balance_ws, seg_off=seg_off, mask=mask,
                         dev_err=self.dev_err)
        self._balance = (balance_coef, z_coef, seg_off, mask)
        return self.balance_losses

    def balance_loss_grad(self, logits, dlosses=None, add_to=None):
        """dlogits [T, E]: add_to (the layer's dlogits after gate_grad, say; None: zeros) plus
        the gradient of <dlosses, losses> of the last balance_loss.  It is the one tensor that
        gate_grad writes too: pass add_to=self.dlogits for the sum of both."""
        cb, cz, seg_off, mask = self._balance
        if getattr(self, "dlogits", None) is None:
            self.dlogits = torch.empty(self.T, self.E, dtype=torch.float32, device=logits.device)
        moe_balance_loss_bwd(logits, self.balance_counts, self.balance_tokens, cb, cz, self.dlogits,
                             dlosses=dlosses, add=add_to, seg_off=seg_off, mask=mask)
        return self.dlogits

    def next_mask(self):
        """Advance the steps of both masks (forward does)."""
        if self.rng is not None:
            self._rng_step.add_(1)

    def _drop_dout(self, dout):
        # the upstream gradient under the output's mask
        p = self._out_drop()
        if not p:
            return dout
        if getattr(self, "dsum", None) is None:
            self.dsum = torch.empty(self.T, self.d, dtype=_ACT[self.dtype], device=self.device)
        moe_dropout(MOE_F32 if self.dtype == MOE_F32 else MOE_BF16, dout, p, self.rng[1], self.dsum)
        return self.dsum

    def forward(self, logits, x, weights=None, residual=None, same_mask=False):
        """out [T, d]: the layer's output, dropped by out_dropout and added to residual [T, d] if
        given (whose gradient is dout itself)."""
        if self.dtype == MOE_INT4:
            if weights is not None or residual is not None:
                raise ValueError("an INT4 layer takes neither weights nor a residual")
            if self.w13_4 is None:
                raise ValueError("forward: the layer has no weights yet (set_weights)")
        self.route(logits)
        if self.dtype == MOE_INT4:
            moe_int4_ffn(self._glu, x, self.s_idx, self.s_w, self.s_dst, self.s_src, self.s_off, self.group,
                         self.w13_4, self.w2_4, self.out, self.int4_ws, dev_err=self.dev_err)
            return self.out
        if self.training and not same_mask:
            self.next_mask()
        self.permute(x)
        self.gemm_fwd()
        self.combine(weights, residual)
        return self.out

    def backward(self, dout, weights=None):
        self._alloc_bwd()
        dout = self._drop_dout(dout)
        act_dt = MOE_F32 if self.dtype == MOE_F32 else MOE_BF16
        self._permute(act_dt, dout, self.dy_perm, None, _p(self._slot_weights(weights)))
        if self._glu is not None:
            moe_grouped_glu_bwd(self.dtype, self._glu[self.training], self.dy_perm, self.x_perm, self.gu, self.h,
                                self.w13, self.w2, self.s_off, self.g_cap, self.dgu, self.dx_perm, self.dw13,
                                self.dw2, ws=self.gemm_ws)
        elif self.dtype == MOE_MXFP8:
            self._gemm_bwd(MOE_MXFP8, self.x_perm, self.x_perm_scales, self.h, self.w13t_q, self.w13t_s, self.w2t_q,
                           self.w2t_s, self.gemm_ws)
        elif self.dtype == MOE_MXFP4:
            if self.w13 is None:
                self._decode_weights()
            self._decode_rows()
            self._gemm_bwd(MOE_BF16, self.x_perm_d, None, self.h_d, self.w13_d, None, self.w2_d, None, self.bwd_ws)
        else:
            self._gemm_bwd(self.dtype, self.x_perm, None, self.h, self.w13, None, self.w2, None, self.gemm_ws)
        self._unpermute(self.dx_perm, None, self.dx)
        return self.dx, self.dw13, self.dw2
