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
import torch

from . import (MOE_BF16, MOE_F32, MOE_GEMM_DGRAD_DOWN, MOE_GEMM_DGRAD_GATE_UP, MOE_GEMM_WGRAD,
               MOE_MXFP4, MOE_MXFP8,
               gemm_tensors, moe_balance_loss, moe_balance_loss_bwd, moe_balance_workspace_bytes,
               moe_dequantize_mxfp4, moe_gemm_workspace_bytes, moe_grouped_gemm_bwd, moe_grouped_gemm_fwd,
               moe_gate_grad, moe_grouped_gemm_op, moe_permute, moe_quantize_mxfp4, moe_quantize_mxfp8,
               moe_route_add_shared, moe_route_topk, moe_route_workspace_bytes, moe_router_logits,
               moe_unpermute_combine)

_ACT = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16, MOE_MXFP8: torch.bfloat16,
        MOE_MXFP4: torch.bfloat16}


class MoELayer:
    """n_shared > 0 adds that many shared experts (ungated, every token, weight
    1) as extra groups E .. E+n_shared-1 of the same grouped GEMM: weights are
    then [E + n_shared, ...] with the shared experts last, and the buffers hold
    the routed rows followed by n_shared * T shared rows.  save=False (MXFP4
    only) keeps no activations for a backward, as serving wants it.
    decode_h=True (MXFP4 only): dw2 from the 4-bit h."""

    def __init__(self, T, d, E, f, k, dtype=MOE_BF16, capacity=0, device="cuda", n_shared=0, save=True,
                 decode_h=False):
        if not save and dtype != MOE_MXFP4:
            raise ValueError("save=False: only the MXFP4 forward runs without its saved activations")
        if decode_h and (dtype != MOE_MXFP4 or not save):
            raise ValueError("decode_h=True: only an MXFP4 layer with saved activations has an h in 4 bits to decode")
        self.save, self.decode_h = save, decode_h
        self.T, self.d, self.E, self.f, self.k = T, d, E, f, k
        self.dtype, self.capacity, self.device = dtype, capacity, device
        self.S = n_shared
        self.K = k + n_shared                  # slots per token (routed, then shared)
        self.G = E + n_shared                  # GEMM groups
        self.R = E * capacity if capacity > 0 else T * k   # routed rows
        self.n_rows = self.R + n_shared * T
        R = self.n_rows
        act = _ACT[dtype]
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
        if dtype == MOE_MXFP8:
            self.x_perm = torch.empty(R, d, dtype=torch.uint8, device=device)
            self.x_perm_scales = torch.empty(R, d // 32, dtype=torch.uint8, device=device)
        elif dtype == MOE_MXFP4:
            self.x_perm = torch.empty(R, d // 2, dtype=torch.uint8, device=device)
            self.x_perm_scales = torch.empty(R, d // 32, dtype=torch.uint8, device=device)
        else:
            self.x_perm = torch.empty(R, d, dtype=act, device=device)
            self.x_perm_scales = None
        self.gu = torch.empty(R, 2 * f, dtype=act, device=device) if save else None
        self.h = torch.empty(R, f, dtype=act, device=device) if save else None
        self.y_perm = torch.empty(R, d, dtype=act, device=device)
        self.out = torch.empty(T, d, dtype=act, device=device)
        self.gemm_ws = None
        wsb = moe_gemm_workspace_bytes(dtype, self.G, R, d, f)
        if wsb:
            self.gemm_ws = torch.empty(wsb, dtype=torch.uint8, device=device)
        self._bwd_alloc = False

    def _alloc_bwd(self):
        if self._bwd_alloc:
            return
        if not self.save:
            raise RuntimeError("a layer made with save=False has no backward")
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
    def set_weights(self, w13, w2):
        """Weights [E, 2f, d] and [E, d, f] (MOE_F32: fp32, otherwise bf16).  For MXFP8
        the forward and backward MXFP8 caches are made here (once per optimizer
        step), for MXFP4 the codes of both; MXFP4 weights that are refused leave
        the layer with the ones it had.  Each call makes new caches and a captured
        graph reads those of its capture: for weights that change under a graph,
        write them into w13 and w2 and call requantize_weights, which works in place."""
        if self.dtype == MOE_MXFP4:
            E, f, d = self.G, self.f, self.d
            for name, w, n in (("w13", w13, E * 2 * f * d), ("w2", w2, E * d * f)):
                if w.dtype is not torch.bfloat16 or w.numel() != n or w.get_device() != self.x_perm.get_device():
                    raise ValueError(f"{name}: expected a torch.bfloat16 tensor of {n} elements on {self.x_perm.device}, "
                                     f"got {w.dtype} {tuple(w.shape)} on {w.device}")
            u8 = dict(dtype=torch.uint8, device=self.device)
            codes = (torch.empty(E, 2 * f, d // 2, **u8), torch.empty(E, 2 * f, d // 32, **u8),
                     torch.empty(E, d, f // 2, **u8), torch.empty(E, d, f // 32, **u8))
            self._quantize_mxfp4(w13, w2, *codes)
            self.set_weights_mxfp4(*codes)
            self.w13, self.w2 = w13, w2
            if self._bwd_alloc:
                self._decode_weights()
            return
        self.w13, self.w2 = w13, w2
        self._stages = None
        if self.dtype != MOE_MXFP8:
            return
        E, f, d = self.G, self.f, self.d
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
        self.w13_q, self.w13_s, self.w2_q, self.w2_s = w13_q, w13_s, w2_q, w2_s
        self.w13 = self.w2 = None   # these codes have no bf16 weights behind them
        self._stages = None

    def _quantize_mxfp4(self, w13, w2, w13_q, w13_s, w2_q, w2_s):
        E, f, d = self.G, self.f, self.d
        moe_quantize_mxfp4(w13.reshape(E * 2 * f, d), w13_q.view(E * 2 * f, -1), w13_s.view(E * 2 * f, -1))
        moe_quantize_mxfp4(w2.reshape(E * d, f), w2_q.view(E * d, -1), w2_s.view(E * d, -1))

    def requantize_weights(self):
        """MXFP8: rebuild the four weight caches (forward and backward direction
        of w13 and w2) from the bf16 weights in place, as an optimizer step does.
        MXFP4: rebuild the codes."""
        E, f, d = self.G, self.f, self.d
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
    def route(self, logits):
        moe_route_topk(logits, self.k, self.capacity, self.topk_idx, self.topk_w, self.counts,
                       self.offsets, self.dst_row, self.src_slot, self.route_ws, self.dev_err)
        if self.S:
            moe_route_add_shared(self.S, self.capacity, self.topk_idx, self.topk_w, self.dst_row,
                                 self.counts, self.offsets, self.src_slot, self.s_idx, self.s_w,
                                 self.s_counts, self.s_off, self.s_dst, self.s_src)

    def permute(self, x):
        moe_permute(self.dtype, x, self.K, self.s_dst, self.x_perm, src_slot=self.s_fill,
                    x_perm_scales=self.x_perm_scales, dev_err=self.dev_err)

    def gemm_fwd(self):
        if self.dtype in (MOE_MXFP8, MOE_MXFP4):
            moe_grouped_gemm_fwd(self.dtype, self.x_perm, self.w13_q, self.w2_q, self.s_off,
                                 self.g_cap, self.gu, self.h, self.y_perm,
                                 x_perm_scales=self.x_perm_scales, w13_scales=self.w13_s,
                                 w2_scales=self.w2_s, ws=self.gemm_ws)
        else:
            moe_grouped_gemm_fwd(self.dtype, self.x_perm, self.w13, self.w2, self.s_off,
                                 self.g_cap, self.gu, self.h, self.y_perm)

    def _slot_weights(self, weights):
        if weights is None or weights is self.s_w:
            return self.s_w
        assert not self.S, "per-row weights are not combined with shared experts"
        return weights

    def combine(self, weights=None):
        moe_unpermute_combine(MOE_F32 if self.dtype == MOE_F32 else MOE_BF16, self.y_perm,
                              self.s_dst, self._slot_weights(weights), self.K, self.out,
                              dev_err=self.dev_err)

    def router_scores(self, x, w_router):
        """Router scores [T, E] fp32 = x . w_router^T (bf16 x and w_router [E, d])."""
        if getattr(self, "logits", None) is None:
            self.logits = torch.empty(self.T, self.E, dtype=torch.float32, device=x.device)
        moe_router_logits(x, w_router, self.logits)
        return self.logits

    def gate_grad(self, dout):
        """dlogits [T, E] fp32: the gradient of <dout, out> through the gate
        weights of the last forward (bf16 activations; call after forward)."""
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

    def forward(self, logits, x, weights=None):
        self.route(logits)
        self.permute(x)
        self.gemm_fwd()
        self.combine(weights)
        return self.out

    def backward(self, dout, weights=None):
        self._alloc_bwd()
        act_dt = MOE_F32 if self.dtype == MOE_F32 else MOE_BF16
        moe_permute(act_dt, dout, self.K, self.s_dst, self.dy_perm, src_slot=self.s_fill,
                    row_scale=self._slot_weights(weights), dev_err=self.dev_err)
        if self.dtype == MOE_MXFP8:
            moe_grouped_gemm_bwd(self.dtype, self.dy_perm, self.x_perm, self.gu, self.h,
                                 self.w13t_q, self.w2t_q, self.s_off, self.g_cap, self.dgu,
                                 self.dx_perm, self.dw13, self.dw2,
                                 x_perm_scales=self.x_perm_scales, w13_scales=self.w13t_s,
                                 w2_scales=self.w2t_s, ws=self.gemm_ws)
        elif self.dtype == MOE_MXFP4:
            if self.w13 is None:
                self._decode_weights()
            self._decode_rows()
            moe_grouped_gemm_bwd(MOE_BF16, self.dy_perm, self.x_perm_d, self.gu, self.h_d, self.w13_d, self.w2_d,
                                 self.s_off, self.g_cap, self.dgu, self.dx_perm, self.dw13, self.dw2,
                                 ws=self.bwd_ws)
        else:
            moe_grouped_gemm_bwd(self.dtype, self.dy_perm, self.x_perm, self.gu, self.h,
                                 self.w13, self.w2, self.s_off, self.g_cap, self.dgu,
                                 self.dx_perm, self.dw13, self.dw2, ws=self.gemm_ws)
        moe_unpermute_combine(act_dt, self.dx_perm, self.s_dst, None, self.K, self.dx,
                              dev_err=self.dev_err)
        return self.dx, self.dw13, self.dw2
