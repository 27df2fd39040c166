"""One GPU's share of a sparse MoE layer as a sequence of libmoe calls on one stream.

    router logits -> route -> dispatch layout -> permute -> grouped SwiGLU FFN (+ shared expert)
    -> combine

("MoE part 4" page, section 4 and 4.2; "EP / DeepEP explanation" page, sections 2-3.)
Given the router weight W_r the layer computes the logits z = x W_r^T itself; without
it, forward takes z.
All buffers are allocated once, at construction, so a forward pass enqueues
only kernels: no allocation, no host synchronisation, no device-to-host copy.

bf16 layers fold the permute into the gate/up GEMM by default (``gather=True``): its
operand rows are read straight from x through the layout's src_slot map, so the
permuted copy of x is never written.  f32 layers run the permute kernel.  fp8 layers with a
shared expert and more than 16 rows per expert on average quantize each token once (its
fp8 payload), turn the codes back into bf16 values once, and gather those rows the same way;
other fp8 layers run the quantize-on-permute kernel.  Layers with gathered rows also run
the shared expert inside the routed GEMM launches by default (``fuse_shared=True``): its
rows follow the routed rows in h and in the expert outputs.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (MOE_ACT_GELU_TANH, MOE_ACT_NONE, MOE_ACT_SILU, MOE_BF16, MOE_BF16X3, MOE_F32, MOE_FP8_E4M3,
               MOE_MX_BLOCK, MOE_OP_ACT_BACKWARD, MOE_OP_BALANCE_LOSS, MOE_OP_DISPATCH_LAYOUT, MOE_OP_EXPERT_DGRAD,
               MOE_OP_EXPERT_GEMM, MOE_OP_EXPERT_LINEAR, MOE_OP_GROUPED_FFN, MOE_OP_ROUTER, MOE_OP_ROUTER_WGRAD,
               moe_balance_loss, moe_balance_loss_backward, moe_combine, moe_combine_backward, moe_combine_dropout,
               moe_combine_dropout_backward, moe_dequantize_fp8, moe_dequantize_mxfp8, moe_dispatch_layout,
               moe_dropout, moe_expert_act_backward, moe_expert_dgrad, moe_expert_down, moe_expert_down_shared,
               moe_expert_down_shared_e4m3, moe_expert_gate_up, moe_expert_gate_up_gathered,
               moe_expert_gate_up_gathered_shared, moe_expert_gate_up_gathered_shared_e4m3, moe_expert_gate_up_mxfp8,
               moe_expert_gate_up_preact, moe_expert_linear, moe_expert_wgrad, moe_grouped_ffn, moe_permute,
               moe_quantize_fp8, moe_quantize_mxfp8, moe_route, moe_router_backward, moe_router_dense_dgrad,
               moe_router_dense_wgrad, moe_router_input_grad, moe_router_logits, moe_swiglu_backward,
               moe_swiglu_backward_mxfp8, moe_workspace_bytes, _balance_args, _expect)


def _expect_dense(name: str, t: Optional[torch.Tensor], align: int = 16) -> None:
    """Raises ValueError unless t (if given) lies in one piece, at a multiple of align bytes."""
    if t is None or (t.is_contiguous() and t.data_ptr() % align == 0):
        return
    raise ValueError(f"{name} must be contiguous" if not t.is_contiguous() else f"{name} must be {align}-byte aligned")


def _check_drop(N, H, dtype, device, residual, dropout, rng):
    """Raises ValueError unless residual, dropout and rng fit a layer's forward."""
    if not 0.0 <= dropout <= 1.0:
        raise ValueError(f"dropout must lie in 0 .. 1, not {dropout}")
    if dropout > 0.0 and rng is None:
        raise ValueError("dropout needs rng, the generator's state (device int64 [2]: seed, offset)")
    _expect("rng", rng, (2,), (torch.int64,), device)
    _expect("residual", residual, (N, H), (dtype,), device)
    _expect_dense("residual", residual)


class MoELayer:
    """Pre-planned MoE layer for fixed sizes.

    ``dtype``: 'f32' (fp32 everywhere), 'bf16' (bf16 storage, fp32 accumulation) or
    'fp8' (bf16 hidden states; e4m3 payload and weights with per-128-column fp32
    scales; bf16 h, expert outputs and y).  Weights come in the storage dtype
    (bf16 for 'fp8'); the fp8 layer quantizes them once here, with the library's
    own row quantizer.  ``w_r`` [E, H] (storage dtype): the router weight; the
    logits then come from moe_router_logits on x.
    """

    def __init__(self, N: int, H: int, E: int, k: int, I: int, dtype: str, w13: torch.Tensor,
                 w2: torch.Tensor, shared_w13: Optional[torch.Tensor] = None,
                 shared_w2: Optional[torch.Tensor] = None, n_group: int = 0, topk_group: int = 0,
                 bias: Optional[torch.Tensor] = None, gather: bool = True, overlap_shared: bool = False,
                 fuse_shared: bool = True, gate_in_down: bool = False, w_r: Optional[torch.Tensor] = None):
        self.N, self.H, self.E, self.k, self.I = N, H, E, k, I
        self.dtype, self.n_group, self.topk_group, self.bias = dtype, n_group, topk_group, bias
        dev = w13.device
        self.device = dev
        self.fp8 = dtype == "fp8"
        # fp8 above decode sizes (more than 16 rows per expert on average) with a shared expert:
        # the gathered, fused path on e4m3 weights; at decode sizes the weight-streaming kernels
        self.fp8_gather = bool(self.fp8 and gather and fuse_shared and shared_w13 is not None and N * k > 16 * E)
        self.gather = gather and (dtype == "bf16" or self.fp8_gather)
        act = torch.float32 if dtype == "f32" else torch.bfloat16
        self.act_dtype = act
        rows = N * k
        if self.fp8:
            self.w13, self.w13_scale = moe_quantize_fp8(w13)
            self.w2, self.w2_scale = moe_quantize_fp8(w2)
            if shared_w13 is not None:
                self.sw13, self.sw13_scale = moe_quantize_fp8(shared_w13)
                self.sw2, self.sw2_scale = moe_quantize_fp8(shared_w2)
        else:
            self.w13, self.w2, self.w13_scale, self.w2_scale = w13, w2, None, None
            self.sw13, self.sw2 = shared_w13, shared_w2
            self.sw13_scale = self.sw2_scale = None
        self.shared = shared_w13 is not None
        self.fuse = bool(fuse_shared and self.shared and self.gather)
        # the routed rows' gates applied in the down GEMM's epilogue (combine then sums)
        self.gate_in_down = bool(gate_in_down and self.fuse and not self.fp8)
        i32 = dict(dtype=torch.int32, device=dev)
        self.w_r = w_r
        if w_r is not None:
            self.z = torch.empty((N, E), dtype=torch.float32, device=dev)
            x_dt = MOE_F32 if dtype == "f32" else MOE_BF16
            self.router_ws = torch.empty(max(moe_workspace_bytes(MOE_OP_ROUTER, N, H, 0, E, 0, x_dt), 256),
                                         dtype=torch.uint8, device=dev)
        self.topk_idx = torch.empty((N, k), **i32)
        self.topk_gate = torch.empty((N, k), dtype=torch.float32, device=dev)
        self.layout = (torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(rows, **i32),
                       torch.empty(rows, **i32))
        self.layout_ws = torch.empty(max(moe_workspace_bytes(MOE_OP_DISPATCH_LAYOUT, N, 0, 0, E, k, 0), 256),
                                     dtype=torch.uint8, device=dev)
        a_dt = MOE_FP8_E4M3 if self.fp8 else (MOE_F32 if dtype == "f32" else MOE_BF16)
        self.a_dt = a_dt
        self.x_perm = None if self.gather else torch.empty((rows, H), dtype=torch.uint8 if self.fp8 else act,
                                                          device=dev)
        self.x_perm_scale = (torch.empty((rows, H // 128), dtype=torch.float32, device=dev)
                             if self.fp8 and not self.gather else None)
        if self.fp8_gather:
            # each token's fp8 payload (codes and block scales) and its values as bf16 rows
            self.x_q = torch.empty((N, H), dtype=torch.uint8, device=dev)
            self.x_q_scale = torch.empty((N, H // 128), dtype=torch.float32, device=dev)
            self.x_deq = torch.empty((N, H), dtype=torch.bfloat16, device=dev)
        self.ffn_ws = None if self.fuse else torch.empty(
            max(moe_workspace_bytes(MOE_OP_GROUPED_FFN, rows, H, I, E, 1, a_dt), 256), dtype=torch.uint8, device=dev)
        if self.fuse:
            # routed rows then the shared expert's N rows, in h and in the expert outputs
            self.h_all = torch.empty((rows + N, I), dtype=torch.bfloat16, device=dev)
            self.out_all = torch.empty((rows + N, H), dtype=act, device=dev)
            self.fused_ws = torch.empty(max(moe_workspace_bytes(MOE_OP_EXPERT_GEMM, rows + N, H, I, E + 1, 1,
                                                                MOE_BF16 if self.fp8 else a_dt), 256),
                                        dtype=torch.uint8, device=dev)
        else:
            self._expert_out = torch.empty((rows, H), dtype=act, device=dev)
        if self.shared and not self.fuse:
            self.shared_offsets = torch.tensor([0, N], **i32)
            self.x_q = torch.empty((N, H), dtype=torch.uint8, device=dev) if self.fp8 else None
            self.x_q_scale = torch.empty((N, H // 128), dtype=torch.float32, device=dev) if self.fp8 else None
            self.shared_ws = torch.empty(max(moe_workspace_bytes(MOE_OP_GROUPED_FFN, N, H, I, 1, 1, a_dt), 256),
                                         dtype=torch.uint8, device=dev)
            self._shared_out = torch.empty((N, H), dtype=act, device=dev)
        # the shared expert needs only x: it runs on a second stream (default priority)
        # beside route / layout / the routed FFN, and combine waits for it
        self.side = torch.cuda.Stream(device=dev) if self.shared and overlap_shared and not self.fuse else None
        self.shared_done = torch.cuda.Event() if self.side is not None else None
        self.y = torch.empty((N, H), dtype=act, device=dev)
        self.save_au = False     # the next forward keeps the gate/up pre-activations (training)
        self.au_saved = False    # the last forward kept them
        self.au_all = None
        self.keep8 = False       # the last forward kept the tokens and pre-activations in 8 bits
        self.kept_x = self.kept_au = None   # (codes, scales) of both
        # the balance loss of the last forward: (loss [1], counts [S, E], mean probabilities [S, E],
        # counted tokens [S]), or None; what its gradient needs; and its buffers and workspace by the
        # power of two that holds S (never replaced: a captured step keeps its memory)
        self.balance = None
        self.balance_args = None
        self.balance_bufs = {}
        self.drop_p = 0.0        # dropout of the last forward, and the generator's state that it used
        self.rng_used = None

    _WEIGHTS = ("w13", "w2", "w13_scale", "w2_scale", "sw13", "sw2", "sw13_scale", "sw2_scale", "w_r", "bias")
    _WEIGHT_GRADS = ("dw13", "dw2", "dsw13", "dsw2", "dw_r")

    def device_bytes(self) -> dict:
        """Bytes of device memory the layer holds, by kind (each allocation counted once).

        weights: the routed, shared and router weights, fp8 scales included; workspace: the
        library's scratch buffers; activations: the forward's other buffers (logits, routes,
        layout, permuted rows, h, expert outputs, y, all from construction on; the kept
        pre-activations, and the 8-bit codes of both, each once a training forward of that kind ran;
        the balance loss's).  After a backward also weight_grads and backward (its intermediates and
        workspaces).  The caller's input x is not the layer's and is not counted.
        """
        seen, out = set(), {"weights": 0, "activations": 0, "workspace": 0}

        def add(kind, v):
            for t in (v if isinstance(v, tuple) else (v,)):
                if isinstance(t, torch.Tensor) and t.is_cuda and t.untyped_storage().data_ptr() not in seen:
                    seen.add(t.untyped_storage().data_ptr())
                    out[kind] = out.get(kind, 0) + t.untyped_storage().nbytes()

        for name, v in vars(self).items():
            if name != "grads":
                add("weights" if name in self._WEIGHTS else "workspace" if name.endswith("_ws") else "activations", v)
        for v in self.balance_bufs.values():
            add("activations", v[:4])
            add("workspace", v[4])
        for name, v in (getattr(self, "grads", None) or {}).items():
            add("weight_grads" if name in self._WEIGHT_GRADS else "backward", v)
        return out

    @property
    def expert_out(self) -> torch.Tensor:
        """The routed experts' outputs [N*k, H] of the last forward."""
        return self.out_all[:self.N * self.k] if self.fuse else self._expert_out

    @property
    def shared_out(self) -> torch.Tensor:
        """The shared expert's output [N, H] of the last forward."""
        return self.out_all[self.N * self.k:] if self.fuse else self._shared_out

    @property
    def h(self) -> torch.Tensor:
        """The intermediate h of the last routed FFN (a view into the workspace)."""
        if self.fuse:
            return self.h_all[:self.N * self.k]
        off = moe_workspace_bytes(MOE_OP_EXPERT_GEMM, self.N * self.k, self.H, self.I, self.E, 1, self.a_dt)
        esz = 4 if self.dtype == "f32" else 2
        n = self.N * self.k * self.I * esz
        return self.ffn_ws[off:off + n].view(torch.float32 if esz == 4 else torch.bfloat16).view(
            self.N * self.k, self.I)

    def router(self, x: torch.Tensor):
        """Router logits z = x W_r^T into self.z."""
        return moe_router_logits(x, self.w_r, self.z, self.router_ws)

    def route(self, z: torch.Tensor):
        return moe_route(z, self.k, self.bias, self.n_group, self.topk_group, self.topk_idx, self.topk_gate)

    def dispatch(self):
        return moe_dispatch_layout(self.topk_idx, self.E, self.layout, self.layout_ws)

    def permute(self, x: torch.Tensor):
        """The permuted payload (nothing to do when the gate/up GEMM gathers its rows)."""
        send_pos = self.layout[2]
        if self.fp8_gather:   # each token once: codes and scales, then their bf16 values
            moe_quantize_fp8(x, self.x_q, self.x_q_scale)
            return moe_dequantize_fp8(self.x_q, self.x_q_scale, self.x_deq)
        if self.gather:
            return None
        if self.fp8:
            return moe_permute(x, send_pos, self.k, MOE_FP8_E4M3, self.x_perm, self.x_perm_scale)
        return moe_permute(x, send_pos, self.k, None, self.x_perm)

    def gate_up(self, x: torch.Tensor):
        """Grouped gate/up GEMM + SwiGLU into h (gathered layers read x directly; fused
        layers also compute the shared expert's rows)."""
        if self.fuse and self.fp8:
            return moe_expert_gate_up_gathered_shared_e4m3(self.x_deq, self.layout[3], self.k, self.layout[1],
                                                           self.w13, self.w13_scale, self.sw13, self.sw13_scale,
                                                           h=self.h_all, ws=self.fused_ws)
        if self.keep8:
            return moe_expert_gate_up_mxfp8(x, self.layout[3], self.k, self.layout[1], self.w13,
                                            self.sw13 if self.fuse else None, h=self.h_all if self.fuse else self.h,
                                            au_q=self.kept_au[0], au_scale=self.kept_au[1],
                                            ws=self.fused_ws if self.fuse else self.ffn_ws)
        if self.fuse:
            return moe_expert_gate_up_gathered_shared(x, self.layout[3], self.k, self.layout[1], self.w13,
                                                      self.sw13, h=self.h_all, ws=self.fused_ws,
                                                      au=self.au_all if self.save_au else None)
        if self.gather:
            return moe_expert_gate_up_gathered(x, self.layout[3], self.k, self.layout[1], self.w13,
                                               h=self.h, ws=self.ffn_ws)
        return moe_expert_gate_up(self.x_perm, self.layout[1], self.w13, self.x_perm_scale, self.w13_scale,
                                  self.h, self.ffn_ws)

    def down(self):
        """Grouped down GEMM of h into the expert outputs."""
        if self.fuse and self.fp8:
            return moe_expert_down_shared_e4m3(self.h_all, self.layout[1], self.w2, self.w2_scale, self.sw2,
                                               self.sw2_scale, self.N * self.k, out=self.out_all, ws=self.fused_ws)
        if self.fuse:
            gates = (self.layout[3], self.topk_gate) if self.gate_in_down else (None, None)
            return moe_expert_down_shared(self.h_all, self.layout[1], self.w2, self.sw2, self.N * self.k,
                                          out=self.out_all, ws=self.fused_ws, src_slot=gates[0],
                                          topk_gate=gates[1])
        return moe_expert_down(self.h, self.layout[1], self.w2, self.w2_scale, self.expert_out, self.ffn_ws)

    def experts(self, x: Optional[torch.Tensor] = None):
        if self.gather:
            self.gate_up(x)
            return self.down()
        return moe_grouped_ffn(self.x_perm, self.layout[1], self.w13, self.w2, self.x_perm_scale,
                               self.w13_scale, self.w2_scale, self.expert_out, self.ffn_ws)

    def shared_expert(self, x: torch.Tensor):
        if self.fuse:
            return None   # computed by gate_up / down
        a, a_scale = x, None
        if self.fp8:
            a, a_scale = moe_quantize_fp8(x, self.x_q, self.x_q_scale)
        return moe_grouped_ffn(a, self.shared_offsets, self.sw13, self.sw2, a_scale, self.sw13_scale,
                               self.sw2_scale, self._shared_out, self.shared_ws)

    def combine(self, residual: Optional[torch.Tensor] = None, dropout: float = 0.0,
                rng: Optional[torch.Tensor] = None):
        """y of the experts' outputs; residual, dropout and rng as forward takes them (what an earlier forward was
        given does not count)."""
        if residual is not None or dropout != 0.0:
            _check_drop(self.N, self.H, self.act_dtype, self.device, residual, dropout, rng)
            return moe_combine_dropout(self.expert_out, self.layout[2], None if self.gate_in_down else self.topk_gate,
                                       dropout, self._drop_state() if rng is None else rng,
                                       self.shared_out if self.shared else None, residual, self.y, k=self.k)
        return moe_combine(self.expert_out, self.layout[2], None if self.gate_in_down else self.topk_gate,
                           self.shared_out if self.shared else None, self.y, k=self.k)

    def _drop_state(self) -> torch.Tensor:
        """The buffer of the generator's state that the last forward used."""
        if self.rng_used is None:
            self.rng_used = torch.zeros(2, dtype=torch.int64, device=self.device)
        return self.rng_used

    def launch_shared_side(self, x: torch.Tensor):
        """Enqueue the shared expert on the side stream, after the work queued so far."""
        main = torch.cuda.current_stream(self.device)
        self.side.wait_stream(main)
        x.record_stream(self.side)
        with torch.cuda.stream(self.side):
            self.shared_expert(x)
            self.shared_done.record(self.side)

    def _keep8_buffers(self):
        """The kept codes and scales of the tokens and of all pre-activation rows."""
        u8 = dict(dtype=torch.uint8, device=self.device)
        rows = self.N * self.k + (self.N if self.fuse else 0)
        self.kept_x = (torch.empty((self.N, self.H), **u8), torch.empty((self.N, self.H // MOE_MX_BLOCK), **u8))
        self.kept_au = (torch.empty((rows, 2 * self.I), **u8), torch.empty((rows, 2 * self.I // MOE_MX_BLOCK), **u8))

    def balance_step(self, z: torch.Tensor, alpha: float, seq_start: Optional[torch.Tensor] = None,
                     token_mask: Optional[torch.Tensor] = None):
        """The balance loss of the routes of z into self.balance (see moe_balance_loss)."""
        S = 1 if seq_start is None else seq_start.numel() - 1
        cap = 1 << max(S - 1, 0).bit_length()   # (every batch may bring another S: a set for each power of two)
        if cap not in self.balance_bufs:
            i32, f32 = dict(dtype=torch.int32, device=self.device), dict(dtype=torch.float32, device=self.device)
            self.balance_bufs[cap] = (
                torch.empty(1, **f32), torch.empty((cap, self.E), **i32), torch.empty((cap, self.E), **f32),
                torch.empty(cap, **i32),
                # (more sequences never need less)
                torch.empty(max(moe_workspace_bytes(MOE_OP_BALANCE_LOSS, self.N, 0, 0, self.E, cap, 0), 256),
                            dtype=torch.uint8, device=self.device))
        loss, counts, prob_mean, tokens, ws = self.balance_bufs[cap]
        out = moe_balance_loss(z, self.topk_idx, alpha, bias=self.bias, seq_start=seq_start, token_mask=token_mask,
                               out=(loss, counts[:S], prob_mean[:S], tokens[:S]), ws=ws)
        self.balance = out
        self.balance_args = dict(z=z, alpha=alpha, seq_start=seq_start, token_mask=token_mask)
        return out

    def forward(self, x: torch.Tensor, z: Optional[torch.Tensor] = None, save_for_backward=False,
                balance_alpha: Optional[float] = None, seq_start: Optional[torch.Tensor] = None,
                token_mask: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                dropout: float = 0.0, rng: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y for tokens x; z: the router logits (computed from W_r when None).

        save_for_backward True: a bf16 layer that runs the shared expert inside the routed
        launches also keeps the gate/up pre-activations, which backward then reads instead of
        recomputing them.  "mxfp8": a bf16 layer that gathers its rows keeps x and the
        pre-activations as 8-bit codes (self.kept_x, self.kept_au); backward then reads nothing
        else of the forward but the routes, neither x nor the expert outputs.
        balance_alpha: also the balance loss of the batch's routes, into self.balance, and its
        gradient in the next backward (seq_start, token_mask: see moe_balance_loss; they, and z
        if it was passed, stay as they are until then).
        residual [N, H] of y's type: y = residual + the layer's sum.  dropout: the sum (not the residual) is
        dropped out with this probability, from the numbers of rng (device int64 [2]: seed, offset; see
        moe_combine_dropout), whose state here is kept for the next backward; the caller advances the
        offset from forward to forward.  The residual's gradient is dy."""
        if isinstance(save_for_backward, str) and save_for_backward != "mxfp8":
            raise ValueError('save_for_backward is False, True or "mxfp8"')
        if balance_alpha is None and (seq_start is not None or token_mask is not None):
            raise ValueError("seq_start and token_mask belong to a balance loss (balance_alpha)")
        keep8 = isinstance(save_for_backward, str)
        # every refusal comes before the first change: what the last forward left stays for its backward
        if keep8:
            if self.dtype != "bf16" or not self.gather or (self.shared and not self.fuse):
                raise ValueError("8-bit keeping is built for bf16 layers that gather their rows from x and run a shared "
                                 "expert inside the routed launches")
            if self.H % 128 or self.I % 128 or self.E >= 1024:
                raise ValueError("8-bit keeping is built for H and I that are multiples of 128 and fewer than 1024 experts")
            _expect("x", x, (self.N, self.H), (torch.bfloat16,), self.device)
        if z is None and self.w_r is None:
            raise ValueError("forward needs the logits z, or a layer built with the router weight w_r")
        _expect_dense("x", x)
        _expect_dense("z", z, 4)
        if balance_alpha is not None:
            S = _balance_args(self.z if z is None else z, self.topk_idx, self.bias, seq_start, token_mask)[3]
            if S > 65535:
                raise ValueError(f"a balance loss takes at most 65535 sequences, not {S}")
        _check_drop(self.N, self.H, self.act_dtype, self.device, residual, dropout, rng)
        self.drop_p = float(dropout)
        if rng is not None and (residual is not None or dropout > 0.0):
            torch.add(rng, 0, out=self._drop_state())   # (the caller may advance rng before the backward)
        self.keep8 = keep8
        self.save_au = bool(save_for_backward and not keep8 and self.fuse and not self.fp8)
        if self.save_au and self.au_all is None:
            self.au_all = torch.empty((self.N * self.k + self.N, 2 * self.I), dtype=torch.bfloat16,
                                      device=self.device)
        self.au_saved = self.save_au
        if keep8:
            if self.kept_x is None:
                self._keep8_buffers()
            moe_quantize_mxfp8(x, *self.kept_x)
        if self.side is not None:
            self.launch_shared_side(x)
        if z is None:
            z = self.router(x)
        self.route(z)
        if balance_alpha is None:
            self.balance = self.balance_args = None
        else:
            self.balance_step(z, balance_alpha, seq_start, token_mask)
        self.dispatch()
        self.permute(x)
        self.experts(x)
        if self.shared:
            if self.side is not None:
                torch.cuda.current_stream(self.device).wait_event(self.shared_done)
            else:
                self.shared_expert(x)
        self.combine(residual, self.drop_p, self.rng_used)
        return self.y

    # ---- backward (bf16 layers that gather their rows from x)

    def _alloc_backward(self, dw_dtype: torch.dtype):
        """The backward's buffers, each on the first step that needs it (a buffer is never replaced
        while dw_dtype stays, so a captured backward keeps its memory)."""
        N, H, E, k, I = self.N, self.H, self.E, self.k, self.I
        rows = N * k
        dev, bf = self.device, torch.bfloat16
        b = getattr(self, "grads", None)
        if b is None or b["dw_dtype"] != dw_dtype:
            b = {"dw_dtype": dw_dtype}

        def need(name, shape, dtype):
            if name not in b:
                b[name] = torch.empty(shape, dtype=dtype, device=dev)

        def need_ws(name, nbytes):
            need(name, (max(nbytes, 256),), torch.uint8)

        need("d_eo", (rows, H), bf)
        need("dg", (N, k), torch.float32)
        if not self.keep8:
            need("au", (rows, 2 * I), bf)
        elif self.shared or self.w_r is not None:
            need("x", (N, H), bf)   # the kept tokens' values
        need("dh", (rows, I), bf)
        need("d_au", (rows, 2 * I), bf)
        need("h", (rows, I), bf)
        need("d_perm", (rows, H), bf)
        need("x_perm", (rows, H), bf)
        need("dw13", (E, 2 * I, H), dw_dtype)
        need("dw2", (E, H, I), dw_dtype)
        need_ws("gemm_ws", moe_workspace_bytes(MOE_OP_EXPERT_GEMM, max(rows, N), H, I, E, 1, MOE_BF16))
        need_ws("dgrad_ws", moe_workspace_bytes(MOE_OP_EXPERT_DGRAD, max(rows, N), 0, 0, E, 0, 0))
        if self.drop_p > 0.0 and (self.shared or self.keep8):
            need("dy_d", (N, H), bf)   # dy behind the dropout
        if self.shared:
            # (the shared expert's steps have workspaces of their own: they may run on a
            # second stream beside the routed ones)
            need_ws("gemm_ws_s", moe_workspace_bytes(MOE_OP_EXPERT_GEMM, N, H, I, 1, 1, MOE_BF16))
            need_ws("dgrad_ws_s", moe_workspace_bytes(MOE_OP_EXPERT_DGRAD, N, 0, 0, 1, 0, 0))
            if "shared_offsets" not in b:
                b["shared_offsets"] = torch.tensor([0, N], dtype=torch.int32, device=dev)
            if not self.keep8:
                need("au_s", (N, 2 * I), bf)
            need("dh_s", (N, I), bf)
            need("d_au_s", (N, 2 * I), bf)
            need("h_s", (N, I), bf)
            need("dx_s", (N, H), bf)
            need("dsw13", (1, 2 * I, H), dw_dtype)
            need("dsw2", (1, H, I), dw_dtype)
        if self.balance_args is not None and self.w_r is not None:
            # the whole logit gradient, fp32 in three bf16 planes (the loss's part is often below half a bf16
            # step of the gates', so one rounding to bf16 would lose it); the first rounded to bf16
            need("dz_planes", (3, N, E), bf)
            b["dz_all"] = b["dz_planes"][0]
            need_ws("wgrad_ws", moe_workspace_bytes(MOE_OP_ROUTER_WGRAD, N, H, 0, E, 0, MOE_BF16X3))
        elif self.balance_args is not None:   # (the caller has the router)
            need("dz_all", (N, E), torch.float32)
        if self.w_r is not None:
            if self.balance_args is None:
                need("dz", (N, k), torch.float32)
            need("dw_r", (E, H), dw_dtype)
            need("dx_r", (N, H), bf)
        need("dx", (N, H), bf)
        self.grads = b

    def _gradients(self) -> dict:
        """self.grads without the logit gradient of the other kind of forward (an earlier one's)."""
        stale = ("dz_all", "dz_planes") if self.balance_args is None else ("dz",)
        return {n: t for n, t in self.grads.items() if n not in stale} if stale[0] in self.grads else self.grads

    def backward_steps(self, x: Optional[torch.Tensor], dy: torch.Tensor, dw_dtype: torch.dtype = torch.bfloat16,
                       d_loss: Optional[torch.Tensor] = None) -> list:
        """The backward pass as (name, call) steps in stream order (see backward)."""
        if self.dtype != "bf16" or not self.gather:
            raise ValueError("the backward pass is built for bf16 layers that gather their rows from x")
        keep8, dense = self.keep8, self.balance_args is not None
        if self.gate_in_down and not keep8:
            raise ValueError("backward needs the unscaled expert outputs (gate_in_down=False)")
        if d_loss is not None and not dense:
            raise ValueError("d_loss is the gradient of a balance loss, and the forward had none (balance_alpha)")
        if x is None and not keep8:
            raise ValueError('backward needs x unless the forward kept it (save_for_backward="mxfp8")')
        self._alloc_backward(dw_dtype)
        b = self.grads
        k, N = self.k, self.N
        rows = N * k
        offsets, send_pos, src_slot = self.layout[1], self.layout[2], self.layout[3]
        st = []
        dy_all, p = dy, self.drop_p
        if p > 0.0 and (self.shared or keep8):
            dy = b["dy_d"]
        if p > 0.0 and keep8:
            st.append(("dy_dropout", lambda: moe_dropout(dy_all, p, self.rng_used, y=dy)))
        if keep8:
            # x's values from its codes; the upstream rows before the gates (they enter behind the
            # down projection, where the gates' own gradient is <dh, h>)
            kx, (qa, sa) = self.kept_x, self.kept_au
            x = b.get("x")
            if x is not None:
                st.append(("x_values", lambda: moe_dequantize_mxfp8(kx[0], kx[1], out=x)))
            st += [
                ("dy_permute", lambda: moe_permute(dy, send_pos, k, None, b["d_eo"])),
                ("down_dgrad", lambda: moe_expert_dgrad(b["d_eo"], offsets, self.w2, b["dh"], b["dgrad_ws"])),
                ("swiglu_bwd", lambda: moe_swiglu_backward_mxfp8(qa[:rows], sa[:rows], b["dh"], send_pos,
                                                                 self.topk_gate, b["d_au"], b["h"], b["dg"])),
            ]
        else:
            st += self._preact_steps(x, dy_all)
        xp = ((lambda: moe_dequantize_mxfp8(kx[0], kx[1], out=b["x_perm"], send_pos=send_pos, k=k)) if keep8 else
              (lambda: moe_permute(x, send_pos, k, None, b["x_perm"])))
        st += [
            ("down_wgrad", lambda: moe_expert_wgrad(b["d_eo"], b["h"], offsets, dw=b["dw2"], rows=rows)),
            # the weight gradient of W13 reads the expert-ordered rows of x (a permuted copy:
            # the wgrad kernel streams its B operand in layout order)
            ("x_permute", xp),
            ("gate_up_wgrad", lambda: moe_expert_wgrad(b["d_au"], b["x_perm"], offsets, dw=b["dw13"], rows=rows)),
            ("gate_up_dgrad", lambda: moe_expert_dgrad(b["d_au"], offsets, self.w13, b["d_perm"], b["dgrad_ws"])),
        ]
        rest = None
        if self.shared:
            so = b["shared_offsets"]
            saved = self.au_saved
            au_s = self.au_all[rows:] if saved else b.get("au_s")
            if not saved and not keep8:
                st.append(("shared_preact", lambda: moe_expert_gate_up_preact(x, so, self.sw13, N, None, 1,
                                                                              b["au_s"], b["gemm_ws_s"])))
            swiglu = ((lambda: moe_swiglu_backward_mxfp8(qa[rows:], sa[rows:], b["dh_s"], d_au=b["d_au_s"], h=b["h_s"]))
                      if keep8 else (lambda: moe_swiglu_backward(au_s, b["dh_s"], b["d_au_s"], b["h_s"])))
            st += [
                ("shared_down_dgrad", lambda: moe_expert_dgrad(dy, so, self.sw2, b["dh_s"], b["dgrad_ws_s"])),
                ("shared_swiglu_bwd", swiglu),
                ("shared_down_wgrad", lambda: moe_expert_wgrad(dy, b["h_s"], so, dw=b["dsw2"], rows=N)),
                ("shared_gate_up_wgrad", lambda: moe_expert_wgrad(b["d_au_s"], x, so, dw=b["dsw13"], rows=N)),
                ("shared_gate_up_dgrad", lambda: moe_expert_dgrad(b["d_au_s"], so, self.sw13, b["dx_s"],
                                                                  b["dgrad_ws_s"])),
            ]
            rest = b["dx_s"]
        if dense:
            # the gates' gradient on the selected logits and the balance loss's on all of them
            ba, (_, counts, _, tokens) = self.balance_args, self.balance
            st.append(("logit_grad", lambda: moe_balance_loss_backward(
                ba["z"], self.topk_idx, ba["alpha"], counts, tokens, bias=self.bias, seq_start=ba["seq_start"],
                token_mask=ba["token_mask"], d_loss=d_loss, topk_gate=self.topk_gate, d_gate=b["dg"],
                dz=b["dz_all"] if self.w_r is None else b["dz_planes"])))
        if self.w_r is not None:
            # sum_j dz_tj W_r[e_tj] (+ the shared expert's input gradient); dense: over all experts
            rest_r = rest
            st += [
                ("router_bwd", lambda: moe_router_dense_wgrad(b["dz_planes"], x, dw=b["dw_r"], ws=b["wgrad_ws"])),
                ("router_dx", lambda: moe_router_dense_dgrad(b["dz_planes"], self.w_r, rest=rest_r, dx=b["dx_r"])),
            ] if dense else [
                ("router_bwd", lambda: moe_router_backward(self.topk_gate, b["dg"], offsets, src_slot, x, b["dz"],
                                                           b["dw_r"])),
                ("router_dx", lambda: moe_router_input_grad(self.w_r, self.topk_idx, b["dz"], rest_r, b["dx_r"])),
            ]
            rest = b["dx_r"]
        rest_x = rest
        st.append(("dx", lambda: moe_combine(b["d_perm"], send_pos, None, rest_x, b["dx"], k=k)))
        return st

    def _preact_steps(self, x: torch.Tensor, dy: torch.Tensor) -> list:
        """Up to the SwiGLU backward, with bf16 pre-activations."""
        b, k = self.grads, self.k
        rows = self.N * k
        offsets, send_pos, src_slot = self.layout[1], self.layout[2], self.layout[3]
        # the pre-activations: kept by the forward, or recomputed here
        saved = self.au_saved
        au = self.au_all[:rows] if saved else b["au"]
        st = [
            ("combine_bwd", lambda: moe_combine_dropout_backward(
                dy, send_pos, self.topk_gate, self.expert_out, self.drop_p, self.rng_used, b["d_eo"], b["dg"],
                b["dy_d"] if self.shared else None) if self.drop_p > 0.0 else
             moe_combine_backward(dy, send_pos, self.topk_gate, self.expert_out, b["d_eo"], b["dg"])),
        ]
        if not saved:
            st.append(("gate_up_preact", lambda: moe_expert_gate_up_preact(x, offsets, self.w13, rows, src_slot, k,
                                                                           b["au"], b["gemm_ws"])))
        st += [
            ("down_dgrad", lambda: moe_expert_dgrad(b["d_eo"], offsets, self.w2, b["dh"], b["dgrad_ws"])),
            ("swiglu_bwd", lambda: moe_swiglu_backward(au, b["dh"], b["d_au"], b["h"])),
        ]
        return st

    def backward(self, x: Optional[torch.Tensor], dy: torch.Tensor, dw_dtype: torch.dtype = torch.bfloat16,
                 overlap_shared: bool = False, d_loss: Optional[torch.Tensor] = None) -> dict:
        """Gradients of the last forward for the upstream gradient dy [N, H] (bf16).

        The backward mirrors the forward ("DeepSeek MoE: EP and FSDP guide": dispatch's
        backward is combine): combine backward (d_expert_out, d_gate); the gate/up
        pre-activations recomputed; dh = d_expert_out W_down; SwiGLU backward; the weight
        gradients dW_down = d_expert_out^T h and dW13 = d_au^T x per expert; the input
        gradient of every slot d_au W13; the same for the shared expert on dy; the gates'
        and router's gradients; dx = the slots' gradients summed back to their tokens plus
        the shared expert's and the router's.  Buffers are allocated on the first call.
        Returns the dict of gradient tensors ('dx', 'dw13', 'dw2', 'dsw13', 'dsw2', 'dw_r', ...).
        With overlap_shared the shared expert's steps (which need only x, dy and its
        pre-activations) run on a second stream (default priority) beside the routed ones, and
        the input-gradient sum waits for them.

        After a forward with save_for_backward="mxfp8" x may be None: the tokens and
        pre-activations are the kept codes' values, h and the gates' gradient come from them
        (d_gate = <dy W_down, h>), and the expert outputs are not read.  After a forward with a
        balance loss its gradient times d_loss ([1] fp32, None: 1) joins the gates' in the logits'
        gradient, which then gives dW_r and the router's share of dx: 'dz_planes' [3, N, E], three bf16
        planes whose sum is the fp32 gradient, the first of them 'dz_all' [N, E] (without w_r only 'dz_all',
        in fp32).
        """
        steps = self.backward_steps(x, dy, dw_dtype, d_loss)
        if not (overlap_shared and self.shared):
            for _, f in steps:
                f()
            return self._gradients()
        main = torch.cuda.current_stream(self.device)
        if getattr(self, "bwd_side", None) is None:
            self.bwd_side = torch.cuda.Stream(device=self.device)
            self.bwd_side_done = torch.cuda.Event()
        side = self.bwd_side
        # what both streams read
        both = ("x_values", "dy_dropout") + (("combine_bwd",) if self.drop_p > 0.0 else ())
        for name, f in steps:
            if name in both:
                f()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for name, f in steps:
                if name.startswith("shared_"):
                    f()
            self.bwd_side_done.record(side)
        for name, f in steps:
            if name.startswith("shared_") or name in both:
                continue
            if name in ("router_dx", "dx") and not getattr(self, "_waited", False):
                main.wait_event(self.bwd_side_done)   # the shared expert's dx joins here
                self._waited = True
            f()
        self._waited = False
        for t in (x, dy):
            if t is not None:
                t.record_stream(side)
        return self._gradients()


class BiasedMoELayer:
    """Pre-planned MoE layer whose experts are act(x W1^T + b1) W2^T + b2.

    The router, layout and combine of MoELayer around other experts: w1 [E, I, H] (gated: [E, 2I, H],
    h = act of the first half times the second), w2 [E, H, I], biases b1 [E, I or 2I] and b2 [E, H]
    (fp32 or the weights' type) or None, act one of MOE_ACT_*.  The weights' type (float32 or bfloat16) is the
    layer's.  forward adds the residual stream and drops out as MoELayer's does; backward is
    built for bf16 layers with H and I multiples of 128 (the sizes of moe_expert_dgrad and
    moe_expert_wgrad).  All buffers are allocated at construction or on the first backward.
    """

    def __init__(self, N: int, H: int, E: int, k: int, I: int, w1: torch.Tensor, w2: torch.Tensor,
                 b1: Optional[torch.Tensor] = None, b2: Optional[torch.Tensor] = None, act: int = MOE_ACT_GELU_TANH,
                 gated: bool = False, n_group: int = 0, topk_group: int = 0, bias: Optional[torch.Tensor] = None,
                 w_r: Optional[torch.Tensor] = None):
        if not MOE_ACT_NONE <= act <= MOE_ACT_SILU:
            raise ValueError(f"act must be one of MOE_ACT_*, not {act}")
        dt, dev = w1.dtype, w1.device
        Nw = 2 * I if gated else I
        if dt not in (torch.float32, torch.bfloat16):
            raise ValueError(f"w1 must be float32 or bfloat16, not {dt}")
        _expect("w1", w1, (E, Nw, H), (dt,), dev)
        _expect("w2", w2, (E, H, I), (dt,), dev)
        _expect("b1", b1, (E, Nw), (torch.float32, dt), dev)
        _expect("b2", b2, (E, H), (torch.float32, dt), dev)
        _expect("bias", bias, (E,), (torch.float32,), dev)
        _expect("w_r", w_r, (E, H), (dt,), dev)
        for name, t in (("w1", w1), ("w2", w2), ("b1", b1), ("b2", b2), ("w_r", w_r)):
            _expect_dense(name, t)
        _expect_dense("bias", bias, 4)
        self.N, self.H, self.E, self.k, self.I = N, H, E, k, I
        self.w1, self.w2, self.b1, self.b2, self.act, self.gated = w1, w2, b1, b2, act, bool(gated)
        self.n_group, self.topk_group, self.bias, self.w_r = n_group, topk_group, bias, w_r
        self.act_dtype, self.device = dt, dev
        c_dt = MOE_F32 if dt == torch.float32 else MOE_BF16
        rows = N * k

        def ws(*args):
            return torch.empty(max(moe_workspace_bytes(*args), 256), dtype=torch.uint8, device=dev)

        i32 = dict(dtype=torch.int32, device=dev)
        if w_r is not None:
            self.z = torch.empty((N, E), dtype=torch.float32, device=dev)
            self.router_ws = ws(MOE_OP_ROUTER, N, H, 0, E, 0, c_dt)
        self.topk_idx = torch.empty((N, k), **i32)
        self.topk_gate = torch.empty((N, k), dtype=torch.float32, device=dev)
        self.layout = (torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(rows, **i32),
                       torch.empty(rows, **i32))
        self.layout_ws = ws(MOE_OP_DISPATCH_LAYOUT, N, 0, 0, E, k, 0)
        self.fc1_ws = ws(MOE_OP_EXPERT_LINEAR, rows, H, Nw, E, 0, c_dt)
        self.fc2_ws = ws(MOE_OP_EXPERT_LINEAR, rows, I, H, E, 0, c_dt)
        self.h = torch.empty((rows, I), dtype=dt, device=dev)
        self.expert_out = torch.empty((rows, H), dtype=dt, device=dev)
        self.y = torch.empty((N, H), dtype=dt, device=dev)
        self.pre = None          # the pre-activations [rows, I or 2I] of a forward that keeps them
        self.saved = False       # the last forward kept them
        self.drop_p = 0.0
        self.rng_used = torch.zeros(2, dtype=torch.int64, device=dev)
        self.grads = None

    def forward(self, x: torch.Tensor, z: Optional[torch.Tensor] = None, save_for_backward: bool = False,
                residual: Optional[torch.Tensor] = None, dropout: float = 0.0,
                rng: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y [N, H] for tokens x (z: the router logits, computed from w_r when None); residual, dropout and rng as
        MoELayer.forward takes them.  save_for_backward keeps the pre-activations for backward."""
        N, E, k, dt = self.N, self.E, self.k, self.act_dtype
        _expect("x", x, (N, self.H), (dt,), self.device)
        if z is None and self.w_r is None:
            raise ValueError("forward needs the logits z, or a layer built with the router weight w_r")
        _expect("z", z, (N, E), (torch.float32,), self.device)
        _expect_dense("x", x)
        _expect_dense("z", z, 4)
        _check_drop(N, self.H, dt, self.device, residual, dropout, rng)
        self.drop_p = float(dropout)
        if rng is not None:
            torch.add(rng, 0, out=self.rng_used)   # (the caller may advance rng before the backward)
        if save_for_backward and self.pre is None:
            self.pre = torch.empty((N * k, self.w1.shape[1]), dtype=dt, device=self.device)
        self.saved = bool(save_for_backward)
        if z is None:
            z = moe_router_logits(x, self.w_r, self.z, self.router_ws)
        moe_route(z, k, self.bias, self.n_group, self.topk_group, self.topk_idx, self.topk_gate)
        _, offsets, send_pos, src_slot = moe_dispatch_layout(self.topk_idx, E, self.layout, self.layout_ws)
        moe_expert_linear(x, self.w1, self.b1, offsets, self.act, self.gated, src_slot, k, out=self.h,
                          z=self.pre if self.saved else None, ws=self.fc1_ws)
        moe_expert_linear(self.h, self.w2, self.b2, offsets, out=self.expert_out, ws=self.fc2_ws)
        return moe_combine_dropout(self.expert_out, send_pos, self.topk_gate, self.drop_p, self.rng_used,
                                   residual=residual, y=self.y)

    def backward(self, x: torch.Tensor, dy: torch.Tensor, dw_dtype: torch.dtype = torch.bfloat16) -> dict:
        """Gradients of the last forward (with save_for_backward) for the upstream gradient dy [N, H] bf16: 'dx',
        'dw1', 'dw2', 'db1', 'db2' (fp32), 'dg' (the gates'), with w_r 'dz' (the selected logits') and 'dw_r'.  The
        residual's gradient is dy."""
        N, H, E, k, I = self.N, self.H, self.E, self.k, self.I
        bf, dev, rows = torch.bfloat16, self.device, self.N * self.k
        if self.act_dtype != bf or H % 128 or I % 128:
            raise ValueError("backward is built for bf16 layers with H and I multiples of 128")
        if not self.saved:
            raise ValueError("backward needs a forward with save_for_backward")
        _expect("x", x, (N, H), (bf,), dev)
        _expect("dy", dy, (N, H), (bf,), dev)
        b = self.grads
        if b is None or b["dw1"].dtype != dw_dtype:
            def new(*shape, dtype=bf):
                return torch.empty(shape, dtype=dtype, device=dev)

            Nw = self.w1.shape[1]
            b = dict(d_eo=new(rows, H), dg=new(N, k, dtype=torch.float32), dh=new(rows, I), dpre=new(rows, Nw),
                     x_perm=new(rows, H), d_perm=new(rows, H), dx=new(N, H),
                     dw1=new(E, Nw, H, dtype=dw_dtype), dw2=new(E, H, I, dtype=dw_dtype),
                     db1=new(E, Nw, dtype=torch.float32), db2=new(E, H, dtype=torch.float32))
            for name, args in (("act_ws", (MOE_OP_ACT_BACKWARD, rows, 0, Nw, E, 0, 0)),
                               ("b2_ws", (MOE_OP_ACT_BACKWARD, rows, 0, H, E, 0, 0)),
                               ("dgrad_ws", (MOE_OP_EXPERT_DGRAD, rows, 0, 0, E, 0, 0))):
                b[name] = torch.empty(max(moe_workspace_bytes(*args), 256), dtype=torch.uint8, device=dev)
            if self.w_r is not None:
                b.update(dz=new(N, k, dtype=torch.float32), dw_r=new(E, H, dtype=dw_dtype), dx_r=new(N, H))
            self.grads = b
        _, offsets, send_pos, src_slot = self.layout
        moe_combine_dropout_backward(dy, send_pos, self.topk_gate, self.expert_out, self.drop_p, self.rng_used, b["d_eo"],
                                     b["dg"])
        moe_expert_act_backward(b["d_eo"], offsets=offsets, want_dz=False, db=b["db2"], ws=b["b2_ws"])
        moe_expert_dgrad(b["d_eo"], offsets, self.w2, b["dh"], b["dgrad_ws"])
        moe_expert_act_backward(b["dh"], self.pre, offsets, self.act, self.gated, dz=b["dpre"], db=b["db1"],
                                ws=b["act_ws"])
        moe_expert_wgrad(b["d_eo"], self.h, offsets, dw=b["dw2"], rows=rows)   # (the h that w2 multiplied)
        moe_permute(x, send_pos, k, None, b["x_perm"])
        moe_expert_wgrad(b["dpre"], b["x_perm"], offsets, dw=b["dw1"], rows=rows)
        moe_expert_dgrad(b["dpre"], offsets, self.w1, b["d_perm"], b["dgrad_ws"])
        rest = None
        if self.w_r is not None:
            moe_router_backward(self.topk_gate, b["dg"], offsets, src_slot, x, b["dz"], b["dw_r"])
            rest = moe_router_input_grad(self.w_r, self.topk_idx, b["dz"], None, b["dx_r"])
        moe_combine(b["d_perm"], send_pos, None, rest, b["dx"], k=k)
        return b


class PipelinedMoE:
    """The layer over C chunks of tokens with one chunk's combine beside the next chunk's GEMMs.

    "EP / DeepEP explanation" page, section 7: cut the batch into chunks so that the dispatch
    and combine of one chunk overlap the expert computation of another (the pipelined time is
    about T_warm + sum over chunks of max(T_dispatch, T_experts, T_combine) + T_drain).  Here
    chunk c's router logits, route, layout and grouped GEMMs run on the caller's stream, and
    its combine on a second stream (default priority) once chunk c's down GEMM is done, while
    chunk c + 1's work starts on the first stream.  Each chunk is a MoELayer of N / C tokens
    over the same weights (bf16 layers); y is one [N, H] buffer, chunk c writing its rows.
    Routing is per token, so the result equals the unchunked layer's up to the tiles' row
    split (the same arithmetic per row).
    """

    def __init__(self, chunks: int, N: int, H: int, E: int, k: int, I: int, w13: torch.Tensor, w2: torch.Tensor,
                 shared_w13: Optional[torch.Tensor] = None, shared_w2: Optional[torch.Tensor] = None,
                 n_group: int = 0, topk_group: int = 0, bias: Optional[torch.Tensor] = None,
                 w_r: Optional[torch.Tensor] = None):
        if chunks < 1 or N % chunks:
            raise ValueError("N must split into equal chunks")
        self.N, self.H, self.chunks = N, H, chunks
        n = N // chunks
        dev = w13.device
        self.y = torch.empty((N, H), dtype=torch.bfloat16, device=dev)
        self.parts = []
        for c in range(chunks):
            lay = MoELayer(n, H, E, k, I, "bf16", w13, w2, shared_w13, shared_w2, n_group, topk_group, bias,
                           w_r=w_r)
            lay.y = self.y[c * n:(c + 1) * n]   # (a contiguous block of rows)
            self.parts.append(lay)
        self.side = torch.cuda.Stream(device=dev)
        self.ready = [torch.cuda.Event() for _ in range(chunks)]
        self.done = torch.cuda.Event()

    def forward(self, x: torch.Tensor, z: Optional[torch.Tensor] = None) -> torch.Tensor:
        main = torch.cuda.current_stream(x.device)
        n = self.N // self.chunks
        self.side.wait_stream(main)
        for c, lay in enumerate(self.parts):
            xc = x[c * n:(c + 1) * n]
            zc = None if z is None else z[c * n:(c + 1) * n]
            if zc is None:
                zc = lay.router(xc)
            lay.route(zc)
            lay.dispatch()
            lay.permute(xc)
            lay.experts(xc)
            self.ready[c].record(main)
            self.side.wait_event(self.ready[c])
            with torch.cuda.stream(self.side):
                lay.combine()
        self.done.record(self.side)
        main.wait_event(self.done)
        x.record_stream(self.side)
        return self.y
