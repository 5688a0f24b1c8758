"""Packed expert layers and the captured layer stack, on top of the C ABI.

Convenience objects that own torch device buffers and call libqmoe; every
step of the computation runs in the library's kernels.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib as L


class PackedLayer:
    """One layer's experts in the packed device layout (qmoe_pack)."""

    def __init__(self, fmt: int, E: int, H: int, I: int, device="cuda"):
        self.fmt, self.E, self.H, self.I = fmt, E, H, I
        self.gate_up = torch.empty(L.qmoe_packed_bytes(fmt, L.GATE_UP, E, H, I), dtype=torch.uint8, device=device)
        self.down = torch.empty(L.qmoe_packed_bytes(fmt, L.DOWN, E, H, I), dtype=torch.uint8, device=device)

    @property
    def nbytes(self) -> int:
        return self.gate_up.numel() + self.down.numel()

    def pack(self, canon: dict, stream=None) -> "PackedLayer":
        """Pack canonical tensors (gate/up/down _codes uint8 and _scales uint16)."""
        L.qmoe_pack(self.fmt, L.GATE_UP, self.E, self.H, self.I, canon["gate_codes"], canon["gate_scales"],
                    canon["up_codes"], canon["up_scales"], self.gate_up, stream)
        L.qmoe_pack(self.fmt, L.DOWN, self.E, self.H, self.I, canon["down_codes"], canon["down_scales"],
                    None, None, self.down, stream)
        return self

    def handle(self) -> L.qmoe_experts:
        return L.qmoe_experts(self.E, self.H, self.I, self.fmt, self.gate_up.data_ptr(), self.down.data_ptr(),
                              self.gate_up.numel(), self.down.numel())


class DecodeStack:
    """L layers of route -> FFN -> residual RMSNorm as one CUDA graph."""

    def __init__(self, layers, routers, biases, T: int, k: int, eps: float, stream=None, timing: bool = False,
                 layerwise: bool = False):
        self.layers, self.routers, self.biases = list(layers), list(routers), biases
        self.L, self.T, self.k = len(self.layers), T, k
        self.H = self.layers[0].H
        self._handles = (L.qmoe_experts * self.L)(*[l.handle() for l in self.layers])
        self._wr = (ctypes.c_void_p * self.L)(*[w.data_ptr() for w in self.routers])
        if biases is not None:
            self._bias = (ctypes.c_void_p * self.L)(*[None if b is None else b.data_ptr() for b in biases])
        else:
            self._bias = None
        self.desc = L.qmoe_stack_desc(self.L, T, k, eps, self._wr, self._bias, self._handles,
                                      (L.STACK_TIMING if timing else 0) | (L.STACK_LAYERWISE if layerwise else 0))
        nbytes = L.qmoe_stack_workspace_bytes(self.desc)
        if nbytes == 0:
            raise L.QmoeError("qmoe_stack_workspace_bytes", 1)
        dev = self.routers[0].device
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        self.handle = L.qmoe_stack_create(self.desc, self.workspace, stream)
        bufs = L.qmoe_stack_buffers(self.handle)
        base = self.workspace.data_ptr()

        def view(ptr, n, dtype):
            off = ptr - base
            esz = torch.tensor([], dtype=dtype).element_size()
            return self.workspace[off:off + n * esz].view(dtype)

        TH = T * self.H
        self.x_in = view(bufs["x_in"], TH, torch.float32).view(T, self.H)
        self.x_out = view(bufs["x_out"], TH, torch.float32).view(T, self.H)
        self.idx = view(bufs["idx"], self.L * T * k, torch.int32).view(self.L, T, k)
        self.gate = view(bufs["gate"], self.L * T * k, torch.float32).view(self.L, T, k)
        self.dev_status = view(bufs["dev_status"], 1, torch.int32)
        self.kernels_per_replay = L.qmoe_stack_kernels_per_replay(self.handle)
        self.path = L.qmoe_stack_path(self.handle)

    def decode(self, stream=None) -> None:
        L.qmoe_stack_decode(self.handle, stream)

    def decode_host(self, x_host, x_out_host, stream=None) -> None:
        L.qmoe_stack_decode_host(self.handle, x_host, x_out_host, stream)

    def layer_times(self):
        """(route_ms, ffn_ms) per layer of the last completed replay (timing stacks)."""
        return L.qmoe_stack_layer_times(self.handle, self.L)

    def phase_trace(self):
        """Per-layer phase stamps of the last replay (fused timing stacks):
        int64 SM cycles [L, CTAs, points]."""
        return L.qmoe_stack_trace(self.handle, self.L)

    def status(self) -> int:
        return L.qmoe_read_status(self.dev_status)

    def close(self) -> None:
        if getattr(self, "handle", None):
            L.qmoe_stack_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class TokenHead:
    """What follows a layer stack: final RMSNorm -> vocabulary product -> sampled tokens, three kernels.

    ``weight`` bf16 or fp32 [V, H]. With ``bits`` 8, the default, its rows are kept as int8 codes and fp32 scales
    (qmoe_quantise_rows) and the normed rows are rounded to 8 bits too, which halves the bytes of a step but is
    coarser than weights given in 16 bits or more; with ``bits`` 16 both are bf16. ``gain`` fp32 [H]
    or None; ``bias`` fp32 [V] or None. All buffers are made here, on ``stream`` where one is given; ``step`` only
    launches, and can be captured. Two steps that overlap on different streams need a head each.
    """

    def __init__(self, weight, T: int, gain=None, bias=None, eps: float = 1e-6, bits: int = 8, stream=None):
        if weight.dim() != 2 or weight.dtype not in (torch.bfloat16, torch.float32):
            raise L.QmoeError("TokenHead (weight must be a bf16 or fp32 matrix)", 1)
        if bits not in (8, 16):
            raise L.QmoeError("TokenHead (bits must be 8 or 16)", 1)
        if T < 1:
            raise L.QmoeError("TokenHead (no tokens)", 1)
        self.V, self.H = weight.shape
        self.T, self.eps, self.bits, self.gain, self.bias = T, eps, bits, gain, bias
        if stream is None:
            self._lay_out(weight)
            return
        # every buffer made and filled on the given stream, behind what has been queued on the current one (the
        # weights, for instance), which in turn goes on behind it: the weights may be dropped after this
        own = torch.cuda.ExternalStream(stream, device=weight.device) if isinstance(stream, int) else stream
        here = torch.cuda.current_stream(weight.device)
        own.wait_stream(here)
        with torch.cuda.stream(own):
            self._lay_out(weight)
        here.wait_stream(own)

    def _lay_out(self, weight) -> None:
        T, dev = self.T, weight.device
        if self.bits == 8:
            self.weight = torch.empty((self.V, self.H), dtype=torch.int8, device=dev)
            self.weight_scale = torch.empty(self.V, dtype=torch.float32, device=dev)
            L.qmoe_quantise_rows(weight, L.BF16 if weight.dtype == torch.bfloat16 else L.F32, self.V, self.H, 0,
                                 self.weight, self.weight_scale)
            self.codes = torch.empty((T, self.H), dtype=torch.int8, device=dev)
            self.scale = torch.empty(T, dtype=torch.float32, device=dev)
            self.norm = None
        else:
            self.weight, self.weight_scale = weight.to(torch.bfloat16).contiguous(), None
            self.norm = torch.empty((T, self.H), dtype=torch.bfloat16, device=dev)
            self.codes = self.scale = None
        # rows of logits start on 16 bytes whatever V is
        self._ld = (self.V + 3) // 4 * 4
        self._logits = torch.empty((T, self._ld), dtype=torch.float32, device=dev)
        self.logits = self._logits[:, :self.V]
        self.token = torch.empty(T, dtype=torch.int32, device=dev)
        self.prob = torch.empty(T, dtype=torch.float32, device=dev)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=dev)

    def step(self, x, u, temperature=None, top_k=None, top_p=None, min_p=None, y=None, stream=None) -> torch.Tensor:
        """``x`` (and ``y``, added to it) fp32 or bf16 [T, H], for instance ``DecodeStack.x_out``; ``u`` fp32 [T] in
        [0, 1), one per row; the rest as in qmoe_sample. Rows lie one behind the other: the last positions of
        [T, S, H] hidden states go in as ``hidden[:, -1].contiguous()``, and as a view they are refused. Returns
        the device tensor ``token`` int32 [T]."""
        if x.dtype not in (torch.bfloat16, torch.float32):
            raise L.QmoeError("TokenHead.step (x must be bf16 or fp32)", 1)
        if x.numel() != self.T * self.H:
            raise L.QmoeError("TokenHead.step (x is not [T, H])", 1)
        L.qmoe_rmsnorm_residual_q8(x, y, L.BF16 if x.dtype == torch.bfloat16 else L.F32, self.gain, self.eps, self.T,
                                   self.H, 0, None, self.norm, self.codes, self.scale, stream)
        a = self.codes if self.bits == 8 else self.norm
        L.qmoe_linear(a, L.I8 if self.bits == 8 else L.BF16, self.weight, self.T, self.V, self.H, self.scale,
                      self.weight_scale, self.bias, L.ACT_NONE, None, self._logits, L.F32, self.dev_status,
                      ldo=self._ld, stream=stream)
        L.qmoe_sample(self._logits, L.F32, self.T, self.V, temperature, top_k, top_p, min_p, u, self.token, self.prob,
                      self.dev_status, ld=self._ld, stream=stream)
        return self.token

    def status(self) -> int:
        """The first error of all steps so far, 0 if there was none (waits for the device). A row out of range stays
        reported until ``dev_status.zero_()``."""
        return L.qmoe_read_status(self.dev_status)
