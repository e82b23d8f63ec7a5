"""EpAdamW: the optimizer step behind the replica gradient reduction.

ep_replica_grad_reduce leaves an expert's whole gradient in its home row, in
fp32; this takes it from there: one launch for up to 256 tensors updates the
fp32 parameters, the moments (fp32, or 8 bits with a scale per block) and, where
asked, the bf16 weights that ep_expert_up and ep_expert_gemm read.  Like
EpLayer it works on static buffers: parameters, gradients and copies are given
once and stay where they are (EpLayer.g_home's rows, for instance).
"""
import torch

from . import EP_ADAMW_BLOCK, adamw_table, ep_adamw


class EpAdamW:
    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, state_bits=32,
                 copies=None, state=None):
        """params: fp32 tensors, updated in place; grads: their gradients, all
        fp32 or all bf16, read at every step; copies: bf16 tensors (or None
        each) that get the rounded parameters.  lr: a number, or an fp32 CUDA
        tensor of one element that a captured step reads again at every replay.
        state_bits 8: the second moment's root is rounded to nearest in the first
        steps and up to beta2 = 0.968, beyond by chance (the same for the same
        step), since steps so small would never move a code: see ep.h.
        state: a state_dict() to go on from (its tensors are used, not copied);
        otherwise the moments start at zero."""
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits {state_bits}, expected 8 or 32")
        params = list(params)
        if not params:
            raise ValueError("no parameters")
        self.params, self.grads = params, list(grads)
        self.copies = None if copies is None else list(copies)
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.state_bits = state_bits
        self.device = params[0].device
        where = [p.data_ptr() for p in params if p.numel()]
        if len(set(where)) != len(where):
            raise ValueError("a parameter stands twice in the list")
        if state is None:
            state = self._fresh()
        self.steps, self.m, self.v = state["step"], list(state["m"]), list(state["v"])
        self.m_scale, self.v_scale = state.get("m_scale"), state.get("v_scale")
        if self.steps.device != self.device:
            raise ValueError(f"tensors on {self.device} and {self.steps.device}")
        if (state_bits == 8) != (self.m_scale is not None):
            raise ValueError(f"state without the scales of {state_bits} bits")
        # the table holds the tensors' addresses, and this object the tensors
        self._table, bits, self._grad_dtype = adamw_table(self.params, self.grads, self.m, self.v, self.m_scale,
                                                          self.v_scale, self.copies)

    def _fresh(self):
        eight = self.state_bits == 8

        def moments():
            return [torch.zeros(p.shape, dtype=torch.float32, device=p.device) if not eight else
                    torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(torch.float8_e4m3fn)
                    for p in self.params]

        def scales():
            return [torch.zeros(-(-p.numel() // EP_ADAMW_BLOCK), dtype=torch.float32, device=p.device)
                    for p in self.params] if eight else None

        return dict(step=torch.zeros(1, dtype=torch.int32, device=self.device), m=moments(), v=moments(),
                    m_scale=scales(), v_scale=scales())

    def step(self, grad_scale=None, stream=None):
        """One step from the gradients as they are now; grad_scale: fp32 CUDA
        tensor of one element that multiplies them (a clipping factor).  A call
        that is refused does not count as a step."""
        self._count(1, stream)
        try:
            ep_adamw(self._table, len(self.params), self.state_bits, self._grad_dtype, self.steps, self.lr, self.betas,
                     self.eps, self.weight_decay, grad_scale, stream)
        except Exception:
            self._count(-1, stream)
            raise

    def _count(self, n, stream):
        if stream is None:
            self.steps.add_(n)
        else:
            with torch.cuda.stream(stream):
                self.steps.add_(n)

    def state_dict(self):
        """The state's own tensors (not copies)."""
        return dict(step=self.steps, m=self.m, v=self.v, m_scale=self.m_scale, v_scale=self.v_scale)
