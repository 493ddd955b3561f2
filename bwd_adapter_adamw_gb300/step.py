"""Host orchestration of one optimizer step through the C ABI.

This module allocates device buffers with torch (flat fp32 arenas for parameters, gradients and
Adam moments; per-stream workspaces) and sequences the library calls: per adapted linear a
forward and a backward over all accumulation chunks, then one grad-prepare and one AdamW launch
over the arena. It computes nothing itself: every number of the step comes from the library's
kernels.

Arena layout (one per adapter set): [A of every linear | B of every linear | DoRA magnitudes],
so a single lora_group describes the global clip ("4.3. Training Guide", Gradient clipping:
clipped globally by L2 norm) and the AdamW kinds. Multi-LoRA uses one group per slot
("Multi-LoRA Training Example (fully-async)", Design: per-slot state, step counts and clipping).
"""
from __future__ import annotations

from dataclasses import dataclass, field
from typing import Dict, List, Optional, Sequence, Tuple

import torch

from . import binding as L

_DT = {"f32": L.LORA_F32, "bf16": L.LORA_BF16, "bf16fp8": L.LORA_BF16_FP8,
       "bf16blk8": L.LORA_BF16_BLK8}


def _ws(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _streams_in_use(step):
    """(k, streams): the first k = min(active_streams, n_streams) side streams, or none for k = 1
    (everything on the caller's current stream)."""
    k = max(1, min(step.active_streams, step.n_streams))
    return k, (step.streams[:k] if (step.streams and k > 1) else [])


def _fork(main, use):
    if use:
        ev = torch.cuda.Event()
        ev.record(main)
        for s in use:
            s.wait_event(ev)


def _join(main, use):
    for s in use:
        ev = torch.cuda.Event()
        ev.record(s)
        main.wait_event(ev)


@dataclass
class Linear:
    """One adapted linear with its activations (device tensors)."""
    layer: int
    proj_id: int
    X: torch.Tensor          # [T, in]
    W: torch.Tensor          # [out, in]
    dY: torch.Tensor         # [T, out]
    Wp: Optional[torch.Tensor] = None   # prepared copy of W (bytes), filled by prepare_weights
    Y: Optional[torch.Tensor] = None
    dX: Optional[torch.Tensor] = None
    H: Optional[torch.Tensor] = None
    # views into the arenas
    A: Optional[torch.Tensor] = None
    B: Optional[torch.Tensor] = None
    gA: Optional[torch.Tensor] = None
    gB: Optional[torch.Tensor] = None
    mag: Optional[torch.Tensor] = None
    gmag: Optional[torch.Tensor] = None
    norm: Optional[torch.Tensor] = None

    @property
    def in_dim(self) -> int:
        return self.W.shape[1]

    @property
    def out_dim(self) -> int:
        return self.W.shape[0]


class Arena:
    """Flat fp32 parameter / gradient / moment arenas with named views."""

    def __init__(self, n: int, device):
        self.n = n
        self.params = torch.zeros(n, dtype=torch.float32, device=device)
        self.grads = torch.zeros(n, dtype=torch.float32, device=device)
        self.m = torch.zeros(n, dtype=torch.float32, device=device)
        self.v = torch.zeros(n, dtype=torch.float32, device=device)

    def view(self, which: str, offset: int, shape) -> torch.Tensor:
        numel = 1
        for s in shape:
            numel *= s
        return getattr(self, which)[offset:offset + numel].view(*shape)


class LoraStep:
    """One optimizer step over a set of independent adapted linears sharing rank/scale/dtype."""

    def __init__(self, linears: Sequence[Linear], *, rank: int, scale: float, dtype: str,
                 tokens: int, chunks: int, dropout_p: float = 0.0, seed: int = 0,
                 dora: bool = False, max_norm: float = 1.0, hp: Optional[L.lora_adamw_hp] = None,
                 n_streams: int = 1, device="cuda", n_extra: int = 0):
        self.linears = list(linears)
        self.rank, self.scale, self.dtype = rank, scale, _DT[dtype]
        self.T, self.chunks = tokens, chunks
        self.dropout_p, self.seed, self.dora = dropout_p, seed, dora
        self.max_norm = max_norm
        self.hp = hp if hp is not None else L.make_hp()
        self.device = torch.device(device)
        # arena: [A ... | B ... | MAG ...], n_extra further parameters at the magnitudes' end
        na = sum(rank * l.in_dim for l in self.linears)
        nb = sum(l.out_dim * rank for l in self.linears)
        nm = (sum(l.out_dim for l in self.linears) if dora else 0) + n_extra
        self.n_a, self.n_b, self.n_mag = na, nb, nm
        self.arena = Arena(na + nb + nm, self.device)
        oa, ob, om = 0, na, na + nb
        for l in self.linears:
            l.A = self.arena.view("params", oa, (rank, l.in_dim))
            l.gA = self.arena.view("grads", oa, (rank, l.in_dim))
            oa += rank * l.in_dim
            l.B = self.arena.view("params", ob, (l.out_dim, rank))
            l.gB = self.arena.view("grads", ob, (l.out_dim, rank))
            ob += l.out_dim * rank
            if dora:
                l.mag = self.arena.view("params", om, (l.out_dim,))
                l.gmag = self.arena.view("grads", om, (l.out_dim,))
                om += l.out_dim
                l.norm = torch.empty(l.out_dim, dtype=torch.float32, device=self.device)
            act = l.X.dtype
            if l.Y is None:
                l.Y = torch.empty((self.T, l.out_dim), dtype=act, device=self.device)
            if l.dX is None:
                l.dX = torch.empty((self.T, l.in_dim), dtype=act, device=self.device)
            if l.H is None:
                l.H = torch.empty((self.T, rank), dtype=torch.float32, device=self.device)
        self.n_streams = max(1, n_streams)
        self.streams = [torch.cuda.Stream(device=self.device) for _ in range(self.n_streams)] \
            if self.n_streams > 1 else []
        self.active_streams = self.n_streams   # streams used by the next enqueue (<= n_streams)
        ws_need = max(L.lora_workspace_size(self.desc(l), self.T) for l in self.linears)
        if self.dora:   # the norm refresh shares the stream's workspace
            ws_need = max(ws_need, max(L.lora_dora_norm_workspace_size(self.desc(l))
                                       for l in self.linears))
        if ws_need == 0:
            raise L.LoraError(L.LORA_ERR_INVALID, "lora_workspace_size")
        self.ws = [_ws(ws_need, self.device) for _ in range(self.n_streams)]
        self.scale_norm = torch.zeros(2, dtype=torch.float64, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._groups_cache = None

    # ------------------------------------------------------------------------------------------
    def desc(self, l: Linear) -> L.lora_desc:
        return L.make_desc(l.in_dim, l.out_dim, self.rank, self.scale, self.dtype, self.dropout_p,
                           self.seed, l.layer, l.proj_id, self.dora)

    def prepare_weights(self, stream=None):
        for l in self.linears:
            if l.Wp is None:
                l.Wp = torch.empty(L.lora_prepared_weight_size(self.desc(l)), dtype=torch.uint8,
                                   device=self.device)
            L.lora_prepare_weight(self.desc(l), l.W, l.Wp, stream)

    def groups(self, lr: float, step: int):
        return L.make_groups([dict(offset=0, n_a=self.n_a, n_b=self.n_b, n_mag=self.n_mag,
                                   grad_scale=1.0 / self.T, max_norm=self.max_norm, lr=lr,
                                   step=step)])

    def prepare_ws(self) -> torch.Tensor:
        g = self.groups(0.0, 0)
        if not hasattr(self, "_prep_ws"):
            self._prep_ws = _ws(L.lora_grad_prepare_workspace_size(g), self.device)
        return self._prep_ws

    # ------------------------------------------------------------------------------------------
    def _enqueue(self, opt_step: int, per_chunk_calls: bool, backward: bool, forward: bool = True,
                 linears: Optional[Sequence[Linear]] = None):
        main = torch.cuda.current_stream(self.device)
        k, use = _streams_in_use(self)
        _fork(main, use)
        ct = self.T // self.chunks
        for i, l in enumerate(self.linears if linears is None else linears):
            st = use[i % k] if use else main
            ws = self.ws[i % k]
            d = self.desc(l)
            if self.dora:
                L.lora_dora_norm(d, l.W, l.A, l.B, l.norm, ws, stream=st)
            if per_chunk_calls:
                spans = [(c, c * ct, ct) for c in range(self.chunks)]
            else:
                spans = [(0, 0, self.T)]
            for (ordinal, t0, n) in spans:
                ctx = L.make_ctx(opt_step, ordinal, ct)
                sl = slice(t0, t0 + n)
                X, dY, Y, dX, H = l.X[sl], l.dY[sl], l.Y[sl], l.dX[sl], l.H[sl]
                if forward:
                    L.lora_forward(d, ctx, n, X, l.W, l.Wp, l.A, l.B, l.mag, l.norm, Y, H, ws, stream=st)
                if backward:
                    L.lora_backward(d, ctx, n, X, l.Wp, l.A, l.B, dY, H, l.mag, l.norm, Y, dX, l.gA,
                                    l.gB, l.gmag, ws, stream=st)
        _join(main, use)

    def forward_backward(self, opt_step: int, per_chunk_calls: bool = False):
        """Enqueue forward + backward of every linear over all chunks (gradients accumulate)."""
        self._enqueue(opt_step, per_chunk_calls, True)

    def optimizer_step(self, lr: float, step: int, zero_grads: bool = True):
        g = self.groups(lr, step)
        ws = self.prepare_ws()
        L.lora_grad_prepare(self.arena.grads, g, self.scale_norm, self.status, ws)
        L.lora_adamw_step(self.arena.params, self.arena.grads, self.arena.m, self.arena.v, g,
                          self.hp, self.scale_norm, self.status, zero_grads)

    def run(self, opt_step: int, lr: float, per_chunk_calls: bool = False, zero_grads: bool = True):
        self.forward_backward(opt_step, per_chunk_calls)
        self.optimizer_step(lr, opt_step, zero_grads)

    def snapshot(self, snap: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Device copy of every adapter's parameters (the best-weights snapshot)."""
        if snap is None:
            snap = torch.empty_like(self.arena.params)
        L.lora_snapshot(self.arena.params, snap, self.groups(0.0, 0))
        return snap

    def restore(self, snap: torch.Tensor, zero_grads: bool = True):
        """Restore a snapshot and reset the optimizer (moments zeroed); the caller's next update
        passes step 0 again."""
        L.lora_restore(self.arena.params, snap, self.arena.grads, self.arena.m, self.arena.v,
                       self.groups(0.0, 0), zero_grads)


class SublayerStep(LoraStep):
    """One optimizer step of a pre-norm sublayer: a layer norm (or RMS norm) in front of adapted
    projections that read its output,
        H = norm(X),  Y_k = projection_k(H),  dX = dX_res + norm'(sum_k dX_k),
    with the norm's weight (and shift) trained beside the adapters. They live in the arena's
    magnitude range, so one group holds the global clip of everything; A and B take the
    orthogonalised update (with `hp`'s decay and LoRA+ ratio unless `muon` is given), the norm's
    parameters AdamW (no decay, plain learning rate)."""

    def __init__(self, X: torch.Tensor, linears: Sequence[Linear], *, kind: str = "layer",
                 eps: float = 1e-5, muon: Optional[L.lora_muon_hp] = None, inner: Sequence[Linear] = (),
                 n_inner: int = 0, **kw):
        """`inner`: further projections of the sublayer, which read something else; n_inner: further
        parameters at the magnitudes' end."""
        if kind not in ("layer", "rms"):
            raise ValueError(f"kind {kind!r}: 'layer' or 'rms'")
        if not 1 <= len(linears) <= L.LORA_SUM_MAX:
            raise ValueError(f"{len(linears)} projections: 1 to {L.LORA_SUM_MAX}")
        if kw.get("dora"):
            raise ValueError("the sublayer's magnitude range holds the norm's parameters")
        if X.dim() != 2 or not X.is_contiguous() or X.shape[0] != kw.get("tokens"):
            raise ValueError(f"X {tuple(X.shape)}: a contiguous [tokens, dim], tokens {kw.get('tokens')}")
        if X.dtype != (torch.float32 if kw.get("dtype") == "f32" else torch.bfloat16):
            raise ValueError(f"X is {X.dtype} in a step of dtype {kw.get('dtype')}")
        for l in linears:
            if l.in_dim != X.shape[1] or tuple(l.dY.shape) != (X.shape[0], l.out_dim) or l.dY.dtype != X.dtype:
                raise ValueError(f"projection {l.proj_id}: W {tuple(l.W.shape)} and dY {tuple(l.dY.shape)} "
                                 f"{l.dY.dtype} do not fit X {tuple(X.shape)} {X.dtype}")
        self.readers = list(linears)                   # the projections that read the norm's output
        self.X_in = X                                  # [T, dim], the sublayer's input
        self.H_norm = torch.empty_like(X)
        for l in linears:
            l.X = self.H_norm
        self.norm = L.make_norm_desc(X.shape[1], L.LORA_NORM_RMS if kind == "rms" else L.LORA_NORM_LAYER,
                                     L.LORA_F32 if X.dtype == torch.float32 else L.LORA_BF16, eps)
        dim, shift = X.shape[1], kind != "rms"
        super().__init__(self.readers + list(inner), n_extra=dim * (2 if shift else 1) + n_inner, **kw)
        base = self.n_a + self.n_b
        self.gamma, self.dgamma = (self.arena.view(w, base, (dim,)) for w in ("params", "grads"))
        self.beta = self.dbeta = None
        if shift:
            self.beta, self.dbeta = (self.arena.view(w, base + dim, (dim,)) for w in ("params", "grads"))
        self.gamma.fill_(1.0)
        self.stats = torch.empty((self.T, 2), dtype=torch.float32, device=self.device)
        self.dX = torch.empty_like(X)
        self.dH_norm = torch.empty_like(X) if len(self.readers) > 1 else None   # the norm output's gradient
        self.norm_ws = _ws(L.lora_norm_backward_workspace_size(self.norm, self.T), self.device)
        self.muon = muon if muon is not None else L.make_muon_hp(weight_decay=self.hp.weight_decay,
                                                                 plus_ratio=self.hp.plus_ratio)
        mats, oa, ob = [], 0, self.n_a
        for l in self.linears:
            mats.append(dict(offset=oa, rows=self.rank, cols=l.in_dim, kind=L.LORA_KIND_A))
            oa += self.rank * l.in_dim
        for l in self.linears:
            mats.append(dict(offset=ob, rows=l.out_dim, cols=self.rank, kind=L.LORA_KIND_B))
            ob += l.out_dim * self.rank
        self.mats = L.make_mats(mats)
        self.muon_ws = _ws(L.lora_muon_workspace_size(self.mats), self.device)

    def forward(self, opt_step: int = 0):
        """The norm and every projection (the serving call)."""
        self._norm_forward()
        self._enqueue(opt_step, False, False)

    def _norm_forward(self):
        L.lora_norm_forward(self.norm, self.T, self.X_in, self.gamma, self.beta, self.H_norm, self.stats)

    def forward_backward(self, opt_step: int, dX_res: Optional[torch.Tensor] = None,
                         per_chunk_calls: bool = False):
        """Forward, every projection's backward, and the norm's backward on the sum of their input
        gradients (added in fp32: rounded once, and dX once more with the residual's gradient)."""
        self._check_residual(dX_res)
        self._norm_forward()
        self._enqueue(opt_step, per_chunk_calls, True)
        self._norm_backward(dX_res)

    def _check_residual(self, dX_res: Optional[torch.Tensor]):
        if dX_res is not None and not (torch.is_tensor(dX_res) and dX_res.shape == self.X_in.shape and
                                       dX_res.dtype == self.X_in.dtype and dX_res.is_contiguous()):
            raise ValueError("dX_res: a contiguous tensor of X's shape and type")

    def _norm_backward(self, dX_res: Optional[torch.Tensor]):
        dH = self.readers[0].dX
        if len(self.readers) > 1:
            dH = self.dH_norm
            L.lora_sum([l.dX for l in self.readers], dH.numel(), self.norm.dtype, dH)
        L.lora_norm_backward(self.norm, self.T, self.X_in, self.gamma, dH, self.stats, dX_res, self.dX,
                             self.dgamma, self.dbeta, self.norm_ws)

    def optimizer_step(self, lr: float, step: int, zero_grads: bool = True):
        g = self.groups(lr, step)
        L.lora_grad_prepare(self.arena.grads, g, self.scale_norm, self.status, self.prepare_ws())
        a = self.arena
        L.lora_muon_step(a.params, a.grads, a.m, g, self.mats, self.muon, self.scale_norm, self.status,
                         zero_grads, self.muon_ws)
        norm = L.make_groups([dict(offset=self.n_a + self.n_b, n_mag=self.n_mag,
                                   grad_scale=1.0 / self.T, max_norm=self.max_norm, lr=lr, step=step)])
        L.lora_adamw_step(a.params, a.grads, a.m, a.v, norm, self.hp, self.scale_norm, self.status,
                          zero_grads)

    def run(self, opt_step: int, lr: float, dX_res: Optional[torch.Tensor] = None,
            zero_grads: bool = True, per_chunk_calls: bool = False):
        self.forward_backward(opt_step, dX_res, per_chunk_calls)
        self.optimizer_step(lr, opt_step, zero_grads)


class AttentionStep(SublayerStep):
    """One optimizer step of an attention sublayer: a norm, adapted query, key and value projections,
    the norm of each query and key head with the rotation by position, causal attention over packed
    sequences, and the adapted output projection,
        Q, K, V = projections(norm(X)),  Y = projection_o(attention(rope(Q), rope(K), V)),
    with the norms' weights trained beside the adapters (as in SublayerStep; without the heads' norms
    with head_norm=False). q, k, v and o are the Linears of the four projections; o.dY is the
    sublayer's output gradient, the other three gradients and the four inputs are the step's own. seq_start: int32 [n + 1]
    on the device, the sequences' first tokens and the last one's end; tokens of no sequence are padding
    (their rows of X have to be finite, their output gradients zero). pos: int32 [tokens], from 0 in each
    sequence unless given (padding's are not read; a negative one in a sequence leaves that token's turned query
    and key zero, which take no gradient). Both are copied; set_sequences gives the step another batch's.
    inv_freq: the rotation's frequencies, rope_base^(-2 i / head_dim) unless given, for n_pos positions
    (the batch's tokens unless given; a position from n_pos on, as in a longer sequence, makes its sequence
    and the gradients NaN)."""

    def __init__(self, X: torch.Tensor, q: Linear, k: Linear, v: Linear, o: Linear, *, q_heads: int,
                 kv_heads: int, head_dim: int, seq_start: torch.Tensor, pos: Optional[torch.Tensor] = None,
                 n_pos: Optional[int] = None, rope_base: float = 10000.0,
                 inv_freq: Optional[torch.Tensor] = None, pairs: bool = False, head_norm: bool = True,
                 head_eps: float = 1e-6, **kw):
        if X.dtype != torch.bfloat16:
            raise ValueError("the attention step takes bf16 activations")
        T, dev, wq, wk = X.shape[0], X.device, q_heads * head_dim, kv_heads * head_dim
        for name, l, width in (("q", q, wq), ("k", k, wk), ("v", v, wk)):
            if l.out_dim != width:
                raise ValueError(f"projection {name}: {l.out_dim} outputs for {width // max(head_dim, 1)} heads of {head_dim}")
        if o.in_dim != wq or tuple(o.dY.shape) != (T, o.out_dim) or o.dY.dtype != X.dtype:
            raise ValueError(f"projection o: W {tuple(o.W.shape)} and dY {tuple(o.dY.shape)} {o.dY.dtype}")
        self._check_sequences(seq_start, pos, T, dev)
        n_pos = T if n_pos is None else n_pos
        if inv_freq is not None and tuple(inv_freq.shape) != (head_dim // 2,):
            raise ValueError("inv_freq: [head_dim / 2]")
        attn = L.make_attn_desc(q_heads, kv_heads, head_dim)
        rope = L.make_rope_desc(q_heads, kv_heads, head_dim, L.LORA_BF16,
                                L.LORA_ROPE_PAIRS if pairs else L.LORA_ROPE_HALVES, head_eps)
        sizes = [L.lora_attn_backward_workspace_size(attn, T), L.lora_rope_backward_workspace_size(rope, T)]
        if 0 in sizes or not 1 <= n_pos <= 1 << 24:
            raise ValueError(f"{q_heads} / {kv_heads} heads of {head_dim}, eps {head_eps}, {n_pos} positions: query heads a "
                             "multiple of the key heads, head_dim 64 or 128, 1 to 2^24 positions")
        new = lambda n: torch.zeros((T, n), dtype=X.dtype, device=dev)   # noqa: E731  (padding rows stay zero)
        for l in (q, k, v):
            l.dY = new(l.out_dim)
        self.q, self.k, self.v, self.o = q, k, v, o
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        o.X = new(wq)                                      # the attention's output
        super().__init__(X, [q, k, v], inner=[o], n_inner=2 * head_dim if head_norm else 0, **kw)
        self.gamma_q = self.gamma_k = self.dgamma_q = self.dgamma_k = None
        if head_norm:
            at = self.n_a + self.n_b + self.n_mag - 2 * head_dim
            self.gamma_q, self.dgamma_q = (self.arena.view(w, at, (head_dim,)) for w in ("params", "grads"))
            self.gamma_k, self.dgamma_k = (self.arena.view(w, at + head_dim, (head_dim,)) for w in ("params", "grads"))
            self.gamma_q.fill_(1.0)
            self.gamma_k.fill_(1.0)
        self.n_seq, self.n_pos = seq_start.numel() - 1, n_pos
        if inv_freq is None:
            inv_freq = rope_base ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)
        self.table = torch.empty((self.n_pos, head_dim // 2, 2), dtype=torch.float32, device=dev)
        L.lora_rope_table(self.n_pos, head_dim, inv_freq.to(device=dev, dtype=torch.float64).contiguous(), self.table)
        self.rope, self.attn = rope, attn
        self.plan = _ws(L.lora_attn_plan_size(T, self.n_seq), dev)
        self.Qr, self.Kr, self.dQr, self.dKr = new(wq), new(wk), new(wq), new(wk)   # turned
        self.lse = torch.zeros((q_heads, T), dtype=torch.float32, device=dev)
        self.attn_ws = _ws(max(sizes), dev)
        self.seq_start = torch.empty_like(seq_start)
        self.pos = torch.empty(T, dtype=torch.int32, device=dev)
        self.set_sequences(seq_start, pos)

    @staticmethod
    def _check_sequences(seq_start: torch.Tensor, pos: Optional[torch.Tensor], T: int, dev: torch.device):
        if seq_start.dtype != torch.int32 or seq_start.dim() != 1 or seq_start.numel() < 2 or \
                seq_start.device != dev or not seq_start.is_contiguous():
            raise ValueError("seq_start: int32 [sequences + 1] on the activations' device")
        if pos is not None and (pos.dtype != torch.int32 or tuple(pos.shape) != (T,) or pos.device != dev):
            raise ValueError("pos: int32 [tokens] on the activations' device")

    @staticmethod
    def _positions(seq_start: torch.Tensor, T: int) -> torch.Tensor:
        """Each token's place in its sequence, -1 in none, of the sequences that the attention's plan makes of a table:
        clamped to the tokens, and each begins no earlier than those before it end."""
        s, at = seq_start.long().clamp(0, T), torch.arange(T, device=seq_start.device)
        end = s[1:].cummax(0).values
        seq = torch.searchsorted(end, at, right=True)      # sequences that end at or before the token
        pos = at - torch.cat((s[:1], end))[seq]
        return torch.where((seq < end.numel()) & (pos >= 0), pos, -1)

    def set_sequences(self, seq_start: torch.Tensor, pos: Optional[torch.Tensor] = None):
        """The sequences (as many as before, empty ones among them) and positions of the steps from here on, on
        the current stream; captured steps take them, too. Rows that were in a sequence and are padding now are
        cleared."""
        T = self.T
        dev = self.X_in.device
        self._check_sequences(seq_start, pos, T, dev)
        if seq_start.numel() != self.n_seq + 1:
            raise ValueError(f"{seq_start.numel() - 1} sequences for a step of {self.n_seq}")
        place = self._positions(seq_start, T)
        pos = place if pos is None else torch.where(place >= 0, pos, -1)   # (whatever is given for padding)
        self.seq_start.copy_(seq_start)
        self.pos.copy_(pos)
        for t in (self.o.X, self.lse, self.Qr, self.Kr, self.dQr, self.dKr, self.q.dY, self.k.dY, self.v.dY):
            t.zero_()
        L.lora_attn_plan_build(T, self.n_seq, self.seq_start, self.plan)

    def _forward(self, opt_step: int, per_chunk_calls: bool):
        """Everything up to the output projection."""
        self._norm_forward()
        self._enqueue(opt_step, per_chunk_calls, False, linears=self.readers)
        T = self.T
        L.lora_rope_forward(self.rope, T, self.q.Y, self.k.Y, self.gamma_q, self.gamma_k, self.pos, self.table,
                            self.n_pos, self.Qr, self.Kr)
        L.lora_attn_forward(self.attn, T, self.n_seq, self.plan, self.Qr, self.Kr, self.v.Y, self.o.X, self.lse)

    def forward(self, opt_step: int = 0):
        self._forward(opt_step, False)
        self._enqueue(opt_step, False, False, linears=[self.o])

    def forward_backward(self, opt_step: int, dX_res: Optional[torch.Tensor] = None,
                         per_chunk_calls: bool = False):
        """Forward and backward of the whole sublayer; gradients accumulate into the arena."""
        self._check_residual(dX_res)
        self._forward(opt_step, per_chunk_calls)
        self._enqueue(opt_step, per_chunk_calls, True, linears=[self.o])
        T = self.T
        L.lora_attn_backward(self.attn, T, self.n_seq, self.plan, self.Qr, self.Kr, self.v.Y, self.o.X, self.lse,
                             self.o.dX, self.dQr, self.dKr, self.v.dY, self.attn_ws)
        L.lora_rope_backward(self.rope, T, self.q.Y, self.k.Y, self.gamma_q, self.gamma_k, self.pos, self.table,
                             self.n_pos, self.dQr, self.dKr, self.q.dY, self.k.dY, self.dgamma_q, self.dgamma_k,
                             self.attn_ws)
        self._enqueue(opt_step, per_chunk_calls, True, forward=False, linears=self.readers)
        self._norm_backward(dX_res)


@dataclass
class FusedGroup:
    """Projections that read one input, run as one fused linear: the stacked frozen weight
    W [sum out_k, in] and output gradient dY [T, sum out_k], projection k in columns
    [off_k, off_k + out_k)."""
    layer: int
    proj_id: int                 # dropout key of the group (one mask for its projections)
    X: torch.Tensor              # [T, in]
    W: torch.Tensor              # [sum out_k, in]
    dY: torch.Tensor             # [T, sum out_k]
    outs: Tuple[int, ...]        # out_k
    Wp: Optional[torch.Tensor] = None
    Y: Optional[torch.Tensor] = None
    dX: Optional[torch.Tensor] = None
    H: Optional[torch.Tensor] = None            # [T, n rank]
    A: Optional[List[torch.Tensor]] = None      # arena views per projection
    B: Optional[List[torch.Tensor]] = None
    gA: Optional[List[torch.Tensor]] = None
    gB: Optional[List[torch.Tensor]] = None

    @property
    def in_dim(self) -> int:
        return self.W.shape[1]

    @property
    def out_dim(self) -> int:
        return self.W.shape[0]


class FusedLoraStep:
    """One optimizer step over groups of fused projections ("LoRA Training and Serving",
    --lora-type: fused projections, one adapter per projection): each group is one fused
    forward and one fused backward call (one frozen product over the stacked weight each, and
    one input gradient summed over the group's projections); the arena, the global clip and
    AdamW are LoraStep's."""

    def __init__(self, groups: Sequence[FusedGroup], *, rank: int, scale: float, dtype: str,
                 tokens: int, chunks: int, dropout_p: float = 0.0, seed: int = 0,
                 max_norm: float = 1.0, hp: Optional[L.lora_adamw_hp] = None,
                 n_streams: int = 1, device="cuda"):
        self.fgroups = list(groups)
        self.rank, self.scale, self.dtype = rank, scale, _DT[dtype]
        self.T, self.chunks = tokens, chunks
        self.dropout_p, self.seed, self.dora = dropout_p, seed, False
        self.max_norm = max_norm
        self.hp = hp if hp is not None else L.make_hp()
        self.device = torch.device(device)
        na = sum(rank * g.in_dim * len(g.outs) for g in self.fgroups)
        nb = sum(g.out_dim * rank for g in self.fgroups)
        self.n_a, self.n_b, self.n_mag = na, nb, 0
        self.arena = Arena(na + nb, self.device)
        oa, ob = 0, na
        for g in self.fgroups:
            if sum(g.outs) != g.out_dim:
                raise ValueError("the projections' widths must add up to the stacked weight's rows")
            g.A, g.gA, g.B, g.gB = [], [], [], []
            for o in g.outs:
                g.A.append(self.arena.view("params", oa, (rank, g.in_dim)))
                g.gA.append(self.arena.view("grads", oa, (rank, g.in_dim)))
                oa += rank * g.in_dim
                g.B.append(self.arena.view("params", ob, (o, rank)))
                g.gB.append(self.arena.view("grads", ob, (o, rank)))
                ob += o * rank
            act = g.X.dtype
            if g.Y is None:
                g.Y = torch.empty((self.T, g.out_dim), dtype=act, device=self.device)
            if g.dX is None:
                g.dX = torch.empty((self.T, g.in_dim), dtype=act, device=self.device)
            if g.H is None:
                g.H = torch.empty((self.T, rank * len(g.outs)), dtype=torch.float32,
                                  device=self.device)
        self.n_streams = max(1, n_streams)
        self.streams = [torch.cuda.Stream(device=self.device) for _ in range(self.n_streams)] \
            if self.n_streams > 1 else []
        self.active_streams = self.n_streams
        need = max(L.lora_fused_workspace_size(self.desc(g), self.T, self.projs(g))
                   for g in self.fgroups)
        if need == 0:
            raise L.LoraError(L.LORA_ERR_INVALID, "lora_fused_workspace_size")
        self.ws = [_ws(need, self.device) for _ in range(self.n_streams)]
        self.scale_norm = torch.zeros(2, dtype=torch.float64, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)

    def desc(self, g: FusedGroup) -> L.lora_desc:
        return L.make_desc(g.in_dim, g.out_dim, self.rank, self.scale, self.dtype, self.dropout_p,
                           self.seed, g.layer, g.proj_id, False)

    def projs(self, g: FusedGroup):
        return L.make_projs([dict(A=a, B=b, dA=ga, dB=gb, out=o)
                             for a, b, ga, gb, o in zip(g.A, g.B, g.gA, g.gB, g.outs)])

    def prepare_weights(self, stream=None):
        for g in self.fgroups:
            if g.Wp is None:
                g.Wp = torch.empty(L.lora_prepared_weight_size(self.desc(g)), dtype=torch.uint8,
                                   device=self.device)
            L.lora_prepare_weight(self.desc(g), g.W, g.Wp, stream)

    def forward_backward(self, opt_step: int, per_chunk_calls: bool = False):
        main = torch.cuda.current_stream(self.device)
        k, use = _streams_in_use(self)
        _fork(main, use)
        ct = self.T // self.chunks
        for i, g in enumerate(self.fgroups):
            st = use[i % k] if use else main
            ws = self.ws[i % k]
            d, pj = self.desc(g), self.projs(g)
            ctx = L.make_ctx(opt_step, 0, ct)
            L.lora_fused_forward(d, ctx, self.T, g.X, g.W, g.Wp, pj, g.Y, g.H, ws, stream=st)
            L.lora_fused_backward(d, ctx, self.T, g.X, g.Wp, pj, g.dY, g.H, g.dX, ws, stream=st)
        _join(main, use)

    groups = LoraStep.groups
    prepare_ws = LoraStep.prepare_ws
    optimizer_step = LoraStep.optimizer_step
    run = LoraStep.run
    snapshot = LoraStep.snapshot
    restore = LoraStep.restore


class ChainStep(LoraStep):
    """One optimizer step over a stack of adapted linears in which layer l's output is layer
    l + 1's input ("4.3. Training Guide", Truncated BPTT: the backward window is one chunk of
    tokens; Gradient accumulation: raw sums over the chunks in order). Each chunk runs forward
    through every layer and then backward through them in reverse, layer l's output gradient
    being layer l + 1's input gradient, all on one stream (each launch depends on the one
    before). The layers share the adapter rank, scale and dtype; W_l is [d_{l+1}, d_l]."""

    def __init__(self, Ws: Sequence[torch.Tensor], X0: torch.Tensor, dY_top: torch.Tensor, *,
                 layer_ids: Optional[Sequence[int]] = None, proj_id: int = 0, **kw):
        if kw.get("dora"):
            raise ValueError("the chained step has no DoRA mode")
        T, act, dev = X0.shape[0], X0.dtype, X0.device
        for l in range(1, len(Ws)):
            if Ws[l].shape[1] != Ws[l - 1].shape[0]:
                raise ValueError("layer widths do not chain")
        ids = list(layer_ids) if layer_ids is not None else list(range(len(Ws)))
        lins = [Linear(ids[l], proj_id, None, W, None) for l, W in enumerate(Ws)]
        for lin in lins:
            lin.Y = torch.empty((T, lin.out_dim), dtype=act, device=dev)
            lin.dX = torch.empty((T, lin.in_dim), dtype=act, device=dev)
        for l, lin in enumerate(lins):
            lin.X = X0 if l == 0 else lins[l - 1].Y          # the previous layer's output
            lin.dY = dY_top if l == len(lins) - 1 else lins[l + 1].dX
        kw["n_streams"] = 1
        super().__init__(lins, tokens=T, **kw)

    def forward_backward(self, opt_step: int, per_chunk_calls: bool = True):
        """Enqueue the chunked forward / reverse backward of the whole stack (gradients
        accumulate into the arena)."""
        st = torch.cuda.current_stream(self.device)
        ws = self.ws[0]
        ct = self.T // self.chunks
        for c in range(self.chunks):
            ctx = L.make_ctx(opt_step, c, ct)
            sl = slice(c * ct, (c + 1) * ct)
            for l in self.linears:
                L.lora_forward(self.desc(l), ctx, ct, l.X[sl], l.W, l.Wp, l.A, l.B, None, None,
                               l.Y[sl], l.H[sl], ws, stream=st)
            for l in reversed(self.linears):
                L.lora_backward(self.desc(l), ctx, ct, l.X[sl], l.Wp, l.A, l.B, l.dY[sl],
                                l.H[sl], None, None, None, l.dX[sl], l.gA, l.gB, None, ws,
                                stream=st)


# ----------------------------------------------------------------------------------------------
@dataclass
class MultiLinear:
    proj_id: int
    X: torch.Tensor
    W: torch.Tensor
    dY: torch.Tensor
    Wp: Optional[torch.Tensor] = None
    Y: Optional[torch.Tensor] = None
    dX: Optional[torch.Tensor] = None
    H: Optional[torch.Tensor] = None
    A: List[torch.Tensor] = field(default_factory=list)    # per slot, views into the arena
    B: List[torch.Tensor] = field(default_factory=list)
    gA: List[torch.Tensor] = field(default_factory=list)
    gB: List[torch.Tensor] = field(default_factory=list)

    @property
    def in_dim(self) -> int:
        return self.W.shape[1]

    @property
    def out_dim(self) -> int:
        return self.W.shape[0]


class MultiLoraStep:
    """Slot-keyed multi-LoRA over a shared frozen base: every linear has one adapter per slot;
    one arena group per slot = [A of the slot over all linears | B of the slot]."""

    def __init__(self, linears: Sequence[MultiLinear], *, slot_ranks: Sequence[int],
                 slot_scales: Sequence[float], dtype: str, tokens: int, seg_start: torch.Tensor,
                 seg_slot: torch.Tensor, dropout_p: float = 0.0, seed: int = 0,
                 max_norm: float = 1.0, hp: Optional[L.lora_adamw_hp] = None, n_streams: int = 1,
                 planned: bool = True, device="cuda"):
        self.linears = list(linears)
        self.ranks, self.scales = list(slot_ranks), list(slot_scales)
        self.n_slots = len(self.ranks)
        self.rmax = max(self.ranks)
        self.dtype = _DT[dtype]
        self.T = tokens
        self.seg_start, self.seg_slot = seg_start, seg_slot
        self.n_seg = int(seg_slot.numel())
        self.dropout_p, self.seed = dropout_p, seed
        self.max_norm = max_norm
        self.hp = hp if hp is not None else L.make_hp()
        self.device = torch.device(device)
        self.slot_off, self.slot_na, self.slot_nb = [], [], []
        off = 0
        for r in self.ranks:
            na = sum(r * l.in_dim for l in self.linears)
            nb = sum(l.out_dim * r for l in self.linears)
            self.slot_off.append(off)
            self.slot_na.append(na)
            self.slot_nb.append(nb)
            off += na + nb
        self.arena = Arena(off, self.device)
        for s, r in enumerate(self.ranks):
            oa, ob = self.slot_off[s], self.slot_off[s] + self.slot_na[s]
            for l in self.linears:
                l.A.append(self.arena.view("params", oa, (r, l.in_dim)))
                l.gA.append(self.arena.view("grads", oa, (r, l.in_dim)))
                oa += r * l.in_dim
                l.B.append(self.arena.view("params", ob, (l.out_dim, r)))
                l.gB.append(self.arena.view("grads", ob, (l.out_dim, r)))
                ob += l.out_dim * r
        for l in self.linears:
            act = l.X.dtype
            if l.Y is None:
                l.Y = torch.empty((self.T, l.out_dim), dtype=act, device=self.device)
            if l.dX is None:
                l.dX = torch.empty((self.T, l.in_dim), dtype=act, device=self.device)
            if l.H is None:
                l.H = torch.empty((self.T, self.rmax), dtype=torch.float32, device=self.device)
        self.n_streams = max(1, n_streams)
        self.streams = [torch.cuda.Stream(device=self.device) for _ in range(self.n_streams)] \
            if self.n_streams > 1 else []
        self.active_streams = self.n_streams   # streams used by the next enqueue (<= n_streams)
        need = max(L.multi_lora_workspace_size(self.desc(l), self.T, self.n_seg, self.slots(l))
                   for l in self.linears)
        if need == 0:
            raise L.LoraError(L.LORA_ERR_INVALID, "multi_lora_workspace_size")
        self.ws = [_ws(need, self.device) for _ in range(self.n_streams)]
        # the routing plan: the batch's token work tables, built once per forward_backward and
        # read by every linear's calls
        self.plan = None
        if planned and self.n_seg >= 1:
            nbytes = L.multi_lora_plan_size(self.T, self.n_seg, self.n_slots)
            if nbytes == 0:
                raise L.LoraError(L.LORA_ERR_INVALID, "multi_lora_plan_size")
            self.plan = _ws(nbytes, self.device)
        self.scale_norm = torch.zeros(2 * self.n_slots, dtype=torch.float64, device=self.device)
        self.status = torch.zeros(self.n_slots, dtype=torch.int32, device=self.device)

    def desc(self, l: MultiLinear) -> L.lora_desc:
        return L.make_desc(l.in_dim, l.out_dim, self.rmax, 0.0, self.dtype, self.dropout_p,
                           self.seed, 0, l.proj_id, False)

    def slots(self, l: MultiLinear):
        return L.make_slots([dict(A=l.A[s], B=l.B[s], dA=l.gA[s], dB=l.gB[s], rank=self.ranks[s],
                                  scale=self.scales[s]) for s in range(self.n_slots)])

    def prepare_weights(self, stream=None):
        for l in self.linears:
            if l.Wp is None:
                l.Wp = torch.empty(L.lora_prepared_weight_size(self.desc(l)), dtype=torch.uint8,
                                   device=self.device)
            L.lora_prepare_weight(self.desc(l), l.W, l.Wp, stream)

    def forward_backward(self, opt_step: int = 0):
        main = torch.cuda.current_stream(self.device)
        if self.plan is not None:
            L.multi_lora_plan_build(self.T, self.n_seg, self.seg_start, self.seg_slot,
                                    self.n_slots, self.plan, stream=main)
        k, use = _streams_in_use(self)
        _fork(main, use)
        for i, l in enumerate(self.linears):
            st = use[i % k] if use else main
            ws = self.ws[i % k]
            d = self.desc(l)
            ctx = L.make_ctx(opt_step, 0, 0)
            sl = self.slots(l)
            if self.plan is not None:
                L.multi_lora_forward_planned(d, ctx, self.T, self.n_seg, self.plan, l.X, l.W, l.Wp,
                                             sl, l.Y, l.H, ws, stream=st)
                L.multi_lora_backward_planned(d, ctx, self.T, self.n_seg, self.plan, l.X, l.Wp, sl,
                                              l.dY, l.H, l.dX, ws, stream=st)
            else:
                L.multi_lora_forward(d, ctx, self.T, l.X, l.W, l.Wp, self.n_seg, self.seg_start,
                                     self.seg_slot, sl, l.Y, l.H, ws, stream=st)
                L.multi_lora_backward(d, ctx, self.T, l.X, l.Wp, self.n_seg, self.seg_start,
                                      self.seg_slot, sl, l.dY, l.H, l.dX, ws, stream=st)
        _join(main, use)

    def groups(self, ready: Sequence[int], gbs: Sequence[int], lrs: Sequence[float],
               steps: Sequence[int]):
        return L.make_groups([dict(offset=self.slot_off[s], n_a=self.slot_na[s],
                                   n_b=self.slot_nb[s], grad_scale=1.0 / gbs[s],
                                   max_norm=self.max_norm, lr=lrs[s], step=steps[s])
                              for s in ready])

    def retire(self, slots: Sequence[int], clear_params: bool = True):
        """Retire finished adapter slots: their gradients (the partial accumulation), moments and,
        with clear_params, weights are zeroed. The caller resets the slots' accumulated sample
        counts and update counts."""
        if not slots:
            return
        g = L.make_groups([dict(offset=self.slot_off[s], n_a=self.slot_na[s],
                                n_b=self.slot_nb[s], grad_scale=1.0) for s in slots])
        L.lora_retire(self.arena.params, self.arena.grads, self.arena.m, self.arena.v, g,
                      clear_params)

    def optimizer_step(self, ready: Sequence[int], gbs, lrs, steps, zero_grads: bool = True):
        """Prepare + AdamW for the slots whose adapter batch is full (one group each); group i of
        the call reports in scale_norm[2i:2i+2] and status[i]."""
        if not ready:
            return
        g = self.groups(ready, gbs, lrs, steps)
        if not hasattr(self, "_prep_ws"):
            full = self.groups(range(self.n_slots), gbs, lrs, steps)
            self._prep_ws = _ws(L.lora_grad_prepare_workspace_size(full), self.device)
        L.lora_grad_prepare(self.arena.grads, g, self.scale_norm, self.status, self._prep_ws)
        L.lora_adamw_step(self.arena.params, self.arena.grads, self.arena.m, self.arena.v, g,
                          self.hp, self.scale_norm, self.status, zero_grads)
