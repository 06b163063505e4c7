"""ReplaySSM decode for B200: Python binding of the C-ABI library in include/rssm.h.

Every call is marshalled straight to ``lib/librssm.so``; PyTorch provides the
device memory (the context's arena, outputs) and the current CUDA stream.

    from hybrid_model_ssm_gdn_b200 import ReplaySSM
    layer = ReplaySSM("mamba2", batch=256, nheads=128, headdim=64, ngroups=8, window=16,
                      A=A, D=D, in_dtype=torch.bfloat16)
    layer.load_checkpoint(S0)            # fp32 [Bt][H][P][N]
    y = layer.mamba2_step(x, B, C, dt)   # fp32 [Bt][H][P]

Prompts and drafts around it: ``ReplaySSM.prefill`` / ``mamba2_scan``, ``ReplaySSM.gdn_prefill`` / ``gdn_scan``,
``shortconv_prefill`` / ``_step`` / ``_verify`` / ``_commit`` and ``accept_drafts``.  Between a layer's projections:
``gdn_inputs``, ``add_rmsnorm`` and ``gated_rmsnorm``.
"""

from __future__ import annotations

import ctypes as C
import functools

import torch

from . import abi
from .abi import RSSMError

__all__ = ["ReplaySSM", "RSSMError", "conv_mamba2_step", "conv_gdn_step", "snap_verify", "snap_commit", "sched_probe",
           "make_config", "abi", "mamba2_scan", "shortconv_prefill", "shortconv_step", "shortconv_verify",
           "shortconv_commit", "accept_drafts", "gdn_scan", "gdn_inputs", "add_rmsnorm", "gated_rmsnorm"]

_DT = {torch.float32: abi.F32, torch.bfloat16: abi.BF16}
_HP = {"f32": abi.HP_F32, "f16sr": abi.HP_F16_SR, "f8sr": abi.HP_F8_SR}
_READ = {"same": abi.READ_SAME, "nvfp4": abi.READ_NVFP4, "shared_nvfp4": abi.READ_SHARED_NVFP4,
         "nvfp4d": abi.READ_NVFP4D}


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream():
    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dev(t, dtype, name, need=None):
    """``t`` after checking that it is a contiguous CUDA tensor of ``dtype`` with at least ``need`` elements
    (what the kernels read or write through it; a smaller buffer would be overrun on the device)."""
    if t is None:
        return None
    if need is not None and t.numel() < need:
        raise ValueError(f"{name}: needs at least {need} elements, got {t.numel()} (shape {tuple(t.shape)})")
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA tensor of {dtype}, got {t.dtype} on {t.device}")
    return t


def make_config(kind, batch, nheads, headdim, dstate=128, ngroups=1, window=16, max_draft=0,
                in_dtype=torch.bfloat16, hp="f32", read="same", seed=0, q_scale=1.0, A=None, D=None,
                skip_tau=0.0) -> abi.Config:
    return abi.Config(kind={"mamba2": abi.MAMBA2, "gdn": abi.GDN}[kind], batch=batch, nheads=nheads,
                      headdim=headdim, dstate=dstate, ngroups=ngroups, window=window, max_draft=max_draft,
                      in_dtype=_DT[in_dtype], hp=_HP[hp], read=_READ[read], seed=seed, q_scale=q_scale,
                      A=None if A is None else A.data_ptr(), D=None if D is None else D.data_ptr(),
                      skip_tau=skip_tau)


class ReplaySSM:
    """One SSM layer's decode state (checkpoint, read copy, input ring, bookkeeping) on the current GPU."""

    def __init__(self, kind, batch, nheads, headdim, dstate=128, ngroups=1, window=16, max_draft=0,
                 in_dtype=torch.bfloat16, hp="f32", read="same", seed=0, q_scale=1.0, A=None, D=None,
                 device=None, skip_tau=0.0):
        self.lib = abi.load()
        self.kind, self.batch, self.nheads, self.headdim = kind, batch, nheads, headdim
        self.ngroups, self.window, self.max_draft, self.in_dtype = ngroups, window, max_draft, in_dtype
        self.device = torch.device(device or "cuda")
        if kind == "mamba2":
            # the kernels read nheads floats from each through raw pointers: check before any device copy
            for name, t in (("A", A), ("D", D)):
                if t is None or t.numel() < nheads:
                    raise ValueError(f"{name}: needs at least {nheads} elements (one per head), got "
                                     f"{None if t is None else t.numel()}")
            self.A = _dev(A.to(self.device, torch.float32).contiguous(), torch.float32, "A", nheads)
            self.D = _dev(D.to(self.device, torch.float32).contiguous(), torch.float32, "D", nheads)
        else:
            self.A = self.D = None
        self.cfg = make_config(kind, batch, nheads, headdim, dstate, ngroups, window, max_draft, in_dtype, hp, read,
                               seed, q_scale, self.A, self.D, skip_tau)
        nbytes = C.c_size_t()
        abi.check(self.lib.rssm_arena_bytes(C.byref(self.cfg), C.byref(nbytes)), "rssm_arena_bytes")
        self.arena_bytes = nbytes.value
        self.arena = torch.empty(self.arena_bytes, dtype=torch.uint8, device=self.device)
        h = C.c_void_p()
        abi.check(self.lib.rssm_create(C.byref(self.cfg), _ptr(self.arena), self.arena_bytes, C.byref(h)),
                  "rssm_create")
        self.handle = h
        self.rows = headdim
        self.dstate = dstate

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value:
            self.lib.rssm_destroy(h)
            self.handle = None

    # ------------------------------------------------------------------ calls
    def load_checkpoint(self, S):
        S = _dev(S, torch.float32, "S", self.batch * self.nheads * self.rows * self.dstate)
        abi.check(self.lib.rssm_load_checkpoint(self.handle, _ptr(S), _stream()), "rssm_load_checkpoint")

    def _out(self, y, lead):
        if y is None:
            y = torch.empty(*lead, self.nheads, self.rows, dtype=torch.float32, device=self.device)
        n = self.nheads * self.rows
        for s in lead:
            n *= s
        return _dev(y, torch.float32, "y", n)

    def _need(self, name, lead):
        """Elements of token input ``name`` with leading dims ``lead`` ([Bt] or [Bt][T])."""
        n = 1
        for s in lead:
            n *= s
        H, R, N, G = self.nheads, self.rows, self.dstate, self.ngroups
        per = {"x": H * R, "B": G * N, "C": G * N, "dt": H, "q": H * N, "k": H * N, "v": H * R,
               "alpha": H, "beta": H}[name]
        return n * per

    def mamba2_step(self, x, B, C_, dt, y=None):
        d = self.in_dtype
        lead = (self.batch,)
        args = [_dev(x, d, "x", self._need("x", lead)), _dev(B, d, "B", self._need("B", lead)),
                _dev(C_, d, "C", self._need("C", lead)), _dev(dt, d, "dt", self._need("dt", lead))]
        y = self._out(y, lead)
        abi.check(self.lib.rssm_mamba2_step(self.handle, *map(_ptr, args), _ptr(y), _stream()), "rssm_mamba2_step")
        return y

    def gdn_step(self, q, k, v, alpha, beta, y=None):
        d = self.in_dtype
        lead = (self.batch,)
        args = [_dev(q, d, "q", self._need("q", lead)), _dev(k, d, "k", self._need("k", lead)),
                _dev(v, d, "v", self._need("v", lead)), _dev(alpha, torch.float32, "alpha", self._need("alpha", lead)),
                _dev(beta, torch.float32, "beta", self._need("beta", lead))]
        y = self._out(y, lead)
        abi.check(self.lib.rssm_gdn_step(self.handle, *map(_ptr, args), _ptr(y), _stream()), "rssm_gdn_step")
        return y

    def verify(self, T, y=None, **tok):
        d = self.in_dtype
        f32 = {"alpha", "beta"}
        t = {k: _dev(v, torch.float32 if k in f32 else d, k, self._need(k, (self.batch, T))) for k, v in tok.items()}
        toks = abi.Tokens(**{k: v.data_ptr() for k, v in t.items()})
        y = self._out(y, (self.batch, T))
        abi.check(self.lib.rssm_verify(self.handle, T, C.byref(toks), _ptr(y), _stream()), "rssm_verify")
        return y

    def commit(self, accepted):
        a = _dev(accepted, torch.int32, "accepted", self.batch)
        abi.check(self.lib.rssm_commit(self.handle, _ptr(a), _stream()), "rssm_commit")

    def prefill(self, x, B, C_, dt, offsets, slots=None, resume=None, y=None, workspace=None):
        """Run packed prompts (rssm_mamba2_prefill): x [total][H][P], B, C [total][G][128], dt [total][H];
        offsets int32 [n+1]; slots int32 [n] (sequence of each prompt), resume uint8 [n] -> y fp32 [total][H][P], with NaN
        for refused prompts where the call makes it."""
        H, P, G = self.nheads, self.rows, self.ngroups
        device = _device(x, "x")
        if self.arena.get_device() != device:
            raise ValueError(f"the context is on {self.arena.device}, but the current device is cuda:{device}")
        total, pr, tok, y = _scan_args(x, B, C_, dt, offsets, slots, resume, y, H, P, G, self.in_dtype, device)
        work = _scan_work(self.lib, self.cfg, total, pr.nseq, workspace, device)
        abi.check(self.lib.rssm_mamba2_prefill(self.handle, C.byref(pr), C.byref(tok), _addr(y), _addr(work),
                                               0 if work is None else work.numel(), _stream_of(device)), "rssm_mamba2_prefill")
        return y

    def gdn_prefill(self, q, k, v, alpha, beta, offsets, slots=None, resume=None, y=None, workspace=None):
        """Run packed prompts (rssm_gdn_prefill): q, k [total][heads or a divisor of them][128], v [total][H][d_v], alpha,
        beta fp32 [total][H]; offsets int32 [n+1]; slots int32 [n], resume uint8 [n] -> y fp32 [total][H][d_v], with NaN for
        refused prompts where the call makes it."""
        device = _device(v, "v")
        if self.arena.get_device() != device:
            raise ValueError(f"the context is on {self.arena.device}, but the current device is cuda:{device}")
        total, pr, tok, y, Hk = _gdn_args(q, k, v, alpha, beta, offsets, slots, resume, y, self.nheads, self.rows,
                                          self.in_dtype, device)
        work = _scan_work(self.lib, self.cfg, total, pr.nseq, workspace, device, "rssm_gdn_scan_workspace")
        abi.check(self.lib.rssm_gdn_prefill(self.handle, Hk, C.byref(pr), C.byref(tok), _addr(y), _addr(work),
                                            0 if work is None else work.numel(), _stream_of(device)), "rssm_gdn_prefill")
        return y

    def flush(self, mask=None):
        m = _dev(mask, torch.uint8, "mask", self.batch)
        abi.check(self.lib.rssm_flush(self.handle, _ptr(m), _stream()), "rssm_flush")

    # ------------------------------------------------------------------ inspection
    def export(self, state=True, ring=True):
        """Return {"S": fp32 checkpoint, "meta": int32 [Bt][4], ring views...} (device tensors)."""
        dev, Bt, H, L, R = self.device, self.batch, self.nheads, self.window, self.rows
        out = {"meta": torch.empty(Bt, 4, dtype=torch.int32, device=dev)}
        if state:
            out["S"] = torch.empty(Bt, H, R, 128, dtype=torch.float32, device=dev)
        raw = None
        if ring:
            nb = C.c_size_t()
            abi.check(self.lib.rssm_ring_bytes(C.byref(self.cfg), C.byref(nb)), "rssm_ring_bytes")
            raw = torch.empty(nb.value, dtype=torch.uint8, device=dev)
        abi.check(self.lib.rssm_export(self.handle, _ptr(out.get("S")), _ptr(raw), _ptr(out["meta"]), _stream()),
                  "rssm_export")
        if raw is not None:
            esz = 2 if self.in_dtype == torch.bfloat16 else 4
            parts = ([("x", (Bt, H, L, R), esz), ("B", (Bt, self.ngroups, L, 128), esz), ("dt", (Bt, H, L), 4)]
                     if self.kind == "mamba2" else
                     [("k", (Bt, H, L, 128), esz), ("v", (Bt, H, L, R), esz), ("alpha", (Bt, H, L), 4),
                      ("beta", (Bt, H, L), 4)])
            off = 0
            for name, shape, sz in parts:
                n = 1
                for s in shape:
                    n *= s
                dt = self.in_dtype if sz == esz and name not in ("dt", "alpha", "beta") else torch.float32
                out["ring_" + name] = raw[off:off + n * sz].view(dt).view(shape)
                off += n * sz
        return out

    def export_read_copy(self):
        dev, Bt, H, R = self.device, self.batch, self.nheads, self.rows
        codes = torch.empty(Bt, H, R, 64, dtype=torch.uint8, device=dev)
        scales = torch.empty(Bt, H, R, 8, dtype=torch.uint8, device=dev)
        g = torch.empty(Bt, H, (R + 63) // 64, dtype=torch.float32, device=dev)
        abi.check(self.lib.rssm_export_read_copy(self.handle, _ptr(codes), _ptr(scales), _ptr(g), _stream()),
                  "rssm_export_read_copy")
        return {"packed": codes, "scales": scales, "g": g}

    def export_column_scales(self):
        """Column-group scales of the two-axis read copy: uint8 E4M3 [Bt][H][ceil(rows/16)][128]."""
        cs = torch.empty(self.batch, self.nheads, (self.rows + 15) // 16, 128, dtype=torch.uint8, device=self.device)
        abi.check(self.lib.rssm_export_column_scales(self.handle, _ptr(cs), _stream()), "rssm_export_column_scales")
        return cs

    def export_skip(self):
        """Decay-aware skip flags uint8 [Bt][H] (1 = the next call skips that head's checkpoint read)."""
        flags = torch.empty(self.batch, self.nheads, dtype=torch.uint8, device=self.device)
        abi.check(self.lib.rssm_export_skip(self.handle, _ptr(flags), _stream()), "rssm_export_skip")
        return flags

    def get_error(self):
        """(code, seq) of the sticky device error word; synchronises the current stream."""
        code, seq = C.c_int(), C.c_int()
        st = self.lib.rssm_get_error(self.handle, C.byref(code), C.byref(seq), _stream())
        if st not in (0, 6):
            abi.check(st, "rssm_get_error")
        return code.value, seq.value


# ---------------------------------------------------------------------- prompts and drafts

def _arr(t, dtype, name, shape, device):
    """The address of ``t`` (None: null) after checking that it is a contiguous tensor of ``dtype`` and exactly ``shape`` on
    the current device, number ``device``."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected a contiguous CUDA tensor of {dtype}, got {t.dtype} on {t.device}")
    raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{device}")


def _device(t, name):
    """The current device's number; ``t`` has to be on a GPU (on which, ``_arr`` and its like check)."""
    if t.get_device() < 0:
        raise ValueError(f"{name}: expected a contiguous CUDA tensor, got {t.dtype} on {t.device}")
    return torch._C._cuda_getDevice()


_stream_of = torch._C._cuda_getCurrentRawStream  # a device's current stream, without building an object


def _addr(t):
    return None if t is None else t.data_ptr()


def _prompts(total, offsets, slots, resume, device, fresh):
    n = offsets.numel() - 1
    if n < 1:
        raise ValueError(f"offsets: needs at least 2 elements, got {n + 1}")
    return abi.Prompts(total, n, _arr(offsets, torch.int32, "offsets", (n + 1,), device),
                       _arr(slots, torch.int32, "slots", (n,), device), _arr(resume, torch.uint8, "resume", (n,), device),
                       fresh)


def _in_dtype(t, name):
    if t.dtype not in _DT:
        raise ValueError(f"{name}: expected torch.float32 or torch.bfloat16, got {t.dtype}")
    return t.dtype


def _scan_args(x, B, C_, dt, offsets, slots, resume, y, H, P, G, dtype, device):
    total = x.shape[0]
    tok = abi.Tokens(_arr(x, dtype, "x", (total, H, P), device), _arr(B, dtype, "B", (total, G, 128), device),
                     _arr(C_, dtype, "C", (total, G, 128), device), _arr(dt, dtype, "dt", (total, H), device))
    pr = _prompts(total, offsets, slots, resume, device, y is None)
    if y is None:
        y = x.new_empty((total, H, P), dtype=torch.float32)
    else:
        _arr(y, torch.float32, "y", (total, H, P), device)
    return total, pr, tok, y


def _scan_work(lib, cfg, total, nseq, workspace, device, size="rssm_mamba2_scan_workspace"):
    """The scratch tensor of a scan: the caller's, or a new one from the caching allocator (None if none is needed)."""
    n = C.c_size_t()
    abi.check(getattr(lib, size)(C.byref(cfg), total, nseq, C.byref(n)), size)
    if n.value == 0:
        return None
    if workspace is not None:
        if workspace.get_device() != device or workspace.dtype != torch.uint8 or \
                not workspace.is_contiguous() or workspace.numel() < n.value:
            raise ValueError(f"workspace: expected a contiguous tensor of uint8 on the current CUDA device with at least "
                             f"{n.value} elements")
        return workspace
    return torch.empty(n.value, dtype=torch.uint8, device="cuda")


def mamba2_scan(S, x, B, C_, dt, A, D, offsets, slots=None, resume=None, y=None, workspace=None):
    """Mamba-2 over packed prompts on the caller's states (rssm_mamba2_scan): S fp32 [batch][H][P][128], the prompts'
    sequences rewritten in place; x [total][H][P], B, C [total][G][128], dt [total][H] (bf16 or fp32), A, D fp32 [H];
    prompt i is rows offsets[i] .. offsets[i+1]-1 and belongs to S[slots[i]] (S[i] without slots), from which it
    continues where resume[i] is set -> y fp32 [total][H][P].  Without ``y``, rows of refused prompts (an offset or slot out
    of range: all rows; a slot named twice) are NaN in the new one; with it they stay as they were.  Rows of no prompt are
    not written in either."""
    if x.dim() != 3 or B.dim() != 3 or S.dim() != 4:
        raise ValueError("x, B and S: expected 3, 3 and 4 dimensions")
    total, H, P = x.shape
    dtype = _in_dtype(x, "x")
    device = _device(S, "S")
    at = _arr(S, torch.float32, "S", (S.shape[0], H, P, 128), device)
    cfg = abi.Config(abi.MAMBA2, S.shape[0], H, P, 128, B.shape[1], 1, 0, _DT[dtype], abi.HP_F32, abi.READ_SAME, 0, 1.0,
                     _arr(A, torch.float32, "A", (H,), device), _arr(D, torch.float32, "D", (H,), device), 0.0)
    total, pr, tok, y = _scan_args(x, B, C_, dt, offsets, slots, resume, y, H, P, B.shape[1], dtype, device)
    lib = abi.load()
    work = _scan_work(lib, cfg, total, pr.nseq, workspace, device)
    abi.check(lib.rssm_mamba2_scan(C.byref(cfg), C.byref(pr), C.byref(tok), at, y.data_ptr(), _addr(work),
                                   0 if work is None else work.numel(), _stream_of(device)), "rssm_mamba2_scan")
    return y


def _gdn_args(q, k, v, alpha, beta, offsets, slots, resume, y, H, R, dtype, device):
    total, Hk = v.shape[0], q.shape[1] if q.dim() == 3 else 0
    if Hk < 1 or H % Hk:
        raise ValueError(f"q: expected [total][heads that divide {H}][128], got {tuple(q.shape)}")
    tok = abi.Tokens(None, None, None, None, _arr(q, dtype, "q", (total, Hk, 128), device),
                     _arr(k, dtype, "k", (total, Hk, 128), device), _arr(v, dtype, "v", (total, H, R), device),
                     _arr(alpha, torch.float32, "alpha", (total, H), device),
                     _arr(beta, torch.float32, "beta", (total, H), device))
    pr = _prompts(total, offsets, slots, resume, device, y is None)
    if y is None:
        y = v.new_empty((total, H, R), dtype=torch.float32)
    else:
        _arr(y, torch.float32, "y", (total, H, R), device)
    return total, pr, tok, y, Hk


def gdn_scan(S, q, k, v, alpha, beta, offsets, slots=None, resume=None, q_scale=1.0, y=None, workspace=None):
    """The gated delta rule over packed prompts on the caller's states (rssm_gdn_scan): S fp32 [batch][H][d_v][128], the
    prompts' sequences rewritten in place; q, k [total][heads or a divisor of them][128], v [total][H][d_v] (bf16 or fp32),
    alpha, beta fp32 [total][H]; offsets, slots, resume, refused prompts and rows of no prompt as for ``mamba2_scan``
    -> y fp32 [total][H][d_v]."""
    if v.dim() != 3 or S.dim() != 4:
        raise ValueError("v and S: expected 3 and 4 dimensions")
    H, R = v.shape[1:]
    dtype = _in_dtype(v, "v")
    device = _device(S, "S")
    at = _arr(S, torch.float32, "S", (S.shape[0], H, R, 128), device)
    cfg = abi.Config(abi.GDN, S.shape[0], H, R, 128, 1, 1, 0, _DT[dtype], abi.HP_F32, abi.READ_SAME, 0, q_scale, None, None,
                     0.0)
    total, pr, tok, y, Hk = _gdn_args(q, k, v, alpha, beta, offsets, slots, resume, y, H, R, dtype, device)
    lib = abi.load()
    work = _scan_work(lib, cfg, total, pr.nseq, workspace, device, "rssm_gdn_scan_workspace")
    abi.check(lib.rssm_gdn_scan(C.byref(cfg), Hk, C.byref(pr), C.byref(tok), at, y.data_ptr(), _addr(work),
                                0 if work is None else work.numel(), _stream_of(device)), "rssm_gdn_scan")
    return y


_I3, _P3 = C.c_int * 3, C.c_void_p * 3


def _row_stride(x, lead, ch):
    """Elements from one row of x [*lead][ch] to the next: rows may lie apart (a slice of a wider projection) but
    evenly, with contiguous channels."""
    if x.is_contiguous():
        return ch
    stride = x.stride(-2) if x.shape[-2] > 1 else ch
    if len(lead) == 2 and lead[0] > 1:
        if lead[1] == 1:
            stride = x.stride(0)
        elif x.stride(0) != lead[1] * stride:
            raise ValueError("x: the rows of all sequences must lie evenly apart")
    if x.stride(-1) != 1 or stride < ch or stride % 8:
        raise ValueError(f"x: expected contiguous channels and a row stride that is a multiple of 8, got {x.stride()}")
    return stride


def _shortconv(hist, cur, x, weight, bias, splits, activation, out, lead):
    """Arguments of a short-convolution call (config, addresses of hist, cur and x, row stride, the outputs and their
    addresses, device); ``lead``: the leading dimensions of x."""
    if hist.dim() != 3 or weight.dim() != 2:
        raise ValueError("hist and weight: expected 3 and 2 dimensions")
    dtype = _in_dtype(x, "x")
    batch, ring, ch = hist.shape
    width = weight.shape[1]
    device = _device(hist, "hist")
    hist_at = _arr(hist, dtype, "hist", (batch, ring, ch), device)
    cur_at = _arr(cur, torch.int32, "cur", (batch,), device)
    splits = (ch,) if splits is None else tuple(splits)
    if len(splits) > 3 or sum(splits) != ch or min(splits) < 1:
        raise ValueError(f"splits: expected up to three positive sizes that sum to {ch}, got {splits}")
    if activation is not None and activation != "silu":
        raise ValueError(f"activation: expected None or 'silu', got {activation!r}")
    if x.shape != (*lead, ch) or x.get_device() != device:
        raise ValueError(f"x: expected shape {(*lead, ch)} on the current CUDA device, got {tuple(x.shape)} on {x.device}")
    stride = _row_stride(x, lead, ch)
    if out is None:
        out = tuple([x.new_empty((*lead, c)) for c in splits])
        ptrs = _P3(*[o.data_ptr() for o in out])
    else:
        if len(out) != len(splits):
            raise ValueError(f"out: expected {len(splits)} tensors, got {len(out)}")
        ptrs = _P3(*[_arr(o, dtype, "out", (*lead, c), device) for o, c in zip(out, splits)])
    cfg = abi.ShortConvConfig(batch, ch, width, ring, _DT[dtype], activation is not None, _I3(*splits),
                              _arr(weight, dtype, "weight", (ch, width), device), _arr(bias, dtype, "bias", (ch,), device))
    return C.byref(cfg), hist_at, cur_at, x.data_ptr(), stride, out, C.byref(ptrs), device


def shortconv_prefill(hist, cur, x, weight, bias, offsets, slots=None, resume=None, splits=None, activation="silu",
                      out=None):
    """Short causal convolution over packed prompts (rssm_shortconv_prefill): x [total][channels]; hist
    [batch][ring][channels] and cur int32 [batch] are the sequences' histories -> one tensor [total][n] a split.
    Without ``out``, rows of refused prompts are NaN."""
    fresh = out is None
    cfg, h, c, at, stride, out, ptrs, device = _shortconv(hist, cur, x, weight, bias, splits, activation, out,
                                                          (x.shape[0],))
    pr = _prompts(x.shape[0], offsets, slots, resume, device, fresh)
    abi.check(abi.load().rssm_shortconv_prefill(cfg, C.byref(pr), h, c, at, stride, ptrs, _stream_of(device)),
              "rssm_shortconv_prefill")
    return out


def shortconv_step(hist, cur, x, weight, bias=None, splits=None, activation="silu", out=None):
    """One token a sequence: x [batch][channels] -> one tensor [batch][n] a split; cur advances."""
    cfg, h, c, at, stride, out, ptrs, device = _shortconv(hist, cur, x, weight, bias, splits, activation, out,
                                                          (hist.shape[0],))
    abi.check(abi.load().rssm_shortconv_step(cfg, h, c, at, stride, ptrs, _stream_of(device)), "rssm_shortconv_step")
    return out


def shortconv_verify(hist, cur, x, weight, bias=None, splits=None, activation="silu", out=None):
    """T tentative tokens a sequence: x [batch][T][channels] -> one tensor [batch][T][n] a split; cur stays until
    ``shortconv_commit``."""
    if x.dim() != 3:
        raise ValueError(f"x: expected 3 dimensions, got {x.dim()}")
    T = x.shape[1]
    cfg, h, c, at, stride, out, ptrs, device = _shortconv(hist, cur, x, weight, bias, splits, activation, out,
                                                          (hist.shape[0], T))
    abi.check(abi.load().rssm_shortconv_verify(cfg, T, h, c, at, stride, ptrs, _stream_of(device)),
              "rssm_shortconv_verify")
    return out


def shortconv_commit(hist, cur, accepted, width):
    """Advance the cursors by the accepted prefixes, int32 [batch]; ``width`` is the filter's."""
    batch, ring = hist.shape[:2]
    device = _device(cur, "cur")
    cfg = abi.ShortConvConfig(batch=batch, width=width, ring=ring)
    abi.check(abi.load().rssm_shortconv_commit(C.byref(cfg), _arr(cur, torch.int32, "cur", (batch,), device),
                                               _arr(accepted, torch.int32, "accepted", (batch,), device),
                                               _stream_of(device)), "rssm_shortconv_commit")


def _rows(t, name, batch, rows, vocab, device):
    """The row stride of [batch][rows][vocab] probabilities whose rows lie evenly apart."""
    if t.shape != (batch, rows, vocab) or t.dtype is not torch.float32 or t.get_device() != device:
        raise ValueError(f"{name}: expected fp32 of shape {(batch, rows, vocab)} on the current CUDA device, got {t.dtype} "
                         f"of {tuple(t.shape)} on {t.device}")
    if t.is_contiguous():
        return vocab
    ld = t.stride(1) if rows > 1 else t.stride(0)
    if t.stride(2) != 1 and vocab > 1 or ld < vocab or (rows > 1 and batch > 1 and t.stride(0) != rows * ld):
        raise ValueError(f"{name}: expected contiguous rows that lie evenly apart, got strides {t.stride()}")
    return ld


def accept_drafts(target, tokens, u, draft=None, count=None):
    """Verify drafts against target probabilities (rssm_accept_drafts): target fp32 [batch][T+1][vocab], tokens int32
    [batch][T], u fp32 [batch][T+1] in [0, 1), draft fp32 [batch][T][vocab] or None (drafts that were looked up), count
    int32 [batch] (drafts of each sequence) -> (accepted, accepted + 1, next token), int32 [batch] each."""
    if target.dim() != 3:
        raise ValueError(f"target: expected 3 dimensions, got {target.dim()}")
    batch, T, vocab = target.shape[0], target.shape[1] - 1, target.shape[2]
    device = _device(target, "target")
    ld_t = _rows(target, "target", batch, T + 1, vocab, device)
    ld_d = 0 if draft is None else _rows(draft, "draft", batch, T, vocab, device)
    got = target.new_empty((3, batch), dtype=torch.int32)
    at = got.data_ptr()
    abi.check(abi.load().rssm_accept_drafts(batch, T, vocab, target.data_ptr(), ld_t, _addr(draft), ld_d,
                                            _arr(tokens, torch.int32, "tokens", (batch, T), device),
                                            _arr(count, torch.int32, "count", (batch,), device),
                                            _arr(u, torch.float32, "u", (batch, T + 1), device),
                                            at, at + 4 * batch, at + 8 * batch, _stream_of(device)), "rssm_accept_drafts")
    return got.unbind(0)


# ---------------------------------------------------------------------- between a layer's projections

def _apart(t, name, lead, width, inner, dtype, device):
    """The row stride of t [*lead][*inner], rows of ``width`` contiguous elements that lie evenly apart."""
    if t.shape != (*lead, *inner) or t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name}: expected {dtype} of shape {(*lead, *inner)} on the current CUDA device, got {t.dtype} of "
                         f"{tuple(t.shape)} on {t.device}")
    if t.is_contiguous():
        return width
    at, step = width, 1
    for n, s in zip(reversed(t.shape[len(lead):]), reversed(t.stride()[len(lead):])):
        if n > 1 and s != step:
            raise ValueError(f"{name}: expected contiguous rows, got strides {t.stride()}")
        step *= n
    step = None
    for n, s in zip(reversed(t.shape[:len(lead)]), reversed(t.stride()[:len(lead)])):
        if n == 1:
            continue
        if step is None:
            at = step = s
        elif s != step:
            raise ValueError(f"{name}: the rows must lie evenly apart, got strides {t.stride()}")
        step *= n
    if at < width:
        raise ValueError(f"{name}: the rows overlap, strides {t.stride()}")
    return at


def _count(shape):
    n = 1
    for s in shape:
        n *= s
    return n


def _steps(shape):
    """(shape, strides of a contiguous tensor): torch.empty_strided takes half the time of new_empty."""
    steps, n = [], 1
    for s in reversed(shape):
        steps.append(n)
        n *= max(s, 1)
    return torch.Size(shape), tuple(reversed(steps))


def _row_step(t, name, shape, lead, inner, width, dtype, device):
    """``_apart`` behind a look for the usual case, a contiguous tensor."""
    if t.shape == shape and t.dtype is dtype and t.get_device() == device and t.is_contiguous():
        return width
    return _apart(t, name, lead, width, inner, dtype, device)


# What follows from sizes, types and numbers alone is worked out once for each (a decode step's calls are as long as their
# checks).  Callers pass plain numbers: a tensor would be looked up by its identity, whatever it holds by then.
@functools.lru_cache(maxsize=1024)
def _inputs_plan(q_shape, a_shape, dtype, expand):
    """(leading sizes, rows, heads of v, of q, of the outputs, shape of q; shapes and strides of the gates and vectors out)"""
    if len(q_shape) < 2 or len(a_shape) < 1:
        raise ValueError("q and a: expected at least 2 dimensions and 1")
    if dtype not in _DT:
        raise ValueError(f"q: expected torch.float32 or torch.bfloat16, got {dtype}")
    lead, Hk, H = q_shape[:-2], q_shape[-2], a_shape[-1]
    if Hk < 1 or H < 1 or H % Hk:
        raise ValueError(f"q: expected [...][heads that divide {H}][128], got {tuple(q_shape)}")
    heads = H if expand else Hk
    return lead, _count(lead), H, Hk, heads, torch.Size((*lead, Hk, 128)), _steps((*lead, H)), _steps((*lead, heads, 128))


def gdn_inputs(q, k, a, b, A_log, dt_bias, eps=1e-6, expand=False, out=None):
    """Inputs of the gated delta rule from a layer's projections and convolution (rssm_gdn_inputs): q, k [...][Hk][128] and
    a, b [...][H] (bf16 or fp32; rows may lie apart), A_log, dt_bias fp32 [H], H a multiple of Hk -> (q, k, alpha, beta):
    q and k with length 1, [...][Hk][128], or with ``expand`` [...][H][128] as the decode calls take them; alpha =
    exp(-exp(A_log) softplus(a + dt_bias)), beta = sigmoid(b), fp32 [...][H]."""
    dtype = q.dtype
    lead, rows, H, Hk, heads, in_shape, gates, vectors = _inputs_plan(q.shape, a.shape, dtype, bool(expand))
    gate_shape, out_shape = gates[0], vectors[0]
    device = _device(q, "q")
    vec, row = 128 * Hk, (Hk, 128)
    strides = (_row_step(q, "q", in_shape, lead, row, vec, dtype, device),
               _row_step(k, "k", in_shape, lead, row, vec, dtype, device),
               _row_step(a, "a", gate_shape, lead, (H,), H, dtype, device),
               _row_step(b, "b", gate_shape, lead, (H,), H, dtype, device))
    if out is None:
        qk = torch.empty_strided(*vectors, dtype=dtype, device=q.device)
        gate = torch.empty_strided(*gates, dtype=torch.float32, device=q.device)
        out = (qk, torch.empty_like(qk), gate, torch.empty_like(gate))
    else:
        for t, n, s, d in zip(out, ("q", "k", "alpha", "beta"), (out_shape, out_shape, gate_shape, gate_shape),
                              (dtype, dtype, torch.float32, torch.float32), strict=True):
            _arr(t, d, "out " + n, s, device)
    cfg = abi.GdnInputsConfig(rows, H, Hk, heads, _DT[dtype], eps, q.data_ptr(), k.data_ptr(), a.data_ptr(), b.data_ptr(),
                              *strides, _arr(A_log, torch.float32, "A_log", (H,), device),
                              _arr(dt_bias, torch.float32, "dt_bias", (H,), device))
    qo, ko, al, be = out
    abi.check(abi.load().rssm_gdn_inputs(C.byref(cfg), qo.data_ptr(), ko.data_ptr(), al.data_ptr(), be.data_ptr(),
                                         _stream_of(device)), "rssm_gdn_inputs")
    return out


_SCALES = {None: abi.SCALE_NONE, "row": abi.SCALE_ROW, "block": abi.SCALE_BLOCK}


@functools.lru_cache(maxsize=1024)
def _norm_plan(shape, x_dtype, weight_shape, weight_dtype, group, eps, offset, out_dtype, scale, gate_dtype, norm_first):
    """(the call's config by reference, (type, shape and strides of the output, those of the scales or None), shape of the
    weight) of a norm over the last dimension"""
    columns, lead = shape[-1], shape[:-1]
    group = group or columns
    if scale not in _SCALES:
        raise ValueError(f"scale: expected None, 'row' or 'block', got {scale!r}")
    if group < 1 or columns % group:
        raise ValueError(f"group: expected a divisor of {columns}, got {group}")
    wcols = columns if _count(weight_shape) == columns else group
    if scale is None:
        if out_dtype not in _DT:
            raise ValueError(f"out_dtype: expected torch.float32 or torch.bfloat16, got {out_dtype}")
        kind, want, scales = _DT[out_dtype], out_dtype, None
    else:
        kind, want = abi.F32, torch.float8_e4m3fn
        scales = _steps(lead if scale == "row" else (*lead, (columns + 127) // 128))
    if weight_dtype not in _DT:
        raise ValueError(f"weight: expected torch.float32 or torch.bfloat16, got {weight_dtype}")
    cfg = abi.NormConfig(_count(lead), columns, group, wcols, _DT[x_dtype], gate_dtype, _DT[weight_dtype], kind, _SCALES[scale],
                         norm_first, eps, offset)
    return C.byref(cfg), (want, _steps(shape), scales), torch.Size((wcols,))


def _norm_out(x, plan, out, device):
    """(output, scales or None, and what the call returns)"""
    want, size, scales = plan
    if out is None:
        y = torch.empty_strided(*size, dtype=want, device=x.device)
        if scales is None:
            return y, None, y
        s = torch.empty_strided(*scales, dtype=torch.float32, device=x.device)
        return y, s, (y, s)
    y, s = (out, None) if scales is None else out
    _arr(y, want, "out", size[0], device)
    if scales is not None:
        _arr(s, torch.float32, "scales", scales[0], device)
    return y, s, out


def add_rmsnorm(x, weight, residual=None, eps=1e-6, offset=0.0, out_dtype=None, scale=None, out=None):
    """Root-mean-square norm over the last dimension with the residual's addition (rssm_add_rmsnorm): h = x + residual goes
    back to ``residual`` in place; x, residual [...][n] (bf16 or fp32; rows may lie apart), weight [n] -> h / rms(h) (offset +
    weight) in ``out_dtype`` (x's), or with ``scale`` "row" or "block" (of 128 columns) the pair (float8_e4m3fn, scales fp32
    [...] or [...][ceil(n/128)])."""
    shape, dtype = x.shape, _in_dtype(x, "x")
    n, lead = shape[-1], shape[:-1]
    device = _device(x, "x")
    stride = _row_step(x, "x", shape, lead, (n,), n, dtype, device)
    r_stride = 0 if residual is None else _row_step(residual, "residual", shape, lead, (n,), n, dtype, device)
    cfg, plan, w_shape = _norm_plan(shape, dtype, weight.shape, weight.dtype, 0, float(eps), float(offset), out_dtype or dtype,
                                    scale, 0, 0)
    y, s, got = _norm_out(x, plan, out, device)
    abi.check(abi.load().rssm_add_rmsnorm(cfg, x.data_ptr(), stride, _addr(residual), r_stride,
                                          _arr(weight, weight.dtype, "weight", w_shape, device), y.data_ptr(), _addr(s),
                                          _stream_of(device)), "rssm_add_rmsnorm")
    return got


def gated_rmsnorm(y, gate, weight, group=None, eps=1e-6, offset=0.0, norm_first=True, out_dtype=None, scale=None, out=None):
    """The gated norm behind a layer (rssm_gated_rmsnorm): y [...][n], gate [...][n] (bf16 or fp32 each; rows may lie apart),
    weight [n], or [group] for all groups -> with s = silu(gate), the norm of each ``group`` columns (all) of y times s, or
    without ``norm_first`` of y s; in ``out_dtype`` (gate's) or in 8 bits as for ``add_rmsnorm``."""
    shape = y.shape
    n, lead = shape[-1], shape[:-1]
    device = _device(y, "y")
    dtype, gate_dtype = _in_dtype(y, "y"), _in_dtype(gate, "gate")
    stride = _row_step(y, "y", shape, lead, (n,), n, dtype, device)
    g_stride = _row_step(gate, "gate", shape, lead, (n,), n, gate_dtype, device)
    cfg, plan, w_shape = _norm_plan(shape, dtype, weight.shape, weight.dtype, group and int(group), float(eps), float(offset),
                                    out_dtype or gate_dtype, scale, _DT[gate_dtype], bool(norm_first))
    o, s, got = _norm_out(y, plan, out, device)
    abi.check(abi.load().rssm_gated_rmsnorm(cfg, y.data_ptr(), stride, gate.data_ptr(), g_stride,
                                            _arr(weight, weight.dtype, "weight", w_shape, device), o.data_ptr(), _addr(s),
                                            _stream_of(device)), "rssm_gated_rmsnorm")
    return got


# ---------------------------------------------------------------------- comparison kernels

def conv_mamba2_step(cfg, S, x, B, C_, dt, y):
    lib = abi.load()
    abi.check(lib.rssm_conv_mamba2_step(C.byref(cfg), *map(_ptr, (S, x, B, C_, dt, y)), _stream()),
              "rssm_conv_mamba2_step")
    return y


def conv_gdn_step(cfg, S, q, k, v, alpha, beta, y):
    lib = abi.load()
    abi.check(lib.rssm_conv_gdn_step(C.byref(cfg), *map(_ptr, (S, q, k, v, alpha, beta, y)), _stream()),
              "rssm_conv_gdn_step")
    return y


def snap_verify(cfg, snaps, cur, T, y, **tok):
    lib = abi.load()
    toks = abi.Tokens(**{k: v.data_ptr() for k, v in tok.items()})
    abi.check(lib.rssm_snap_verify(C.byref(cfg), _ptr(snaps), _ptr(cur), T, C.byref(toks), _ptr(y), _stream()),
              "rssm_snap_verify")
    return y


def sched_probe(units, blocks):
    """Run the unit-scheduler self-test (no caller device memory): -> (units drawn per block, units not drawn
    exactly once)."""
    lib = abi.load()
    per_block = (C.c_int * blocks)()
    bad = C.c_int(-1)
    abi.check(lib.rssm_sched_probe(units, blocks, C.cast(per_block, C.c_void_p), C.cast(C.pointer(bad), C.c_void_p),
                                   _stream()), "rssm_sched_probe")
    return list(per_block), bad.value


def snap_commit(cfg, cur, accepted):
    lib = abi.load()
    abi.check(lib.rssm_snap_commit(C.byref(cfg), _ptr(cur), _ptr(accepted), _stream()), "rssm_snap_commit")
