"""ctypes binding of ``libflashloop.so`` (declared in ``include/flashloop.h``).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  torch provides device memory (the workspace and the weight tensors)
and streams.  Loading fails loudly when the library is missing; there is no
fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libflashloop.so")

FL_OK = 0
FL_OPT_USE_GRAPH = 1
FL_OPT_PROFILE = 2
FL_OPT_PDL = 3
FL_OPT_GEMM_TIMES = 5
FL_OPT_TC_PREFILL = 6
FL_OPT_CORR_CLUSTER = 7
KINDS = ["gemm", "attn", "dscore", "correct", "kv", "select", "norm", "other"]
STATUS = {0: "ok", 1: "invalid argument", 2: "capacity exceeded", 3: "workspace", 4: "cuda error",
          5: "timeout", 6: "nonfinite", 7: "unsupported"}


class FlashLoopError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        super().__init__(f"{what}: {STATUS.get(status, status)} ({status}) {detail}".strip())
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int), ("n_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("ffn_dim", ctypes.c_int), ("n_layers", ctypes.c_int),
                ("n_loops", ctypes.c_int), ("rho", ctypes.c_double), ("c_cols", ctypes.c_int),
                ("q_tile", ctypes.c_int), ("resid_bits", ctypes.c_int), ("group_size", ctypes.c_int),
                ("resid_scale", ctypes.c_float), ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float),
                ("vocab", ctypes.c_int), ("max_batch", ctypes.c_int), ("max_ctx", ctypes.c_int),
                ("max_tokens", ctypes.c_int), ("kv_mode", ctypes.c_int), ("n_prelude", ctypes.c_int),
                ("n_coda", ctypes.c_int), ("loop_embed", ctypes.c_int), ("inject_scale", ctypes.c_float),
                ("resid_rows", ctypes.c_int)]


LAYER_FIELDS = ("attn_norm", "w_qkv", "w_o", "mlp_norm", "w_gate", "w_up", "w_down")


class Layers(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in LAYER_FIELDS]


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in LAYER_FIELDS + ("final_norm", "w_out")] + [
        ("prelude", Layers), ("coda", Layers), ("loop_embed", ctypes.c_void_p)]


_I2 = ctypes.c_int64 * 2
_I3 = ctypes.c_int64 * 3


def _fields(names, kind):
    return [(n, kind) for n in names.split()]


class PrefixArgs(ctypes.Structure):
    _fields_ = (_fields("q k_prefix v_prefix k v out lse lens q_lens", ctypes.c_void_p)
                + _fields("B Tq H Hkv hd P S", ctypes.c_int) + [("scale", ctypes.c_float)]
                + _fields("q_stride out_stride", _I3) + _fields("kp_stride vp_stride", _I2)
                + _fields("k_stride v_stride", _I3))


class WeightsArgs(ctypes.Structure):
    _fields_ = (_fields("q k lse acc out lens q_lens", ctypes.c_void_p) + _fields("B Tq H Hkv hd S", ctypes.c_int)
                + [("scale", ctypes.c_float)] + _fields("q_stride k_stride", _I3))


class EvictArgs(ctypes.Structure):
    _fields_ = (_fields("k v acc pos lens k_out v_out acc_out pos_out lens_out", ctypes.c_void_p)
                + _fields("B Hkv S hd keep recent sinks", ctypes.c_int) + _fields("k_stride v_stride", _I3)
                + _fields("acc_stride pos_stride", _I2) + _fields("k_out_stride v_out_stride", _I3)
                + _fields("acc_out_stride pos_out_stride", _I2))


class VerifyArgs(ctypes.Structure):
    _fields_ = (_fields("logits draft_logits draft u n_draft tokens n_accepted", ctypes.c_void_p)
                + _fields("B D V", ctypes.c_int) + [("temperature", ctypes.c_float)]
                + _fields("logits_stride draft_logits_stride", _I2))


_P = ctypes.c_void_p
_I = ctypes.c_int
_SIG = {
    "flashloop_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(Config)]),
    "flashloop_init": (_I, [ctypes.POINTER(Config), ctypes.POINTER(Weights), _P, ctypes.c_size_t, _P,
                            ctypes.POINTER(_P)]),
    "flashloop_prefill": (_I, [_P, _P, _I, _I, _P, _P, _P]),
    "flashloop_decode_step": (_I, [_P, _P, _I, _P, _P, _P]),
    "flashloop_kv_bytes": (_I, [_P, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_double),
                                ctypes.POINTER(ctypes.c_double)]),
    "flashloop_kv_bytes_for": (_I, [ctypes.POINTER(Config), ctypes.POINTER(ctypes.c_size_t),
                                    ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]),
    "flashloop_reset": (_I, [_P, _P, _P]),
    "flashloop_sync_status": (_I, [_P, _P]),
    "flashloop_destroy": (None, [_P]),
    "flashloop_status_string": (ctypes.c_char_p, [_I]),
    "flashloop_last_cuda_error": (ctypes.c_char_p, [_P]),
    "flashloop_import_lazy": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P]),
    "flashloop_import_dense": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "flashloop_import_extra": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "flashloop_export_slice": (_I, [_P, _I, _I, _I, _I, _I, _P, _P, _P]),
    "flashloop_force_selection": (_I, [_P, _P, _I, _I, _P, _P, _I]),
    "flashloop_read_trace": (_I, [_P, _P, _P, _P, _P, _P]),
    "flashloop_set_trace": (_I, [_P, _P, _I, _P, _I]),
    "flashloop_force_codes": (_I, [_P, _P, _P, _I]),
    "flashloop_set_option": (_I, [_P, _I, _I]),
    "flashloop_profile": (_I, [_P, _P, _P, _P]),
    "flashloop_kernels_per_call": (_I, [_P]),
    "flashloop_gemm_times": (_I, [_P, _P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_I)]),
    "fl_test_topk": (_I, [_P, _I, _I, _I, _P, _P]),
    "fl_test_quantize": (_I, [_P, _I, _I, _I, _I, _P, _P, _P]),
    "fl_test_quantize_residual": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _P]),
    "fl_test_gemm_scratch_bytes": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "fl_test_gemm": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, ctypes.c_size_t, _P]),
    "fl_gemm_skinny_noalloc": (_I, [_P, _P, _P, _I, _I, _I, _P]),
    "flashloop_share_prefix_scratch_bytes": (ctypes.c_size_t, [ctypes.POINTER(Config), _I, _I]),
    "flashloop_share_prefix": (_I, [_P, _I, _I, _P, ctypes.c_size_t]),
    "flashloop_prefix_attention_scratch_bytes": (ctypes.c_size_t, [_I] * 7),
    "flashloop_prefix_attention": (_I, [_P, _P, ctypes.c_size_t, _P]),
    "flashloop_column_weights_scratch_bytes": (ctypes.c_size_t, [_I] * 6),
    "flashloop_column_weights": (_I, [_P, _P, ctypes.c_size_t, _P]),
    "flashloop_evict_scratch_bytes": (ctypes.c_size_t, [_I] * 4),
    "flashloop_evict": (_I, [_P, _P, ctypes.c_size_t, _P]),
    "flashloop_verify_draft_scratch_bytes": (ctypes.c_size_t, [_I] * 3),
    "flashloop_verify_draft": (_I, [_P, _P, ctypes.c_size_t, _P]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise FileNotFoundError(f"{LIB_PATH} is missing: run `python -m cross_loop_sparsity_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIG.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(st: int, what: str, ctx=None):
    if st != FL_OK:
        e = lib().flashloop_last_cuda_error(ctx)
        detail = e.decode() if e else ""
        raise FlashLoopError(st, what, detail)


def make_config(cfg, max_batch: int, max_ctx: int, max_tokens: int = 0, resid_bits: int | None = None) -> Config:
    """Fill the C config from a ``synth.LoopConfig``-like object."""
    return Config(cfg.d_model, cfg.n_heads, cfg.n_kv_heads, cfg.head_dim, cfg.ffn_dim, cfg.n_layers, cfg.n_loops,
                  float(cfg.rho), cfg.c_cols, cfg.q_tile, cfg.resid_bits if resid_bits is None else resid_bits,
                  cfg.group_size, float(cfg.resid_scale), float(cfg.rms_eps), float(cfg.rope_theta), cfg.vocab,
                  max_batch, max_ctx, max_tokens, int(getattr(cfg, "kv_mode", 0)),
                  int(getattr(cfg, "n_prelude", 0)), int(getattr(cfg, "n_coda", 0)),
                  int(getattr(cfg, "loop_embed", 0)), float(getattr(cfg, "inject_scale", 0.0)),
                  int(getattr(cfg, "resid_rows", 0)))


def workspace_bytes(c: Config) -> int:
    return int(lib().flashloop_workspace_bytes(ctypes.byref(c)))


def kv_bytes_for(c: Config):
    tot, per, dense = ctypes.c_size_t(), ctypes.c_double(), ctypes.c_double()
    _check(lib().flashloop_kv_bytes_for(ctypes.byref(c), ctypes.byref(tot), ctypes.byref(per), ctypes.byref(dense)),
           "kv_bytes_for")
    return int(tot.value), per.value, dense.value


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream):
    return None if stream is None else ctypes.c_void_p(stream.cuda_stream)


def upload_weights(w: dict, device="cuda"):
    """Stack the generator's per-layer weights into device tensors (bf16 bits as int16)."""
    import torch

    def stack(layers, name, dt=np.uint16):
        a = np.stack([lw[name] for lw in layers]).astype(dt, copy=False)
        if dt == np.uint16:
            return torch.from_numpy(a.view(np.int16)).to(device)
        return torch.from_numpy(a).to(device)

    def layer_stack(layers):
        return {n: stack(layers, n, np.float32 if n.endswith("norm") else np.uint16) for n in LAYER_FIELDS}

    out = layer_stack(w["layers"])
    out["final_norm"] = torch.from_numpy(np.asarray(w["final_norm"], np.float32)).to(device)
    out["w_out"] = torch.from_numpy(np.asarray(w["w_out"]).view(np.int16)).to(device)
    for part in ("prelude", "coda"):
        if w.get(part):
            out[part] = layer_stack(w[part])
    if "loop_embed" in w:
        out["loop_embed"] = torch.from_numpy(np.asarray(w["loop_embed"], np.float32)).to(device)
    return out


class FlashLoop:
    """One context: a KV cache and the per-call state in a torch-owned workspace."""

    def __init__(self, cfg, dev_weights: dict, max_batch: int, max_ctx: int, max_tokens: int = 0,
                 resid_bits: int | None = None, stream=None):
        import torch
        self.cfg = cfg
        self.c = make_config(cfg, max_batch, max_ctx, max_tokens, resid_bits)
        self.weights = dev_weights  # keep alive: the library borrows these pointers
        nbytes = workspace_bytes(self.c)
        if nbytes == 0:
            raise FlashLoopError(1, "workspace_bytes", "invalid config")
        self.workspace = torch.empty(nbytes + 256, dtype=torch.uint8, device="cuda")
        off = (-self.workspace.data_ptr()) % 256
        self._ws_ptr = self.workspace.data_ptr() + off
        self._ws_bytes = nbytes
        def layers(d):
            return Layers(*[d[n].data_ptr() for n in LAYER_FIELDS]) if d else Layers()

        wt = Weights(*[dev_weights[n].data_ptr() for n in LAYER_FIELDS + ("final_norm", "w_out")],
                     layers(dev_weights.get("prelude")), layers(dev_weights.get("coda")),
                     dev_weights["loop_embed"].data_ptr() if "loop_embed" in dev_weights else None)
        self._wstruct = wt
        ctx = ctypes.c_void_p()
        st = lib().flashloop_init(ctypes.byref(self.c), ctypes.byref(wt), ctypes.c_void_p(self._ws_ptr),
                                  ctypes.c_size_t(nbytes), _stream_ptr(stream), ctypes.byref(ctx))
        _check(st, "flashloop_init")
        self.ctx = ctx
        self.lazy = self.c.resid_bits != 16
        self._share_scratch, self._share_kept = None, []

    def close(self):
        if getattr(self, "ctx", None):
            lib().flashloop_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- calls ---------------------------------------------------------------
    def prefill(self, h0, B: int, T: int, h_out=None, logits=None, stream=None):
        _check(lib().flashloop_prefill(self.ctx, _ptr(h0), B, T, _ptr(h_out), _ptr(logits), _stream_ptr(stream)),
               "flashloop_prefill", self.ctx)

    def decode_step(self, h0, B: int, h_out=None, logits=None, stream=None):
        if self._share_scratch is not None:
            self._share_used(stream)
        _check(lib().flashloop_decode_step(self.ctx, _ptr(h0), B, _ptr(h_out), _ptr(logits), _stream_ptr(stream)),
               "flashloop_decode_step", self.ctx)

    def kv_bytes(self):
        tot, per, dense = ctypes.c_size_t(), ctypes.c_double(), ctypes.c_double()
        _check(lib().flashloop_kv_bytes(self.ctx, ctypes.byref(tot), ctypes.byref(per), ctypes.byref(dense)),
               "flashloop_kv_bytes")
        return int(tot.value), per.value, dense.value

    def reset(self, lens=None, stream=None):
        arr = None
        if lens is not None:
            v = np.zeros(self.c.max_batch, np.int32)
            v[:len(lens)] = np.asarray(lens, np.int32)
            arr = v.ctypes.data_as(ctypes.c_void_p)
            self._lens_keep = v
        _check(lib().flashloop_reset(self.ctx, arr, _stream_ptr(stream)), "flashloop_reset", self.ctx)

    def share_prefix(self, n_seq: int, n: int, stream=None):
        """Sequences 0..n_seq-1 hold the same first n positions: decode steps read them once for
        the batch (``flashloop_share_prefix``).  n = 0 ends it.  ``stream``: the stream of the steps to come, to
        which the scratch belongs; a scratch that another call replaces goes back to torch's allocator when the
        steps issued until then are done, on whatever stream they run.  (One that a captured step uses is kept.)"""
        import torch
        _need_sizes("flashloop_share_prefix", n_seq=n_seq, n=n)
        scratch, nbytes = None, 0
        if n:
            nbytes = int(lib().flashloop_share_prefix_scratch_bytes(ctypes.byref(self.c), n_seq, n))
            with torch.cuda.stream(self._stream_of(stream)):
                scratch = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.workspace.device)
        _check(lib().flashloop_share_prefix(self.ctx, n_seq, n, None if scratch is None else _ptr(scratch), nbytes),
               "flashloop_share_prefix", self.ctx)
        self._share_scratch = scratch   # keep alive: the library borrows it

    def _stream_of(self, stream):
        """The torch stream of a context's call (None: the legacy default stream)."""
        import torch
        return torch.cuda.default_stream(self.workspace.device) if stream is None else stream

    def _share_used(self, stream):
        """A step on ``stream`` writes the scratch of a shared prefix: not to be given out again before it is done."""
        import torch
        if torch.cuda.is_current_stream_capturing():   # replays come at any time
            if not any(t is self._share_scratch for t in self._share_kept):
                self._share_kept.append(self._share_scratch)
        else:
            self._share_scratch.record_stream(self._stream_of(stream))

    def sync_status(self, stream=None) -> int:
        return int(lib().flashloop_sync_status(self.ctx, _stream_ptr(stream)))

    def profile(self, stream=None):
        """{kind: (ms, launches)} of the last call made with FL_OPT_PROFILE on."""
        ms = (ctypes.c_float * len(KINDS))()
        n = (ctypes.c_int * len(KINDS))()
        _check(lib().flashloop_profile(self.ctx, _stream_ptr(stream), ms, n), "flashloop_profile", self.ctx)
        return {k: (float(ms[i]), int(n[i])) for i, k in enumerate(KINDS)}

    def gemm_times(self, stream=None):
        """(summed device ms, launches) of the last call's GEMMs (FL_OPT_GEMM_TIMES on)."""
        ms, n = ctypes.c_double(), ctypes.c_int()
        _check(lib().flashloop_gemm_times(self.ctx, _stream_ptr(stream), ctypes.byref(ms), ctypes.byref(n)),
               "gemm_times", self.ctx)
        return ms.value, n.value

    def kernels_per_call(self) -> int:
        return int(lib().flashloop_kernels_per_call(self.ctx))

    def set_option(self, opt: int, value: int):
        _check(lib().flashloop_set_option(self.ctx, opt, value), "flashloop_set_option")

    # -- cache import / export --------------------------------------------------
    def import_lazy(self, layer, seq, base_k, base_v, codes_k, codes_v, scales_k, scales_v, stream=None):
        n = base_k.shape[1]
        _check(lib().flashloop_import_lazy(self.ctx, layer, seq, n, _ptr(base_k), _ptr(base_v), _ptr(codes_k),
                                           _ptr(codes_v), _ptr(scales_k), _ptr(scales_v), _stream_ptr(stream)),
               "flashloop_import_lazy", self.ctx)

    def import_dense(self, layer, seq, kv_k, kv_v, stream=None):
        n = kv_k.shape[2]
        _check(lib().flashloop_import_dense(self.ctx, layer, seq, n, _ptr(kv_k), _ptr(kv_v), _stream_ptr(stream)),
               "flashloop_import_dense", self.ctx)

    def load_context(self, ctx: dict, dense: bool = False):
        """Import a cache given as host arrays (the layout ``synth.make_context`` /
        ``make_dense_context`` returns) slice by slice, then set the lengths."""
        import torch
        cfg = self.cfg
        lens = ctx["lens"]
        for j in range(cfg.n_layers):
            for b, n in enumerate(lens):
                n = int(n)
                if n == 0:
                    continue
                if dense:
                    kk = torch.from_numpy(np.ascontiguousarray(ctx["kv_k"][j, :, b, :, :n]).view(np.int16)).cuda()
                    vv = torch.from_numpy(np.ascontiguousarray(ctx["kv_v"][j, :, b, :, :n]).view(np.int16)).cuda()
                    self.import_dense(j, b, kk, vv)
                    continue
                a = {}
                for nm in ("k", "v"):
                    a["base_" + nm] = torch.from_numpy(
                        np.ascontiguousarray(ctx["base_" + nm][j, b, :, :n]).view(np.int16)).cuda()
                    a["codes_" + nm] = torch.from_numpy(np.ascontiguousarray(ctx["codes_" + nm][j, :, b, :, :n])).cuda()
                    a["scales_" + nm] = torch.from_numpy(
                        np.ascontiguousarray(ctx["scales_" + nm][j, :, b, :, :n]).view(np.int16)).cuda()
                self.import_lazy(j, b, a["base_k"], a["base_v"], a["codes_k"], a["codes_v"], a["scales_k"],
                                 a["scales_v"])
                torch.cuda.synchronize()   # the import copies read the staged tensors
        if "extra_k" in ctx:             # the prelude / coda layers' one-pass KV
            for x in range(ctx["extra_k"].shape[0]):
                for b, n in enumerate(lens):
                    n = int(n)
                    if n == 0:
                        continue
                    kk = torch.from_numpy(np.ascontiguousarray(ctx["extra_k"][x, b, :, :n]).view(np.int16)).cuda()
                    vv = torch.from_numpy(np.ascontiguousarray(ctx["extra_v"][x, b, :, :n]).view(np.int16)).cuda()
                    _check(lib().flashloop_import_extra(self.ctx, x, b, n, _ptr(kk), _ptr(vv), None),
                           "flashloop_import_extra", self.ctx)
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        self.reset([int(x) for x in lens])
        torch.cuda.synchronize()

    def load_context_device(self, lens, seed=None, dense: bool = False):
        """Import a synthetic context drawn on the device (``synth.context_slices_device``)
        slice by slice, then set the lengths."""
        import torch
        from cross_loop_sparsity_b200 import synth
        for sl in synth.context_slices_device(self.cfg, lens, seed=seed, dense=dense):
            if dense:
                self.import_dense(*sl)
            else:
                self.import_lazy(*sl)
            torch.cuda.synchronize()    # the import copies read the drawn tensors
        self.reset([int(x) for x in lens])
        torch.cuda.synchronize()

    def export_slice(self, layer, loop, seq, which, n, stream=None):
        """Returns (codes, scales) numpy arrays; loop 1 (or dense) returns (bf16 bits [Hkv][n][hd], None)."""
        import torch
        c = self.c
        if not self.lazy or loop == 1:
            out = torch.empty((c.n_kv_heads, n, c.head_dim), dtype=torch.int16, device="cuda")
            _check(lib().flashloop_export_slice(self.ctx, layer, loop, seq, which, n, _ptr(out), None,
                                                _stream_ptr(stream)), "export", self.ctx)
            torch.cuda.synchronize()
            return out.cpu().numpy().view(np.uint16), None
        rb = c.head_dim * c.resid_bits // 8
        codes = torch.empty((c.n_kv_heads, n, rb), dtype=torch.uint8, device="cuda")
        scales = torch.empty((c.n_kv_heads, n, c.head_dim // c.group_size), dtype=torch.int16, device="cuda")
        _check(lib().flashloop_export_slice(self.ctx, layer, loop, seq, which, n, _ptr(codes), _ptr(scales),
                                            _stream_ptr(stream)), "export", self.ctx)
        torch.cuda.synchronize()
        return codes.cpu().numpy(), scales.cpu().numpy().view(np.float16)

    def force_selection(self, sel=None, cols=None, ncols=None, n_tiles: int = 0):
        """sel int32 [K-1][n_sel] and/or cols int32 [M][n_tiles][Hkv][c] with
        ncols [M][n_tiles][Hkv]; a part left None stays free; all None clears."""
        sel_p, n_loops, n_sel = None, 0, 0
        cols_p = ncols_p = None
        keep = []
        if sel is not None:
            sel = np.ascontiguousarray(sel, np.int32)
            keep.append(sel)
            sel_p, n_loops, n_sel = sel.ctypes.data_as(ctypes.c_void_p), sel.shape[0], sel.shape[1]
        if cols is not None:
            cols = np.ascontiguousarray(cols, np.int32)
            ncols = np.ascontiguousarray(ncols, np.int32)
            keep += [cols, ncols]
            cols_p, ncols_p = cols.ctypes.data_as(ctypes.c_void_p), ncols.ctypes.data_as(ctypes.c_void_p)
        self._forced_keep = keep
        _check(lib().flashloop_force_selection(self.ctx, sel_p, n_loops, n_sel, cols_p, ncols_p,
                                               n_tiles if cols is not None else 0),
               "force_selection", self.ctx)

    def force_codes(self, codes=None, scales=None):
        """codes int8 [M][K-1][n_sel][2][Hkv][hd], scales float16 [M][K-1][n_sel][2][Hkv][hd/g]; None clears."""
        if codes is None:
            _check(lib().flashloop_force_codes(self.ctx, None, None, 0), "force_codes")
            return
        codes = np.ascontiguousarray(codes, np.int8)
        scales = np.ascontiguousarray(scales, np.float16).view(np.uint16)
        self._forced_codes_keep = (codes, scales)
        _check(lib().flashloop_force_codes(self.ctx, codes.ctypes.data_as(ctypes.c_void_p),
                                           scales.ctypes.data_as(ctypes.c_void_p), codes.shape[2]),
               "force_codes", self.ctx)

    def set_trace(self, kv_rows=None, n_slots: int = 0, col_keys=None, n_tiles: int = 0):
        """Check buffers (cuda float32 tensors, or None): kv_rows [M][K-1][n_slots][2][Hkv][hd]
        receives the new K/V rows each lazy loop quantised; col_keys [M][n_tiles][Hkv][max_ctx]
        the delta-score keys of every column set the call chose."""
        self._trace_keep = (kv_rows, col_keys)
        _check(lib().flashloop_set_trace(self.ctx, None if kv_rows is None else _ptr(kv_rows), n_slots,
                                         None if col_keys is None else _ptr(col_keys), n_tiles),
               "set_trace", self.ctx)

    def read_trace(self, N: int, n_sel: int, n_tiles: int, stream=None):
        c = self.c
        L = c.n_loops - 1
        sel = np.zeros((L, n_sel), np.int32)
        keys = np.zeros((L, N), np.float32)
        cols = np.zeros((c.n_layers, n_tiles, c.n_kv_heads, c.c_cols), np.int32)
        ncols = np.zeros((c.n_layers, n_tiles, c.n_kv_heads), np.int32)
        _check(lib().flashloop_read_trace(self.ctx, sel.ctypes.data_as(ctypes.c_void_p),
                                          keys.ctypes.data_as(ctypes.c_void_p), cols.ctypes.data_as(ctypes.c_void_p),
                                          ncols.ctypes.data_as(ctypes.c_void_p), _stream_ptr(stream)),
               "read_trace", self.ctx)
        return sel, keys, cols, ncols


# ---------------------------------------------------------------------------- unit entry points
def topk(keys, k: int, stream=None):
    """keys: cuda float32 [n_seg, n]; returns cuda int32 [n_seg, min(k, n)]."""
    import torch
    n_seg, n = keys.shape
    out = torch.empty((n_seg, min(k, n)), dtype=torch.int32, device=keys.device)
    _check(lib().fl_test_topk(_ptr(keys), n_seg, n, k, _ptr(out), _stream_ptr(stream)), "fl_test_topk")
    return out


def quantize(r, g: int, bits: int, stream=None):
    """r: cuda float32 [rows, width]; returns (packed codes uint8, fp16 scale bits int16)."""
    import torch
    rows, width = r.shape
    codes = torch.empty((rows, width * bits // 8), dtype=torch.uint8, device=r.device)
    scales = torch.empty((rows, width // g), dtype=torch.int16, device=r.device)
    _check(lib().fl_test_quantize(_ptr(r), rows, width, g, bits, _ptr(codes), _ptr(scales), _stream_ptr(stream)),
           "fl_test_quantize")
    return codes, scales


def quantize_residual(x, prev, g: int, bits: int, stream=None):
    """x: cuda float32 [rows, width], prev: cuda bf16 (or int16 bits) [rows, width]; quantises
    r = x - prev; returns (packed codes uint8, fp16 scale bits int16)."""
    import torch
    rows, width = x.shape
    codes = torch.empty((rows, width * bits // 8), dtype=torch.uint8, device=x.device)
    scales = torch.empty((rows, width // g), dtype=torch.int16, device=x.device)
    _check(lib().fl_test_quantize_residual(_ptr(x), _ptr(prev), rows, width, g, bits, _ptr(codes), _ptr(scales),
                                           _stream_ptr(stream)), "fl_test_quantize_residual")
    return codes, scales


def gemm(A, B, swap_ab: bool = False, stream=None):
    """D = A @ B.T on the tcgen05 kernel; A [m,k], B [n,k] bf16 (cuda); returns fp32 [m,n]."""
    import torch
    m, k = A.shape
    n = B.shape[0]
    D = torch.empty((m, n), dtype=torch.float32, device=A.device)
    nb = int(lib().fl_test_gemm_scratch_bytes(m, n, k, int(swap_ab)))
    scratch = torch.empty(max(nb, 256) + 256, dtype=torch.uint8, device=A.device)
    sp = scratch.data_ptr() + ((-scratch.data_ptr()) % 256)
    _check(lib().fl_test_gemm(_ptr(A), _ptr(B), _ptr(D), m, n, k, int(swap_ab), ctypes.c_void_p(sp), nb,
                              _stream_ptr(stream)), "fl_test_gemm")
    return D


def gemm_noalloc(A, B, out=None, stream=None):
    """D = A @ B.T (m <= 64) through the entry point that allocates nothing:
    its split-K scratch is an array inside the library.  ``out`` (fp32 [m, n])
    may be given so the call itself allocates nothing on the torch side either."""
    import torch
    m, k = A.shape
    n = B.shape[0]
    D = out if out is not None else torch.empty((m, n), dtype=torch.float32, device=A.device)
    _check(lib().fl_gemm_skinny_noalloc(_ptr(A), _ptr(B), _ptr(D), m, n, k, _stream_ptr(stream)),
           "fl_gemm_skinny_noalloc")
    return D


# ---------------------------------------------------------------------------- serving operators
# Tensors stay where they are and are taken with their strides.  Work goes to
# ``stream``, or to torch's current stream of the tensors' device, so the calls
# may be captured with ``torch.cuda.graph``.  ``scratch`` (a uint8 cuda tensor of
# the *_scratch_bytes figure, 256-byte aligned as torch allocates) is allocated
# per call unless given; a decode loop keeps one.
#
# A call's argument block is its pointers followed by sizes and strides.  The
# second part depends on shapes, strides and types alone: it is checked and built
# once for each of those and kept, so a repeated call only looks it up and adds
# the pointers (a few microseconds of a call that may itself take as few).
_blocks: dict = {}
_MAX_BLOCKS = 4096


def _need(ok: bool, what: str, why: str):
    if not ok:
        raise FlashLoopError(1, what, why)


def _fits(*sizes):
    """Whether the sizes are what the library's ints hold (ctypes would cut them to 32 bits)."""
    return all(-2 ** 31 <= n < 2 ** 31 for n in sizes)


def _need_sizes(what: str, **sizes):
    for name, n in sizes.items():
        _need(_fits(n), what, f"{name} = {n} is out of range")


def _scratch_bytes(what: str, *sizes) -> int:
    return int(getattr(lib(), what + "_scratch_bytes")(*sizes)) if _fits(*sizes) else 0


def _sig(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _check_tensor(what: str, name: str, t, dtype, shape, device: int, contiguous=False):
    if t is None:
        return
    _need(t.dtype == dtype and tuple(t.shape) == tuple(shape), what,
          f"{name} must be {dtype} {list(shape)}, not {t.dtype} {list(t.shape)}")
    _need(t.is_cuda and t.get_device() == device, what, f"{name} must be on cuda device {device}")
    if contiguous:
        _need(t.is_contiguous(), what, f"{name} must be contiguous")
    else:
        _need(t.shape[-1] <= 1 or t.stride(-1) == 1, what, f"{name}'s last dimension must be contiguous")


def _block(key, make):
    """The (bytes after the pointers, scratch bytes) of an argument block, made on first use."""
    got = _blocks.get(key)
    if got is None:
        args, n_ptr, nbytes = make()
        _need(nbytes > 0, key[0], "a size is out of range")
        if len(_blocks) >= _MAX_BLOCKS:
            _blocks.clear()
        got = _blocks[key] = (bytes(args)[8 * n_ptr:], nbytes)
    return got


def _addr(t):
    return 0 if t is None else t.data_ptr()


def _on(stream):
    """Buffers a call allocates belong to the stream it runs on, and are filled there."""
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _run(what: str, fn, ptrs: bytes, block, scratch, stream, device: int):
    import torch
    tail, nbytes = block
    if torch._C._cuda_getDevice() != device:
        with torch.cuda.device(device):
            return _run(what, fn, ptrs, block, scratch, stream, device)
    if scratch is None:
        with _on(stream):
            scratch = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", device))
    elif scratch.get_device() != device or not scratch.is_contiguous():
        raise FlashLoopError(1, what, f"scratch must be contiguous and on cuda device {device}")
    s = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
    st = fn(ptrs + tail, scratch.data_ptr(), scratch.nbytes, s)
    if st != FL_OK:
        _check(st, what)


_ptrs7, _ptrs9, _ptrs10 = (struct.Struct(f"={n}Q").pack for n in (7, 9, 10))


def prefix_attention_scratch_bytes(B, Tq, H, Hkv, hd, P, S) -> int:
    return _scratch_bytes("flashloop_prefix_attention", B, Tq, H, Hkv, hd, P, S)


def prefix_attention(q, k_prefix, v_prefix, k, v, lens, q_lens=None, scale=None, out=None, lse=None, scratch=None,
                     stream=None):
    """Attention of B sequences that share a prefix (``flashloop_prefix_attention``).

    q: bf16 [B, Tq, H, hd], the last ``q_lens[b]`` (default Tq) tokens of each sequence; k_prefix,
    v_prefix: bf16 [Hkv, P, hd], common to all, or None; k, v: bf16 [B, Hkv, S, hd], each
    sequence's own rows after the prefix, ``lens[b]`` of them valid (the queries' own
    included), or None.  scale defaults to hd ** -0.5.  Returns (out bf16 like q, lse fp32
    [B, Tq, H]); rows t >= q_lens[b] of both keep what the given buffers hold (new
    buffers: 0 and -inf)."""
    import torch
    what = "flashloop_prefix_attention"
    _need(q.dim() == 4, what, "q must be [B, Tq, H, hd]")
    if out is None or lse is None:
        with _on(stream):
            if out is None:
                out = torch.zeros(q.shape, dtype=torch.bfloat16, device=q.device)
            if lse is None:
                lse = torch.full(q.shape[:3], -float("inf"), device=q.device)
    dev = q.get_device()

    def make():
        B, Tq, H, hd = q.shape
        own, pre = k if k is not None else v, k_prefix if k_prefix is not None else v_prefix
        _need(own is None or own.dim() == 4, what, "k and v must be [B, Hkv, S, hd]")
        _need(pre is None or pre.dim() == 3, what, "k_prefix and v_prefix must be [Hkv, P, hd]")
        _need(own is not None or pre is not None, what, "neither a prefix nor rows of the sequences' own")
        Hkv = own.shape[1] if own is not None else pre.shape[0]
        S, P = own.shape[2] if own is not None else 0, pre.shape[1] if pre is not None else 0
        _need_sizes(what, B=B, Tq=Tq, H=H, Hkv=Hkv, hd=hd, P=P, S=S)
        bf = torch.bfloat16
        for name, t, dt, shape, contiguous in (
                ("q", q, bf, (B, Tq, H, hd), False), ("out", out, bf, (B, Tq, H, hd), False),
                ("k_prefix", k_prefix, bf, (Hkv, P, hd), False), ("v_prefix", v_prefix, bf, (Hkv, P, hd), False),
                ("k", k, bf, (B, Hkv, S, hd), False), ("v", v, bf, (B, Hkv, S, hd), False),
                ("lse", lse, torch.float32, (B, Tq, H), True), ("lens", lens, torch.int32, (B,), True),
                ("q_lens", q_lens, torch.int32, (B,), True)):
            _check_tensor(what, name, t, dt, shape, dev, contiguous)
        a = PrefixArgs(*[None] * 9, B, Tq, H, Hkv, hd, P, S, hd ** -0.5 if scale is None else scale,
                       _I3(*q.stride()[:3]), _I3(*out.stride()[:3]),
                       _I2(*k_prefix.stride()[:2]) if k_prefix is not None else _I2(),
                       _I2(*v_prefix.stride()[:2]) if v_prefix is not None else _I2(),
                       _I3(*k.stride()[:3]) if k is not None else _I3(),
                       _I3(*v.stride()[:3]) if v is not None else _I3())
        return a, 9, prefix_attention_scratch_bytes(B, Tq, H, Hkv, hd, P, S)

    block = _block((what, scale, _sig(q), _sig(k_prefix), _sig(v_prefix), _sig(k), _sig(v), _sig(out), _sig(lse),
                    _sig(lens), _sig(q_lens)), make)
    _run(what, lib().flashloop_prefix_attention,
         _ptrs9(q.data_ptr(), _addr(k_prefix), _addr(v_prefix), _addr(k), _addr(v), out.data_ptr(), lse.data_ptr(),
                _addr(lens), _addr(q_lens)), block, scratch, stream, dev)
    return out, lse


def column_weights_scratch_bytes(B, Tq, H, Hkv, hd, S) -> int:
    return _scratch_bytes("flashloop_column_weights", B, Tq, H, Hkv, hd, S)


def column_weights(q, k, lse, acc, lens=None, q_lens=None, scale=None, out=None, scratch=None, stream=None):
    """acc plus the attention weight of every key column (``flashloop_column_weights``).

    q: bf16 [B, Tq, H, hd]; k: bf16 [B, Hkv, S, hd]; lse: fp32 [B, Tq, H], as
    ``prefix_attention`` returns it; acc: fp32 [B, Hkv, S].  lens (with q_lens): causal, as there;
    None: every query sees every column.  ``out=acc`` adds in place.  The columns of a
    shared prefix are one sequence of B * Tq queries:
    ``column_weights(q.view(1, B * Tq, H, hd), k_prefix[None], lse.view(1, B * Tq, H), acc_prefix[None])``;
    queries whose lse is -inf add nothing."""
    import torch
    what = "flashloop_column_weights"
    if out is None:
        with _on(stream):
            out = torch.empty(acc.shape, device=acc.device)
    dev = q.get_device()

    def make():
        _need(q.dim() == 4 and k.dim() == 4, what, "q must be [B, Tq, H, hd] and k [B, Hkv, S, hd]")
        _need(q_lens is None or lens is not None, what, "q_lens goes with lens")
        B, Tq, H, hd = q.shape
        Hkv, S = k.shape[1], k.shape[2]
        _need_sizes(what, B=B, Tq=Tq, H=H, Hkv=Hkv, hd=hd, S=S)
        bf, f32 = torch.bfloat16, torch.float32
        for name, t, dt, shape, contiguous in (
                ("q", q, bf, (B, Tq, H, hd), False), ("k", k, bf, (B, Hkv, S, hd), False),
                ("lse", lse, f32, (B, Tq, H), True), ("acc", acc, f32, (B, Hkv, S), True),
                ("out", out, f32, (B, Hkv, S), True), ("lens", lens, torch.int32, (B,), True),
                ("q_lens", q_lens, torch.int32, (B,), True)):
            _check_tensor(what, name, t, dt, shape, dev, contiguous)
        a = WeightsArgs(*[None] * 7, B, Tq, H, Hkv, hd, S, hd ** -0.5 if scale is None else scale,
                        _I3(*q.stride()[:3]), _I3(*k.stride()[:3]))
        return a, 7, column_weights_scratch_bytes(B, Tq, H, Hkv, hd, S)

    block = _block((what, scale, _sig(q), _sig(k), _sig(lse), _sig(acc), _sig(out), _sig(lens), _sig(q_lens)), make)
    _run(what, lib().flashloop_column_weights,
         _ptrs7(q.data_ptr(), k.data_ptr(), lse.data_ptr(), acc.data_ptr(), out.data_ptr(), _addr(lens),
                _addr(q_lens)), block, scratch, stream, dev)
    return out


def evict_scratch_bytes(B, Hkv, S, keep) -> int:
    return _scratch_bytes("flashloop_evict", B, Hkv, S, keep)


def evict(k, v, acc, pos, lens, keep: int, recent: int = 0, sinks: int = 0, out=None, scratch=None, stream=None):
    """Keep the ``keep`` columns of most accumulated weight of every (sequence, KV head) (``flashloop_evict``).

    k, v: [B, Hkv, S, hd] of a 2-byte type; acc: fp32, pos: int32 [B, Hkv, S]; lens: int32 [B].  The
    ``recent`` newest tokens (by pos) and those at pos < ``sinks`` are always kept.  In place,
    or into out = (k, v, acc, pos, lens) with ``keep`` slots per head.  Returns those five."""
    import torch
    what = "flashloop_evict"
    ko, vo, ao, po, lo = (k, v, acc, pos, lens) if out is None else out
    dev = k.get_device()

    def make():
        _need(k.dim() == 4 and k.element_size() == 2, what, "k must be [B, Hkv, S, hd] of a 2-byte type")
        B, Hkv, S, hd = k.shape
        _need_sizes(what, B=B, Hkv=Hkv, S=S, hd=hd, keep=keep, recent=recent, sinks=sinks)
        f32, i32 = torch.float32, torch.int32
        n = S if out is None else keep
        for name, t, dt, shape, contiguous in (
                ("k", k, k.dtype, (B, Hkv, S, hd), False), ("v", v, k.dtype, (B, Hkv, S, hd), False),
                ("acc", acc, f32, (B, Hkv, S), False), ("pos", pos, i32, (B, Hkv, S), False),
                ("lens", lens, i32, (B,), True), ("out k", ko, k.dtype, (B, Hkv, n, hd), False),
                ("out v", vo, k.dtype, (B, Hkv, n, hd), False), ("out acc", ao, f32, (B, Hkv, n), False),
                ("out pos", po, i32, (B, Hkv, n), False), ("out lens", lo, i32, (B,), True)):
            _check_tensor(what, name, t, dt, shape, dev, contiguous)
        a = EvictArgs(*[None] * 10, B, Hkv, S, hd, keep, recent, sinks, _I3(*k.stride()[:3]), _I3(*v.stride()[:3]),
                      _I2(*acc.stride()[:2]), _I2(*pos.stride()[:2]), _I3(*ko.stride()[:3]), _I3(*vo.stride()[:3]),
                      _I2(*ao.stride()[:2]), _I2(*po.stride()[:2]))
        return a, 10, evict_scratch_bytes(B, Hkv, S, keep)

    block = _block((what, keep, recent, sinks, out is None, _sig(k), _sig(v), _sig(acc), _sig(pos), _sig(lens), _sig(ko),
                    _sig(vo), _sig(ao), _sig(po), _sig(lo)), make)
    _run(what, lib().flashloop_evict,
         _ptrs10(k.data_ptr(), v.data_ptr(), acc.data_ptr(), pos.data_ptr(), lens.data_ptr(), ko.data_ptr(),
                 vo.data_ptr(), ao.data_ptr(), po.data_ptr(), lo.data_ptr()), block, scratch, stream, dev)
    return ko, vo, ao, po, lo


def verify_draft_scratch_bytes(B, D, V) -> int:
    return _scratch_bytes("flashloop_verify_draft", B, D, V)


def verify_draft(logits, draft_logits, draft, u, n_draft=None, temperature: float = 1.0, tokens=None, n_accepted=None,
                 scratch=None, stream=None):
    """Verify drafted tokens and sample the next one (``flashloop_verify_draft``).

    logits: fp32 [B, D + 1, V], the target's at every drafted position and after the last;
    draft_logits: fp32 [B, D, V], or None (a draft without probabilities); draft: int32 [B, D]; u: fp32
    [B, D + 1] uniform in [0, 1), the last column for the sampled token (None when greedy);
    n_draft: int32 [B], or None for D; temperature 0: greedy.  Returns (tokens int32
    [B, D + 1], padded with -1; n_accepted int32 [B])."""
    import torch
    what = "flashloop_verify_draft"
    _need(logits.dim() == 3 and logits.shape[1] >= 1, what, "logits must be [B, D + 1, V]")
    if tokens is None or n_accepted is None:
        with _on(stream):
            if tokens is None:
                tokens = torch.empty(logits.shape[:2], dtype=torch.int32, device=logits.device)
            if n_accepted is None:
                n_accepted = torch.empty(logits.shape[:1], dtype=torch.int32, device=logits.device)
    if logits.shape[1] == 1:   # nothing drafted: one token is sampled
        draft = draft_logits = None
    dev = logits.get_device()

    def make():
        B, D, V = logits.shape[0], logits.shape[1] - 1, logits.shape[2]
        _need_sizes(what, B=B, D=D, V=V)
        # (a smaller one may become 0 in 32 bits, and be taken for greedy)
        _need(temperature == 0 or temperature >= 1e-20, what, "temperature must be 0, or finite and at least 1e-20")
        f32, i32 = torch.float32, torch.int32
        for name, t, dt, shape, contiguous in (
                ("logits", logits, f32, (B, D + 1, V), False), ("draft_logits", draft_logits, f32, (B, D, V), False),
                ("draft", draft, i32, (B, D), True), ("u", u, f32, (B, D + 1), True),
                ("n_draft", n_draft, i32, (B,), True), ("tokens", tokens, i32, (B, D + 1), True),
                ("n_accepted", n_accepted, i32, (B,), True)):
            _check_tensor(what, name, t, dt, shape, dev, contiguous)
        a = VerifyArgs(*[None] * 7, B, D, V, temperature, _I2(*logits.stride()[:2]),
                       _I2(*draft_logits.stride()[:2]) if draft_logits is not None else _I2())
        return a, 7, verify_draft_scratch_bytes(B, D, V)

    block = _block((what, temperature, _sig(logits), _sig(draft_logits), _sig(draft), _sig(u), _sig(n_draft),
                    _sig(tokens), _sig(n_accepted)), make)
    _run(what, lib().flashloop_verify_draft,
         _ptrs7(logits.data_ptr(), _addr(draft_logits), _addr(draft), _addr(u), _addr(n_draft), tokens.data_ptr(),
                n_accepted.data_ptr()), block, scratch, stream, dev)
    return tokens, n_accepted
