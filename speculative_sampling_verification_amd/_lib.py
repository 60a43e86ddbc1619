"""ctypes binding to libspecverify.so.

Argument marshalling only: tensors are checked for device, dtype and layout, and their
``data_ptr()`` values and torch's current HIP stream are passed to the C ABI.  Every step of
the computation runs in the library's kernels.  There is no fallback: if the library is
missing the import fails.
"""

from __future__ import annotations

import ctypes
import os
import threading

import torch  # loaded first so that the library binds to torch's HIP runtime

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "libspecverify.so")

SV_OK = 0
SV_ERR_SCRATCH_TOO_SMALL = 5
NOALLOC_SCRATCH_BYTES = 64 << 20  # SPEC_VERIFY_NOALLOC_SCRATCH_BYTES
SV_DTYPE_F32 = 0
SV_DTYPE_BF16 = 1


class SVSampling(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_k", ctypes.c_int32),
                ("top_p", ctypes.c_float), ("lenience", ctypes.c_float),
                ("mentor_kl", ctypes.c_float)]


class SVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("layers", ctypes.c_int32), ("pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("layer_stride", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("seqs", ctypes.c_int32),
                ("table_width", ctypes.c_int32), ("page_table", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("seq_pages", ctypes.c_void_p),
                ("refcount", ctypes.c_void_p)]


EXPORTS = [
    "spec_verify_workspace_size", "spec_verify", "spec_verify_profiled",
    "spec_sample_workspace_size", "spec_sample",
    "spec_verify_tree_workspace_size", "spec_verify_tree", "spec_verify_tree_profiled",
    "spec_build_tree", "spec_philox_uniform", "spec_acceptance_rate", "spec_verify_rates",
    "spec_verify_presampled", "spec_verify_noalloc",
    "spec_tree_attention_workspace_size", "spec_tree_attention", "spec_cache_append",
    "spec_cache_commit", "spec_cache_resize", "spec_cache_fork",
    "spec_expected_tokens",
    "spec_walltime_speedup", "spec_ops_factor", "spec_optimal_gamma",
    "spec_verify_status_string",
]


def load(path=LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with speculative_sampling_verification_amd.build.build()")
    lib = ctypes.CDLL(path)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    psamp = ctypes.POINTER(SVSampling)
    lib.spec_verify_workspace_size.argtypes = [i32, i32, i32, i32, psamp]
    lib.spec_verify_workspace_size.restype = sz
    lib.spec_verify.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp, psamp, vp, vp, vp, vp, vp,
                                vp, sz, vp]
    lib.spec_verify.restype = i32
    lib.spec_verify_profiled.argtypes = lib.spec_verify.argtypes + [vp, i32]
    lib.spec_verify_profiled.restype = i32
    lib.spec_verify_rates.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp, psamp, vp, vp, vp,
                                      vp, vp, vp, vp, sz, vp]
    lib.spec_verify_rates.restype = i32
    lib.spec_verify_presampled.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, psamp, vp, vp, vp,
                                           vp, vp, vp, sz, vp, sz, vp]
    lib.spec_verify_presampled.restype = i32
    lib.spec_verify_noalloc.argtypes = lib.spec_verify.argtypes[:15] + [vp]
    lib.spec_verify_noalloc.restype = i32
    lib.spec_sample_workspace_size.argtypes = [i32, i32, i32, psamp]
    lib.spec_sample_workspace_size.restype = sz
    lib.spec_sample.argtypes = [vp, i32, i32, i32, vp, psamp, vp, vp, sz, vp]
    lib.spec_sample.restype = i32
    lib.spec_verify_tree_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.spec_verify_tree_workspace_size.restype = sz
    lib.spec_verify_tree.argtypes = [vp, i32, i32, i32, i32, vp, vp, i32, vp, vp, vp, vp, sz, vp]
    lib.spec_verify_tree.restype = i32
    lib.spec_verify_tree_profiled.argtypes = lib.spec_verify_tree.argtypes + [vp, i32]
    lib.spec_verify_tree_profiled.restype = i32
    lib.spec_build_tree.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    lib.spec_build_tree.restype = i32
    u64 = ctypes.c_uint64
    lib.spec_philox_uniform.argtypes = [u64, u64, u64, ctypes.c_int64, vp, vp]
    lib.spec_philox_uniform.restype = i32
    lib.spec_acceptance_rate.argtypes = [vp, vp, i32, i32, i32, i32, i32, psamp, vp, vp, sz, vp]
    lib.spec_acceptance_rate.restype = i32
    pcache, f32 = ctypes.POINTER(SVCache), ctypes.c_float
    lib.spec_tree_attention_workspace_size.argtypes = [pcache, i32, i32]
    lib.spec_tree_attention_workspace_size.restype = sz
    lib.spec_tree_attention.argtypes = [vp, vp, i32, i32, pcache, i32, vp, vp, f32, vp, vp, vp,
                                        sz, vp]
    lib.spec_tree_attention.restype = i32
    lib.spec_cache_append.argtypes = [vp, vp, vp, i32, pcache, i32, vp, vp]
    lib.spec_cache_append.restype = i32
    lib.spec_cache_commit.argtypes = [pcache, vp, vp, i32, vp, vp]
    lib.spec_cache_commit.restype = i32
    lib.spec_cache_resize.argtypes = [pcache, vp, vp, vp, vp]
    lib.spec_cache_resize.restype = i32
    lib.spec_cache_fork.argtypes = [pcache, vp, vp, i32, vp, vp]
    lib.spec_cache_fork.restype = i32
    dbl = ctypes.c_double
    lib.spec_expected_tokens.argtypes = [dbl, i32]
    lib.spec_expected_tokens.restype = dbl
    lib.spec_walltime_speedup.argtypes = [dbl, i32, dbl]
    lib.spec_walltime_speedup.restype = dbl
    lib.spec_ops_factor.argtypes = [dbl, i32, dbl]
    lib.spec_ops_factor.restype = dbl
    lib.spec_optimal_gamma.argtypes = [dbl, dbl, i32]
    lib.spec_optimal_gamma.restype = i32
    lib.spec_verify_status_string.argtypes = [i32]
    lib.spec_verify_status_string.restype = ctypes.c_char_p
    return lib


_lib = load()


def lib():
    return _lib


def status_string(code):
    return _lib.spec_verify_status_string(int(code)).decode()


class SpecVerifyError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed: {status_string(code)} (status {code})")
        self.code = code


# Held while a call enqueues its kernels: several of them share a workspace (one per stream), and
# another thread's kernels on the same stream must not come between.
_launches = threading.RLock()


def _launch(name, fn, *args):
    with _launches:
        code = fn(*args)
    if code != SV_OK:
        raise SpecVerifyError(name, code)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return SV_DTYPE_BF16
    if t.dtype == torch.float32:
        return SV_DTYPE_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, name, device, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def sampling(temperature=1.0, top_k=0, top_p=1.0, lenience=1.0, mentor_kl=0.0):
    return SVSampling(float(temperature), int(top_k), float(top_p), float(lenience),
                      float(mentor_kl))


_workspaces = {}
_outgrown = []  # replaced workspaces, kept alive: a captured HIP graph may still use them


def workspace(device, nbytes, stream=None):
    """A cached uint8 device buffer of at least nbytes, one per (device, stream): calls that
    share a workspace must be ordered on one stream.  Grown on demand; a buffer it replaces is
    never freed, so work already captured in a HIP graph keeps valid memory."""
    s = stream if stream is not None else torch.cuda.current_stream(device)
    key = (device.type, device.index, s.cuda_stream)
    with _launches:
        buf = _workspaces.get(key)
        if buf is None or buf.numel() < nbytes:
            if buf is not None:
                _outgrown.append(buf)
            with torch.cuda.stream(s):  # memory whose earlier users are ordered before s's work
                buf = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
            _workspaces[key] = buf
    return buf


def release_workspaces(device=None):
    """Frees the cached workspaces (of one device, or of all) and the outgrown ones kept for
    captured graphs, after the device has finished the work queued on them.  A HIP graph
    captured over calls of this binding must not be replayed afterwards; the next call
    allocates afresh.  Returns the number of bytes released."""
    with _launches:
        return _release(device)


def _release(device):
    freed = 0
    devs = {d for (_, d, _) in _workspaces} | {b.device.index for b in _outgrown}
    for d in devs:
        if device is None or torch.device(device).index in (None, d):
            torch.cuda.synchronize(d)
    keep = {}
    for key, buf in _workspaces.items():
        if device is None or torch.device(device).index in (None, key[1]):
            freed += buf.numel()
        else:
            keep[key] = buf
    _workspaces.clear()
    _workspaces.update(keep)
    rest = []
    for buf in _outgrown:
        if device is None or torch.device(device).index in (None, buf.device.index):
            freed += buf.numel()
        else:
            rest.append(buf)
    _outgrown[:] = rest
    return freed


def _stream(device, stream):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def spec_verify(target_logits, draft_logits, draft_tokens, uniforms, *, temperature=1.0, top_k=0,
                top_p=1.0, lenience=1.0, mentor_kl=0.0, out=None, want_probs=True,
                want_rates=False, presampled=None, stream=None, events=None):
    """Verify-and-resample for a batch (see include/spec_verify.h).

    target_logits [B, K+1, V], draft_logits [B, K or K+1, V] (bf16 or fp32, same dtype),
    draft_tokens [B, K] int32, uniforms [B, K+1] float32, all on one GPU.
    Returns a dict: tokens [B, K+1], num_accepted [B], and if want_probs accept_prob / q_draft /
    p_draft [B, K].  ``out`` may hold preallocated tensors under the same keys.
    ``mentor_kl`` > 0 selects mentored decoding with that KL bound (needs lenience 1 and, for
    temperature > 0, top_k in 1..256).
    ``want_rates``: also return rate [B, K], the acceptance rate sum_x min(p, q/l) of each
    position (spec_verify_rates: the same results plus the rates, one pass over the logits).
    ``presampled``: the ``summary`` buffer of a spec_sample call on draft_logits viewed as
    [B*K, V] with the same sampling parameters (spec_verify_presampled: the draft rows are not
    streamed again; same results).
    ``events``: optional list of >= 2 hipEvent_t handles (ints) for per-phase timing.
    """
    dev = target_logits.device
    B, K1, V = target_logits.shape
    K = K1 - 1
    _need(target_logits, "target_logits", dev)
    dt = _dtype_code(target_logits)
    if K > 0:
        _need(draft_logits, "draft_logits", dev, target_logits.dtype)
        if draft_logits.dim() != 3 or draft_logits.shape[0] != B or draft_logits.shape[2] != V:
            raise ValueError("draft_logits must be [B, K or K+1, V]")
        draft_rows = draft_logits.shape[1]
        _need(draft_tokens, "draft_tokens", dev, torch.int32, (B, K))
    else:
        draft_rows = 0
    _need(uniforms, "uniforms", dev, torch.float32, (B, K + 1))
    out = dict(out or {})
    if "tokens" not in out:
        out["tokens"] = torch.empty((B, K + 1), dtype=torch.int32, device=dev)
    if "num_accepted" not in out:
        out["num_accepted"] = torch.empty((B,), dtype=torch.int32, device=dev)
    if want_probs:
        for k in ("accept_prob", "q_draft", "p_draft"):
            if k not in out:
                out[k] = torch.empty((B, K), dtype=torch.float32, device=dev)
    _need(out["tokens"], "out tokens", dev, torch.int32, (B, K + 1))
    _need(out["num_accepted"], "out num_accepted", dev, torch.int32, (B,))
    for k in ("accept_prob", "q_draft", "p_draft"):
        if k in out:
            _need(out[k], f"out {k}", dev, torch.float32, (B, K))
    if want_rates:
        if events is not None:
            raise ValueError("want_rates and events cannot be combined")
        if "rate" not in out:
            out["rate"] = torch.empty((B, K), dtype=torch.float32, device=dev)
        _need(out["rate"], "out rate", dev, torch.float32, (B, K))
    samp = sampling(temperature, top_k, top_p, lenience, mentor_kl)
    need = _lib.spec_verify_workspace_size(B, K, V, dt, ctypes.byref(samp))
    if need == 0:
        raise SpecVerifyError("spec_verify_workspace_size", 1)
    ws = workspace(dev, need, stream)
    args = [_ptr(target_logits), _ptr(draft_logits) if K > 0 else None, dt, B, K, V, draft_rows,
            _ptr(draft_tokens) if K > 0 else None, _ptr(uniforms), ctypes.byref(samp),
            _ptr(out["tokens"]), _ptr(out["num_accepted"]), _ptr(out.get("accept_prob")),
            _ptr(out.get("q_draft")), _ptr(out.get("p_draft")), _ptr(ws), ws.numel(),
            _stream(dev, stream)]
    if presampled is not None:
        if want_rates or events is not None:
            raise ValueError("presampled cannot be combined with want_rates or events")
        if draft_rows != K:
            raise ValueError("presampled needs draft_logits [B, K, V]")
        _need(presampled, "presampled", dev, torch.uint8)
        _launch("spec_verify_presampled", _lib.spec_verify_presampled, args[0], args[1], dt, B, K,
                V, *args[7:15], _ptr(presampled), presampled.numel(), *args[15:])
    elif want_rates:
        _launch("spec_verify_rates", _lib.spec_verify_rates, *args[:15], _ptr(out["rate"]),
                *args[15:])
    elif events is None:
        _launch("spec_verify", _lib.spec_verify, *args)
    else:
        arr = (ctypes.c_void_p * len(events))(*events)
        _launch("spec_verify_profiled", _lib.spec_verify_profiled, *args, arr, len(events))
    return out


def spec_verify_noalloc(target_logits, draft_logits, draft_tokens, uniforms, out, *,
                        temperature=1.0, top_k=0, top_p=1.0, lenience=1.0, mentor_kl=0.0,
                        stream=None):
    """spec_verify through the entry point that takes no workspace (the library's own scratch
    buffer, one per GPU; see include/spec_verify.h), for callers that cannot allocate.  ``out``
    must hold the output tensors (tokens, num_accepted and optionally accept_prob, q_draft,
    p_draft), so that this call allocates nothing.  Raises SpecVerifyError with status 5 when
    the problem needs more scratch than the buffer holds."""
    dev = target_logits.device
    B, K1, V = target_logits.shape
    K = K1 - 1
    _need(target_logits, "target_logits", dev)
    dt = _dtype_code(target_logits)
    if K > 0:
        _need(draft_logits, "draft_logits", dev, target_logits.dtype)
        if draft_logits.dim() != 3 or draft_logits.shape[0] != B or draft_logits.shape[2] != V:
            raise ValueError("draft_logits must be [B, K or K+1, V]")
        draft_rows = draft_logits.shape[1]
        _need(draft_tokens, "draft_tokens", dev, torch.int32, (B, K))
    else:
        draft_rows = 0
    _need(uniforms, "uniforms", dev, torch.float32, (B, K + 1))
    _need(out["tokens"], "out tokens", dev, torch.int32, (B, K + 1))
    _need(out["num_accepted"], "out num_accepted", dev, torch.int32, (B,))
    for k in ("accept_prob", "q_draft", "p_draft"):
        if k in out:
            _need(out[k], f"out {k}", dev, torch.float32, (B, K))
    samp = sampling(temperature, top_k, top_p, lenience, mentor_kl)
    _launch("spec_verify_noalloc", _lib.spec_verify_noalloc, _ptr(target_logits),
            _ptr(draft_logits) if K > 0 else None, dt, B, K, V, draft_rows,
            _ptr(draft_tokens) if K > 0 else None, _ptr(uniforms), ctypes.byref(samp),
            _ptr(out["tokens"]), _ptr(out["num_accepted"]), _ptr(out.get("accept_prob")),
            _ptr(out.get("q_draft")), _ptr(out.get("p_draft")), _stream(dev, stream))
    return out


def sample_summary(R, V, dtype, *, temperature=1.0, top_k=0, top_p=1.0, device=None):
    """A device buffer for spec_sample(summary=...) over R rows of V logits of torch dtype
    ``dtype``: it keeps the rows' summaries for spec_verify(presampled=...)."""
    dt = _dtype_code(torch.empty(0, dtype=dtype))
    samp = sampling(temperature, top_k, top_p, 1.0)
    need = _lib.spec_sample_workspace_size(R, V, dt, ctypes.byref(samp))
    if need == 0:
        raise SpecVerifyError("spec_sample_workspace_size", 1)
    return torch.empty(need, dtype=torch.uint8,
                       device=device if device is not None else torch.device("cuda"))


def spec_sample(logits, uniforms, *, temperature=1.0, top_k=0, top_p=1.0, out=None,
                summary=None, stream=None):
    """One token per row of logits [R, V] from its processed distribution; uniforms [R].
    ``summary``: a buffer from sample_summary; the rows' summaries are kept there (instead of
    the stream's shared workspace) for a later spec_verify(presampled=summary)."""
    dev = logits.device
    R, V = logits.shape
    _need(logits, "logits", dev)
    dt = _dtype_code(logits)
    _need(uniforms, "uniforms", dev, torch.float32, (R,))
    if out is None:
        out = torch.empty((R,), dtype=torch.int32, device=dev)
    _need(out, "out", dev, torch.int32, (R,))
    samp = sampling(temperature, top_k, top_p, 1.0)
    need = _lib.spec_sample_workspace_size(R, V, dt, ctypes.byref(samp))
    if need == 0:
        raise SpecVerifyError("spec_sample_workspace_size", 1)
    if summary is not None:
        _need(summary, "summary", dev, torch.uint8)
        ws = summary
    else:
        ws = workspace(dev, need, stream)
    _launch("spec_sample", _lib.spec_sample, _ptr(logits), dt, R, V, _ptr(uniforms),
            ctypes.byref(samp), _ptr(out), _ptr(ws), ws.numel(), _stream(dev, stream))
    return out


def spec_verify_tree(target_logits, parent, node_tokens, max_depth, *, out=None, stream=None,
                     events=None):
    """Greedy tree verification: target_logits [B, N, V], parent / node_tokens [B, N] int32.

    ``events``: optional list of >= 2 hipEvent_t handles (ints) for per-phase timing.
    """
    dev = target_logits.device
    B, N, V = target_logits.shape
    _need(target_logits, "target_logits", dev)
    dt = _dtype_code(target_logits)
    _need(parent, "parent", dev, torch.int32, (B, N))
    _need(node_tokens, "node_tokens", dev, torch.int32, (B, N))
    out = dict(out or {})
    out.setdefault("tokens", torch.empty((B, max_depth + 1), dtype=torch.int32, device=dev))
    out.setdefault("num_accepted", torch.empty((B,), dtype=torch.int32, device=dev))
    out.setdefault("last_node", torch.empty((B,), dtype=torch.int32, device=dev))
    _need(out["tokens"], "out tokens", dev, torch.int32, (B, max_depth + 1))
    _need(out["num_accepted"], "out num_accepted", dev, torch.int32, (B,))
    _need(out["last_node"], "out last_node", dev, torch.int32, (B,))
    need = _lib.spec_verify_tree_workspace_size(B, N, V, dt)
    if need == 0:
        raise SpecVerifyError("spec_verify_tree_workspace_size", 1)
    ws = workspace(dev, need, stream)
    args = (_ptr(target_logits), dt, B, N, V, _ptr(parent), _ptr(node_tokens), int(max_depth),
            _ptr(out["tokens"]), _ptr(out["num_accepted"]), _ptr(out["last_node"]), _ptr(ws),
            ws.numel(), _stream(dev, stream))
    if events is None:
        _launch("spec_verify_tree", _lib.spec_verify_tree, *args)
    else:
        arr = (ctypes.c_void_p * len(events))(*events)
        _launch("spec_verify_tree_profiled", _lib.spec_verify_tree_profiled, *args, arr,
                len(events))
    return out


def spec_build_tree(candidates, N, *, want_mask=True, out=None, stream=None):
    """REST draft tree from candidates [B, M, L] int32 (a candidate ends at its first negative
    entry): returns parent, tokens, depth, weight [B, N], num_nodes [B] and, if want_mask,
    mask [B, N, N] uint8 (see include/spec_verify.h)."""
    dev = candidates.device
    _need(candidates, "candidates", dev, torch.int32)
    if candidates.dim() != 3:
        raise ValueError("candidates must be [B, M, L]")
    B, M, L = candidates.shape
    out = dict(out or {})
    for k in ("parent", "tokens", "depth", "weight"):
        out.setdefault(k, torch.empty((B, N), dtype=torch.int32, device=dev))
        _need(out[k], f"out {k}", dev, torch.int32, (B, N))
    out.setdefault("num_nodes", torch.empty((B,), dtype=torch.int32, device=dev))
    _need(out["num_nodes"], "out num_nodes", dev, torch.int32, (B,))
    if want_mask:
        out.setdefault("mask", torch.empty((B, N, N), dtype=torch.uint8, device=dev))
        _need(out["mask"], "out mask", dev, torch.uint8, (B, N, N))
    _launch("spec_build_tree", _lib.spec_build_tree, _ptr(candidates), B, M, L, int(N),
            _ptr(out["parent"]), _ptr(out["tokens"]), _ptr(out["num_nodes"]), _ptr(out["depth"]),
            _ptr(out["weight"]), _ptr(out.get("mask")), _stream(dev, stream))
    return out


def spec_philox_uniform(key, counter, n, *, device=None, out=None, stream=None):
    """n float32 uniforms of the Philox4x64-10 stream (key = (k0, k1), 64-bit start counter)
    generated on the GPU (see include/spec_verify.h)."""
    if out is None:
        out = torch.empty((int(n),), dtype=torch.float32, device=device or "cuda")
    dev = out.device
    _need(out, "out", dev, torch.float32)
    if out.numel() < n:
        raise ValueError("out is too small")
    k0, k1 = (int(k) & (2**64 - 1) for k in key)
    _launch("spec_philox_uniform", _lib.spec_philox_uniform, k0, k1, int(counter) & (2**64 - 1),
            int(n), _ptr(out) if n else None, _stream(dev, stream))
    return out


def spec_acceptance_rate(target_logits, draft_logits, *, temperature=1.0, top_k=0, top_p=1.0,
                         lenience=1.0, out=None, stream=None):
    """beta [B, K] = sum_x min(p(x), q(x) / l) per draft position (see include/spec_verify.h)."""
    dev = target_logits.device
    B, K1, V = target_logits.shape
    K = K1 - 1
    _need(target_logits, "target_logits", dev)
    dt = _dtype_code(target_logits)
    _need(draft_logits, "draft_logits", dev, target_logits.dtype)
    if draft_logits.dim() != 3 or draft_logits.shape[0] != B or draft_logits.shape[2] != V:
        raise ValueError("draft_logits must be [B, K or K+1, V]")
    if out is None:
        out = torch.empty((B, K), dtype=torch.float32, device=dev)
    _need(out, "out", dev, torch.float32, (B, K))
    samp = sampling(temperature, top_k, top_p, lenience)
    need = _lib.spec_verify_workspace_size(B, K, V, dt, ctypes.byref(samp))
    if need == 0:
        raise SpecVerifyError("spec_verify_workspace_size", 1)
    ws = workspace(dev, need, stream)
    _launch("spec_acceptance_rate", _lib.spec_acceptance_rate, _ptr(target_logits),
            _ptr(draft_logits), dt, B, K, V, draft_logits.shape[1], ctypes.byref(samp), _ptr(out),
            _ptr(ws), ws.numel(), _stream(dev, stream))
    return out


class PagedCache:
    """A paged key/value cache (sv_cache of include/spec_verify.h): the caller's tensors, checked
    once and kept (their contents change, the tensors do not).

    k, v        [layers, pages, page_size, kv_heads, head_dim], or without the layers; bf16 or
                fp32, any strides with rows on 16 bytes and apart (both tensors alike)
    page_table  [seqs, width] int32
    seq_lens    [seqs] int32, committed tokens
    seq_pages, refcount   [seqs], [pages] int32: needed by spec_cache_resize and spec_cache_fork;
                with them the other calls leave alone what another sequence holds by now
    """

    _FIXED = frozenset(("k", "v", "page_table", "seq_lens", "seq_pages", "refcount", "device", "dtype",
                        "layers", "pages", "page_size", "kv_heads", "head_dim", "seqs"))

    def __init__(self, k, v, page_table, seq_lens, *, seq_pages=None, refcount=None):
        dev = k.device
        if k.dim() == 4:
            k, v = k.unsqueeze(0), v.unsqueeze(0)
        if k.dim() != 5:
            raise ValueError("k must be [layers, pages, page_size, kv_heads, head_dim]")
        if v.device != dev or v.dtype != k.dtype or v.shape != k.shape:
            raise ValueError("k and v must agree in device, dtype and shape")
        strides = k.stride()
        if any(n > 1 and x != y for n, x, y in zip(k.shape, strides, v.stride())):
            raise ValueError("k and v must have the same strides")
        if k.shape[4] > 1 and strides[4] != 1:
            raise ValueError("head_dim must be contiguous")
        if page_table.dim() != 2:
            raise ValueError("page_table must be [seqs, width]")
        seqs, width = page_table.shape
        _need(page_table, "page_table", dev, torch.int32)
        _need(seq_lens, "seq_lens", dev, torch.int32, (seqs,))
        if seq_pages is not None:
            _need(seq_pages, "seq_pages", dev, torch.int32, (seqs,))
        if refcount is not None:
            _need(refcount, "refcount", dev, torch.int32, (k.shape[1],))
        self.k, self.v, self.page_table, self.seq_lens = k, v, page_table, seq_lens
        self.seq_pages, self.refcount = seq_pages, refcount
        self.device, self.dtype = dev, k.dtype
        self.layers, self.pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        self.seqs = seqs
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self._c = SVCache(ptr(k), ptr(v), _dtype_code(k), *k.shape, *strides[:4], seqs, width,
                          ptr(page_table), ptr(seq_lens), ptr(seq_pages), ptr(refcount))
        self._ref = ctypes.byref(self._c)
        self._index = dev.index
        self._workspace_bytes = {}

    def __setattr__(self, name, value):
        # the addresses are taken once: another tensor in an attribute's place would be ignored
        if name in self._FIXED and self.__dict__.get(name, value) is not value:
            raise AttributeError(f"{name} is fixed: change the tensor in place, or make another "
                                 "PagedCache")
        object.__setattr__(self, name, value)

    def _attention_workspace(self, N, q_heads):
        need = self._workspace_bytes.get((N, q_heads))
        if need is None:
            need = _lib.spec_tree_attention_workspace_size(self._ref, N, q_heads)
            if need == 0:
                raise SpecVerifyError("spec_tree_attention_workspace_size", 1)
            self._workspace_bytes[(N, q_heads)] = need
        return need


def _new_like(t, stream):
    """An output tensor with a dense tensor's shape and type, of the stream that will write it."""
    if stream is None:
        return torch.empty_like(t)
    with torch.cuda.stream(stream):
        return torch.empty_like(t)


def _arg(t, name, cache, dtype, shape):
    """The address of an optional contiguous tensor argument on the cache's device."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.device == cache.device and t.is_contiguous()):
        _need(t, name, cache.device, dtype, shape)  # says what is wrong
    return t.data_ptr()


def _raw_stream(cache, stream):
    """The handle of the stream to launch on.  The lookup behind torch.cuda.current_stream, as
    these calls are short enough for a Stream object to show."""
    if cache._index is None:
        raise ValueError(f"the cache is on {cache.device}, expected a GPU")
    if stream is not None:
        if stream.device != cache.device:
            raise ValueError(f"the stream is on {stream.device}, the cache on {cache.device}")
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(cache._index)


def _capturing(cache):
    """Whether the cache's device's current stream is being captured into a graph."""
    if torch._C._cuda_getDevice() == cache._index:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.device(cache._index):
        return torch.cuda.is_current_stream_capturing()


def _cache_call(cache, name, fn, *args):
    """Calls fn with the cache's device current (a null stream is that device's)."""
    if torch._C._cuda_getDevice() == cache._index:
        _launch(name, fn, *args)
    else:
        with torch.cuda.device(cache._index):
            _launch(name, fn, *args)


def _row_strides(t, name, cache, heads):
    """The element strides of a [seqs, N, heads, head_dim] tensor, None where it is dense."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != cache.device:
        raise ValueError(f"{name} is on {t.device}, expected {cache.device}")
    if t.dtype is not cache.dtype:
        raise TypeError(f"{name} must be {cache.dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 4 or shape[0] != cache.seqs or shape[3] != cache.head_dim or (
            heads is not None and shape[2] != heads):
        raise ValueError(f"{name} must be [{cache.seqs}, N, {heads or 'heads'}, "
                         f"{cache.head_dim}], got {tuple(shape)}")
    if t.is_contiguous():
        return None
    s = t.stride()
    if s[3] != 1:
        raise ValueError(f"{name}'s head_dim must be contiguous")
    return (ctypes.c_int64 * 3)(*(x if n > 1 else 0 for n, x in zip(shape, s[:3])))


def spec_tree_attention(q, cache, *, layer=0, mask=None, num_nodes=None, scale=None,
                        want_lse=False, out=None, stream=None):
    """Attention of drafted nodes over a PagedCache's committed tokens and the nodes each may see
    (see include/spec_verify.h).

    q [seqs, N, q_heads, head_dim] of the cache's dtype (strided views with contiguous head_dim
    are taken as they are); node i's own key lies at position seq_lens + i (spec_cache_append).
    mask [seqs, N, N] uint8 as spec_build_tree makes it, or None for a chain (and for N = 1,
    plain decoding); num_nodes [seqs] int32 or None; scale defaults to head_dim ** -0.5.
    Returns a dict: out (like q, dense) and, if want_lse, lse [seqs, N, q_heads] float32.
    ``out`` may hold preallocated tensors under the same keys.
    """
    if stream is not None:
        _raw_stream(cache, stream)  # refuses a stream of another device
        with torch.cuda.stream(stream):
            return spec_tree_attention(q, cache, layer=layer, mask=mask, num_nodes=num_nodes,
                                       scale=scale, want_lse=want_lse, out=out)
    strides = _row_strides(q, "q", cache, None)
    shape = q.shape
    B, N, H, D = shape
    dev = cache.device
    mask_at = _arg(mask, "mask", cache, torch.uint8, (B, N, N))
    nodes_at = _arg(num_nodes, "num_nodes", cache, torch.int32, (B,))
    out = dict(out) if out else {}
    if "out" not in out:
        out["out"] = torch.empty_like(q) if strides is None else torch.empty(
            shape, dtype=q.dtype, device=dev)
    if want_lse and "lse" not in out:
        out["lse"] = torch.empty((B, N, H), dtype=torch.float32, device=dev)
    out_at = _arg(out["out"], "out out", cache, q.dtype, shape)
    lse_at = _arg(out.get("lse"), "out lse", cache, torch.float32, (B, N, H))
    need = cache._attention_workspace(N, H)
    raw = _raw_stream(cache, None)
    if _capturing(cache):  # the graph's own: graphs may run side by side
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        ws = _workspaces.get((dev.type, cache._index, raw))
        if ws is None or ws.numel() < need:
            ws = workspace(dev, need)
    _cache_call(cache, "spec_tree_attention", _lib.spec_tree_attention, q.data_ptr(), strides, N,
                H, cache._ref, layer, mask_at, nodes_at, D ** -0.5 if scale is None else scale,
                out_at, lse_at, ws.data_ptr(), ws.numel(), raw)
    return out


def spec_cache_append(k_new, v_new, cache, *, layer=0, num_nodes=None, stream=None):
    """Writes k_new, v_new [seqs, N, kv_heads, head_dim] of each sequence's nodes to positions
    seq_lens + 0 .. num_nodes - 1 of one layer (see include/spec_verify.h).  Both tensors may be
    strided views, with the same strides."""
    strides = _row_strides(k_new, "k_new", cache, cache.kv_heads)
    v_strides = _row_strides(v_new, "v_new", cache, cache.kv_heads)
    if k_new.shape != v_new.shape:
        raise ValueError("k_new and v_new must have the same shape")
    if strides is not v_strides and (strides is None or v_strides is None
                                     or list(strides) != list(v_strides)):
        raise ValueError("k_new and v_new must have the same strides")
    nodes_at = _arg(num_nodes, "num_nodes", cache, torch.int32, (cache.seqs,))
    _cache_call(cache, "spec_cache_append", _lib.spec_cache_append, k_new.data_ptr(),
                v_new.data_ptr(), strides, k_new.shape[1], cache._ref, layer, nodes_at,
                _raw_stream(cache, stream))


def spec_cache_commit(cache, last_node, *, parent=None, num_nodes=None, out=None, stream=None):
    """Moves the rows of each sequence's accepted path together in every layer and returns the
    new lengths [seqs] int32 (see include/spec_verify.h); seq_lens itself stays until
    spec_cache_resize(new_lens=...) stores it.

    last_node [seqs] int32: spec_verify_tree's last_node with its parent [seqs, N]; without
    parent (a chain of num_nodes nodes, default 2048) spec_verify's num_accepted."""
    seqs = (cache.seqs,)
    last_at = _arg(last_node, "last_node", cache, torch.int32, seqs)
    if last_at is None:
        raise TypeError("last_node must be a torch.Tensor")
    if parent is not None:
        N = parent.shape[-1] if isinstance(parent, torch.Tensor) else 0
        parent_at = _arg(parent, "parent", cache, torch.int32, (cache.seqs, N))
    else:
        N = 2048 if num_nodes is None else int(num_nodes)
        parent_at = None
    if out is None:
        out = _new_like(last_node, stream)
    _cache_call(cache, "spec_cache_commit", _lib.spec_cache_commit, cache._ref, last_at,
                parent_at, N, _arg(out, "out", cache, torch.int32, seqs),
                _raw_stream(cache, stream))
    return out


def spec_cache_resize(cache, want, *, new_lens=None, out=None, stream=None):
    """Gives back and takes pages so that each sequence holds those of want [seqs] int32 tokens
    (< 0: left alone, 0: freed); new_lens [seqs] int32 is stored to seq_lens first.  Returns ok
    [seqs] int32 (see include/spec_verify.h)."""
    seqs = (cache.seqs,)
    want_at = _arg(want, "want", cache, torch.int32, seqs)
    lens_at = _arg(new_lens, "new_lens", cache, torch.int32, seqs)
    if out is None:
        out = _new_like(want, stream)
    _cache_call(cache, "spec_cache_resize", _lib.spec_cache_resize, cache._ref, want_at, lens_at,
                _arg(out, "out", cache, torch.int32, seqs), _raw_stream(cache, stream))
    return out


def spec_cache_fork(cache, src, dst, *, out=None, stream=None):
    """Continues sequences src [F] int32 as the empty sequences dst [F] int32: full pages shared,
    a begun page copied in every layer.  Returns ok [F] int32 (see include/spec_verify.h)."""
    if not isinstance(src, torch.Tensor):
        raise TypeError("src must be a torch.Tensor")
    if src.dim() != 1:
        raise ValueError("src must be [F]")
    F = src.shape
    src_at = _arg(src, "src", cache, torch.int32, F)
    dst_at = _arg(dst, "dst", cache, torch.int32, F)
    if out is None:
        out = _new_like(src, stream)
    _cache_call(cache, "spec_cache_fork", _lib.spec_cache_fork, cache._ref, src_at, dst_at, F[0],
                _arg(out, "out", cache, torch.int32, F), _raw_stream(cache, stream))
    return out


def expected_tokens(alpha, gamma):
    return _lib.spec_expected_tokens(float(alpha), int(gamma))


def walltime_speedup(alpha, gamma, c):
    return _lib.spec_walltime_speedup(float(alpha), int(gamma), float(c))


def ops_factor(alpha, gamma, c_hat):
    return _lib.spec_ops_factor(float(alpha), int(gamma), float(c_hat))


def optimal_gamma(alpha, c, max_gamma):
    return _lib.spec_optimal_gamma(float(alpha), float(c), int(max_gamma))
