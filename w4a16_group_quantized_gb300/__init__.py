"""Thin Python binding of libw4a16.so (the C ABI in include/w4a16.h).

Argument marshalling only: every step of the quantized linear layer runs in
the library's CUDA kernels. PyTorch supplies device memory and the current
stream. There is no CPU or PyTorch fallback: if the library is missing or a
call fails, a ``W4Error`` is raised.

Names follow the C ABI:

    qw, scales, zeros = w4_pack(W, g)                 # fp16 [N,K] cuda -> canonical packed form
    packed = w4_repack(qw, scales, zeros, N, K, g)    # -> the GEMM's tile layout (uint8 buffer)
    y = w4a16_gemm(x, packed, N, K, g)                # fp16 [M,K] -> fp16 [M,N]

uint32 words are carried in torch.int32 tensors (same bits).
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading

import torch

__all__ = [
    "W4Error", "lib_path", "load", "w4_pack", "w4_repack", "w4_repacked_bytes", "w4a16_gemm",
    "w4a16_gemm_ex", "w4a16_gemm_opts", "w4a16_workspace_bytes", "w4a16_workspace_bytes_ex",
    "w4a16_workspace_bytes_opts", "w4a16_gemm_plan", "w4_last_device_error", "w4_status_string", "Workspace",
    "Options", "STATUS", "KERNEL_DECODE", "KERNEL_TMEM", "FLAG_WEIGHTS_STATIC", "FLAG_TEST_TIMEOUT",
    "Epilogue", "Problem", "EPI_NONE", "EPI_SILU_MUL", "EPI_QKV_SPLIT", "w4a16_gemm_grouped",
    "w4a16_grouped_workspace_bytes", "w4a16_gemm_silu_mul", "w4a16_gemm_qkv", "interleave_gate_up",
    "qkv_head_group_rows", "w4_route", "w4a16_experts", "w4a16_experts_workspace_bytes", "w4_lora_add",
    "w4_lora_workspace_bytes", "w4_qk_norm_rope", "w4_kv_append", "w4_kv_attention", "w4_kv_attention_workspace_bytes",
    "w4_prompt_attention", "w4_prompt_attention_workspace_bytes",
]

KERNEL_DECODE = 1
KERNEL_TMEM = 2
FLAG_WEIGHTS_STATIC = 1
FLAG_TEST_TIMEOUT = 2


class Options(ctypes.Structure):
    """w4a16_options of the C ABI (all zero: automatic)."""

    _fields_ = [("kernel", ctypes.c_int32), ("block_n", ctypes.c_int32), ("ctas", ctypes.c_int32),
                ("schedule", ctypes.c_int32), ("cluster", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("wait_limit_cycles", ctypes.c_uint64), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]

EPI_NONE, EPI_SILU_MUL, EPI_QKV_SPLIT = 0, 1, 2


class Epilogue(ctypes.Structure):
    """w4a16_epilogue of the C ABI."""

    _fields_ = [("kind", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("q_per_group", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("k_dev", ctypes.c_void_p), ("v_dev", ctypes.c_void_p)]


class Problem(ctypes.Structure):
    """w4a16_problem of the C ABI."""

    _fields_ = [("x_dev", ctypes.c_void_p), ("packed_dev", ctypes.c_void_p), ("y_dev", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("epilogue", Epilogue)]


_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libw4a16.so")

STATUS = {
    0: "W4_OK", 1: "W4_ERR_INVALID_ARG", 2: "W4_ERR_UNSUPPORTED_SHAPE", 3: "W4_ERR_MISALIGNED",
    4: "W4_ERR_WORKSPACE_TOO_SMALL", 5: "W4_ERR_CUDA", 6: "W4_ERR_TIMEOUT",
}

_lib = None
_lock = threading.Lock()


class W4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {w4_status_string(status)} ({status})")


def load() -> ctypes.CDLL:
    """Load libw4a16.so (built by ``python -m w4a16_group_quantized_gb300.build``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(lib_path):
            raise ImportError(f"{lib_path} is missing: build it with `python -m w4a16_group_quantized_gb300.build`")
        lib = ctypes.CDLL(lib_path)
        P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        sigs = {
            "w4_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "w4_pack": ([P, I64, I64, I32, P, P, P, P], ctypes.c_int),
            "w4_pack_ex": ([P, I64, I64, I32, I32, I32, P, P, P, P], ctypes.c_int),
            "w4_repacked_bytes": ([I64, I64, I32], SZ),
            "w4_repack": ([P, P, P, I64, I64, I32, P, P], ctypes.c_int),
            "w4a16_workspace_bytes": ([I64, I64, I64, I32], SZ),
            "w4a16_workspace_bytes_ex": ([I64, I64, I64, I32, I32, I32, I32], SZ),
            "w4a16_gemm": ([P, P, I64, I64, I64, I32, P, P, SZ, P], ctypes.c_int),
            "w4a16_gemm_ex": ([P, P, I64, I64, I64, I32, P, P, SZ, I32, I32, I32, P], ctypes.c_int),
            "w4a16_gemm_plan": ([I64, I64, I64, I32, ctypes.POINTER(I32), ctypes.POINTER(I32),
                                 ctypes.POINTER(I32)], ctypes.c_int),
            "w4_last_device_error": ([P, P], ctypes.c_int),
            "w4a16_gemm_opts": ([P, P, I64, I64, I64, I32, P, P, SZ, ctypes.POINTER(Options), P], ctypes.c_int),
            "w4a16_workspace_bytes_opts": ([I64, I64, I64, I32, ctypes.POINTER(Options)], SZ),
            "w4a16_gemm_grouped": ([ctypes.POINTER(Problem), I32, I64, I32, P, SZ, ctypes.POINTER(Options), P],
                                   ctypes.c_int),
            "w4a16_grouped_workspace_bytes": ([ctypes.POINTER(Problem), I32, I64, I32, ctypes.POINTER(Options)], SZ),
            "w4_route": ([P, I64, I32, I64, P, ctypes.c_char_p, P, P, P], ctypes.c_int),
            "w4a16_experts": ([ctypes.c_char_p, P, SZ, P], ctypes.c_int),
            "w4a16_experts_opts": ([ctypes.c_char_p, P, SZ, ctypes.POINTER(Options), P], ctypes.c_int),
            "w4a16_experts_workspace_bytes": ([I64, I64, I64, I32, I32, I32], SZ),
            "w4_lora_add": ([ctypes.c_char_p, P, SZ, P], ctypes.c_int),
            "w4_lora_workspace_bytes": ([I64, I64, I64, I32, I32], SZ),
            "w4_qk_norm_rope": ([ctypes.c_char_p, P], ctypes.c_int),
            "w4_kv_append": ([ctypes.c_char_p, P], ctypes.c_int),
            "w4_kv_attention": ([ctypes.c_char_p, P, SZ, P], ctypes.c_int),
            "w4_kv_attention_workspace_bytes": ([I32, I32, I32, I32, I32], SZ),
            "w4_prompt_attention": ([ctypes.c_char_p, P, SZ, P], ctypes.c_int),
            "w4_prompt_attention_opts": ([ctypes.c_char_p, P, SZ, ctypes.POINTER(Options), P], ctypes.c_int),
            "w4_prompt_attention_workspace_bytes": ([I64, I32, I32], SZ),
        }
        for name, (args, res) in sigs.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def w4_status_string(status: int) -> str:
    return load().w4_status_string(int(status)).decode()


def _check(rc: int, what: str):
    if rc != 0:
        raise W4Error(rc, what)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t: torch.Tensor, name: str) -> ctypes.c_void_p:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """What a call makes for its caller, in the memory of the stream that the call runs on: a block that another stream is not
    done with would be written too early. The caller's stream may use it too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _ngroups(K: int, g: int) -> int:
    return -(-K // g)


_DTYPES = {torch.float16: 0, torch.bfloat16: 1}


def w4_pack(W: torch.Tensor, g: int, stream=None, symmetric: bool = False):
    """fp16 or bf16 W [N,K] (cuda) -> (qw int32 [N,ceil(K/8)], scales [N,G] of W's dtype,
    zeros int32 [N,ceil(G/8)]). symmetric: z = 8 and the range +-max|w| (w4_pack_ex)."""
    if W.dtype not in _DTYPES or W.dim() != 2:
        raise ValueError("W must be a 2-D fp16 or bf16 tensor")
    N, K = W.shape
    G = _ngroups(K, g) if g > 0 else 1
    qw = _empty((N, -(-K // 8)), torch.int32, W.device, stream)
    scales = _empty((N, G), W.dtype, W.device, stream)
    zeros = _empty((N, -(-G // 8)), torch.int32, W.device, stream)
    _check(load().w4_pack_ex(_dev(W, "W"), N, K, g, _DTYPES[W.dtype], int(bool(symmetric)), _dev(qw, "qw"),
                             _dev(scales, "scales"), _dev(zeros, "zeros"), _stream(stream)), "w4_pack")
    return qw, scales, zeros


def w4_repacked_bytes(N: int, K: int, g: int) -> int:
    return int(load().w4_repacked_bytes(N, K, g))


def w4_repack(qw: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, N: int, K: int, g: int,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Canonical packed form -> uint8 buffer in the GEMM's tile layout."""
    nbytes = w4_repacked_bytes(N, K, g)
    if nbytes == 0:
        raise W4Error(1, "w4_repack")
    if out is None:
        out = _empty(nbytes, torch.uint8, qw.device, stream)
    elif out.numel() * out.element_size() < nbytes:
        raise ValueError("out is too small")
    _check(load().w4_repack(_dev(qw, "qw"), _dev(scales, "scales"), _dev(zeros, "zeros"), N, K, g,
                            _dev(out, "out"), _stream(stream)), "w4_repack")
    return out


def w4a16_workspace_bytes(M: int, N: int, K: int, g: int) -> int:
    return int(load().w4a16_workspace_bytes(M, N, K, g))


def w4a16_workspace_bytes_ex(M: int, N: int, K: int, g: int, block_n: int, ctas: int, schedule: int) -> int:
    return int(load().w4a16_workspace_bytes_ex(M, N, K, g, block_n, ctas, schedule))


def w4a16_workspace_bytes_opts(M: int, N: int, K: int, g: int, opts: Options) -> int:
    return int(load().w4a16_workspace_bytes_opts(M, N, K, g, ctypes.byref(opts)))


def w4a16_gemm_plan(M: int, N: int, K: int, g: int):
    """(block_n, ctas, schedule) that w4a16_gemm picks on the current device (schedule 1 stream-K, 2 whole tiles)."""
    b, s, c = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(load().w4a16_gemm_plan(M, N, K, g, ctypes.byref(b), ctypes.byref(s), ctypes.byref(c)), "w4a16_gemm_plan")
    return b.value, s.value, c.value


class Workspace:
    """A zero-filled device workspace that grows on demand (reuse it across calls on one stream: a stream other than the one it
    was made on waits for that one first, as for any tensor). ``scratch`` is a second buffer, for the calls that leave
    arbitrary bytes behind (w4a16_experts, w4_lora_add, the attention calls): the GEMMs' counters in the first have to stay zero.

    A buffer that was outgrown is kept: calls that are still running, or graphs that were captured, use it. Each buffer is
    at least twice the one before, so all of them together are less than twice the last."""

    def __init__(self, device=None):
        device = torch.device(device or "cuda")
        if device.type == "cuda" and device.index is None:  # it grows there, whichever device is then the current one
            device = torch.device("cuda", torch.cuda.current_device())
        self.device = device
        self.buf = torch.zeros(256, dtype=torch.uint8, device=self.device)
        self.scratch = torch.zeros(256, dtype=torch.uint8, device=self.device)
        self._outgrown = []

    def get(self, nbytes: int, stream=None) -> torch.Tensor:
        """The first buffer, of ``nbytes`` at least, for a call on ``stream`` (None: the current one)."""
        if self.buf.numel() < nbytes:
            self._outgrown.append(self.buf)
            with torch.cuda.stream(stream):
                self.buf = torch.zeros(max(nbytes, 2 * self.buf.numel()), dtype=torch.uint8, device=self.device)
        return self.buf

    def get_scratch(self, nbytes: int, stream=None) -> torch.Tensor:
        """The second buffer, of ``nbytes`` at least, for a call on ``stream`` (None: the current one)."""
        if self.scratch.numel() < nbytes:
            old = self.scratch
            self._outgrown.append(old)
            with torch.cuda.stream(stream):
                self.scratch = torch.empty(max(nbytes, 2 * old.numel()), dtype=torch.uint8, device=self.device)
                self.scratch[:256] = old[:256]  # the error word
        return self.scratch


def _gemm_workspace(workspace, device, nbytes: int, stream) -> torch.Tensor:
    if workspace is None:
        with torch.cuda.stream(stream):
            workspace = Workspace(device)
    return workspace.get(nbytes, stream) if isinstance(workspace, Workspace) else workspace


def _gemm_common(x, packed, N, K, g, y, workspace, block_n, ctas, schedule, stream):
    if x.dtype != torch.float16 or x.dim() != 2 or x.shape[1] != K:
        raise ValueError("x must be fp16 [M, K]")
    M = x.shape[0]
    if y is None:
        y = _empty((M, N), torch.float16, x.device, stream)
    elif y.dtype != torch.float16 or tuple(y.shape) != (M, N):
        raise ValueError("y must be fp16 [M, N]")
    need = w4a16_workspace_bytes_ex(M, N, K, g, block_n, ctas, schedule)
    if need == 0:
        raise W4Error(1, "w4a16_workspace_bytes")
    ws = _gemm_workspace(workspace, x.device, need, stream)
    nbytes = ws.numel() * ws.element_size()
    lib = load()
    if block_n == 0 and ctas == 0 and schedule == 0:
        rc = lib.w4a16_gemm(_dev(x, "x"), _dev(packed, "packed"), M, N, K, g, _dev(y, "y"), _dev(ws, "workspace"),
                            nbytes, _stream(stream))
    else:
        rc = lib.w4a16_gemm_ex(_dev(x, "x"), _dev(packed, "packed"), M, N, K, g, _dev(y, "y"),
                               _dev(ws, "workspace"), nbytes, block_n, ctas, schedule, _stream(stream))
    _check(rc, "w4a16_gemm")
    return y


def w4a16_gemm(x: torch.Tensor, packed: torch.Tensor, N: int, K: int, g: int, y: torch.Tensor | None = None,
               workspace=None, stream=None, weights_static: bool = False) -> torch.Tensor:
    """y [M,N] = x [M,K] . dequant(packed)^T, fp16 or bf16 (x's dtype: the packed scales must be of the
    same type). ``workspace``: a Workspace or a zeroed uint8 tensor. ``weights_static``: the kernel
    launched just before this call on the stream does not write ``packed`` (W4_FLAG_WEIGHTS_STATIC: the
    decode kernel may then fetch weights before that kernel ends)."""
    if weights_static or x.dtype == torch.bfloat16:
        return w4a16_gemm_opts(x, packed, N, K, g, flags=FLAG_WEIGHTS_STATIC if weights_static else 0, y=y,
                               workspace=workspace, stream=stream)
    return _gemm_common(x, packed, N, K, g, y, workspace, 0, 0, 0, stream)


def w4a16_gemm_opts(x: torch.Tensor, packed: torch.Tensor, N: int, K: int, g: int, *, kernel: int = 0,
                    block_n: int = 0, ctas: int = 0, schedule: int = 0, cluster: int = 0, flags: int = 0,
                    wait_limit_cycles: int = 0, y: torch.Tensor | None = None, workspace=None,
                    stream=None) -> torch.Tensor:
    """w4a16_gemm with the options of w4a16_options (see include/w4a16.h); the dtype option follows x."""
    if x.dtype not in _DTYPES or x.dim() != 2 or x.shape[1] != K:
        raise ValueError("x must be fp16 or bf16 [M, K]")
    M = x.shape[0]
    if y is None:
        y = _empty((M, N), x.dtype, x.device, stream)
    elif y.dtype != x.dtype or tuple(y.shape) != (M, N):
        raise ValueError("y must be [M, N] of x's dtype")
    o = Options(kernel, block_n, ctas, schedule, cluster, flags, wait_limit_cycles, _DTYPES[x.dtype], 0)
    need = w4a16_workspace_bytes_opts(M, N, K, g, o)
    if need == 0:
        raise W4Error(1, "w4a16_workspace_bytes_opts")
    ws = _gemm_workspace(workspace, x.device, need, stream)
    nbytes = ws.numel() * ws.element_size()
    rc = load().w4a16_gemm_opts(_dev(x, "x"), _dev(packed, "packed"), M, N, K, g, _dev(y, "y"),
                                _dev(ws, "workspace"), nbytes, ctypes.byref(o), _stream(stream))
    _check(rc, "w4a16_gemm_opts")
    return y


def w4a16_gemm_ex(x, packed, N, K, g, block_n: int = 0, ctas: int = 0, schedule: int = 0, y=None, workspace=None,
                  stream=None):
    """w4a16_gemm with the schedule forced: block_n in {8,16,32,64,128} (8: the register-operand decode
    kernel; 16..128: the tensor-memory kernel), ctas >= 1, schedule 1 stream-K or 2 whole tiles (0 = automatic
    for each)."""
    return _gemm_common(x, packed, N, K, g, y, workspace, block_n, ctas, schedule, stream)


def w4_last_device_error(workspace, stream=None) -> int:
    """Reads and clears the workspace's device error word, or a Workspace's two, of the GEMMs and of w4a16_experts (synchronises
    the stream). After W4_ERR_TIMEOUT from a GEMM the workspace's tile counters are undefined too: zero it before reuse."""
    buffers = (workspace.buf, workspace.scratch) if isinstance(workspace, Workspace) else (workspace,)
    found = [int(load().w4_last_device_error(_dev(ws, "workspace"), _stream(stream))) for ws in buffers]
    return next((rc for rc in found if rc), 0)


# ----------------------------------------------------------------------------- groups and epilogues

def _problem_array(problems, M, dtype, device, stream=None):
    """(ctypes array of Problem, outputs per problem, tensors to keep alive)."""
    arr = (Problem * len(problems))()
    outs, keep = [], []
    for i, pr in enumerate(problems):
        x, packed, N, K = pr["x"], pr["packed"], int(pr["N"]), int(pr["K"])
        if x.dtype != dtype or x.dim() != 2 or tuple(x.shape) != (M, K):
            raise ValueError(f"problem {i}: x must be [{M}, {K}] of the group's dtype")
        epi = Epilogue()
        if pr.get("silu_mul"):
            epi.kind = EPI_SILU_MUL
            y = pr.get("y")
            if y is None:
                y = _empty((M, N // 2), dtype, device, stream)
            elif y.dtype != dtype or tuple(y.shape) != (M, N // 2):
                raise ValueError(f"problem {i}: y must be [{M}, {N // 2}]")
            out = y
        elif pr.get("qkv"):
            head_dim, q_per_group = pr["qkv"]
            span = (q_per_group + 2) * head_dim
            if N % span:
                raise ValueError(f"problem {i}: N must be a multiple of (q_per_group + 2) * head_dim")
            groups = N // span
            epi.kind, epi.head_dim, epi.q_per_group = EPI_QKV_SPLIT, head_dim, q_per_group
            shapes = ((M, groups * q_per_group * head_dim), (M, groups * head_dim), (M, groups * head_dim))
            if pr.get("out") is not None:
                q, k, v = pr["out"]
                if any(t.dtype != dtype or tuple(t.shape) != sh for t, sh in zip((q, k, v), shapes)):
                    raise ValueError(f"problem {i}: out must be q, k, v of shapes {shapes}")
            else:
                q, k, v = (_empty(sh, dtype, device, stream) for sh in shapes)
            epi.k_dev, epi.v_dev = k.data_ptr(), v.data_ptr()
            y, out = q, (q, k, v)
            keep += [k, v]
        else:
            y = pr.get("y")
            if y is None:
                y = _empty((M, N), dtype, device, stream)
            elif y.dtype != dtype or tuple(y.shape) != (M, N):
                raise ValueError(f"problem {i}: y must be [{M}, {N}]")
            out = y
        arr[i] = Problem(_dev(x, "x").value, _dev(packed, "packed").value, _dev(y, "y").value, N, K, epi)
        outs.append(out)
        keep += [x, packed, y]
    return arr, outs, keep


def w4a16_grouped_workspace_bytes(problems, g: int, **opts) -> int:
    x0 = problems[0]["x"]
    arr, _, _ = _problem_array(problems, x0.shape[0], x0.dtype, x0.device)
    o = Options(opts.get("kernel", 0), opts.get("block_n", 0), opts.get("ctas", 0), opts.get("schedule", 0),
                opts.get("cluster", 0), opts.get("flags", 0), opts.get("wait_limit_cycles", 0), _DTYPES[x0.dtype], 0)
    return int(load().w4a16_grouped_workspace_bytes(arr, len(problems), x0.shape[0], g, ctypes.byref(o)))


def w4a16_gemm_grouped(problems, g: int, *, kernel: int = 0, block_n: int = 0, ctas: int = 0, schedule: int = 0,
                       cluster: int = 0, flags: int = 0, wait_limit_cycles: int = 0, workspace=None, stream=None):
    """Independent GEMMs of one M, g and dtype in one call (w4a16_gemm_grouped). Each problem is a dict
    with x [M, K], packed, N, K, and optionally y (the output), silu_mul=True (y [M, N/2] =
    silu(gate) * up for weight rows alternating gate, up) or qkv=(head_dim, q_per_group) (weight rows in
    head groups; the output is (q, k, v), given as out=(q, k, v) or allocated). Returns the outputs in
    order."""
    if not problems:
        raise ValueError("empty group")
    x0 = problems[0]["x"]
    if x0.dtype not in _DTYPES:
        raise ValueError("x must be fp16 or bf16")
    M = x0.shape[0]
    arr, outs, keep = _problem_array(problems, M, x0.dtype, x0.device, stream)
    o = Options(kernel, block_n, ctas, schedule, cluster, flags, wait_limit_cycles, _DTYPES[x0.dtype], 0)
    need = int(load().w4a16_grouped_workspace_bytes(arr, len(problems), M, g, ctypes.byref(o)))
    if need == 0:
        raise W4Error(1, "w4a16_grouped_workspace_bytes")
    ws = _gemm_workspace(workspace, x0.device, need, stream)
    nbytes = ws.numel() * ws.element_size()
    rc = load().w4a16_gemm_grouped(arr, len(problems), M, g, _dev(ws, "workspace"), nbytes, ctypes.byref(o),
                                   _stream(stream))
    _check(rc, "w4a16_gemm_grouped")
    del keep
    return outs


def w4a16_gemm_silu_mul(x, packed, N: int, K: int, g: int, y=None, workspace=None, stream=None, **opts):
    """h [M, N/2] = silu(x . gate^T) * (x . up^T) for packed weight rows alternating gate, up."""
    return w4a16_gemm_grouped([dict(x=x, packed=packed, N=N, K=K, y=y, silu_mul=True)], g, workspace=workspace,
                              stream=stream, **opts)[0]


def w4a16_gemm_qkv(x, packed, N: int, K: int, g: int, head_dim: int, q_per_group: int, workspace=None, stream=None,
                   **opts):
    """(q, k, v) of a fused projection whose weight rows come in head groups (see qkv_head_group_rows)."""
    return w4a16_gemm_grouped([dict(x=x, packed=packed, N=N, K=K, qkv=(head_dim, q_per_group))], g,
                              workspace=workspace, stream=stream, **opts)[0]


def interleave_gate_up(gate: torch.Tensor, up: torch.Tensor) -> torch.Tensor:
    """[2 I, K] weights with row 2j = gate row j and row 2j + 1 = up row j (offline weight preparation)."""
    if gate.shape != up.shape or gate.dim() != 2:
        raise ValueError("gate and up must be [I, K] each")
    return torch.stack([gate, up], dim=1).reshape(2 * gate.shape[0], gate.shape[1])


def qkv_head_group_rows(wq: torch.Tensor, wk: torch.Tensor, wv: torch.Tensor, head_dim: int) -> torch.Tensor:
    """Fused q/k/v weights in head groups (r query heads, one key head, one value head per group), the row
    order W4_EPI_QKV_SPLIT reads (offline weight preparation)."""
    groups = wk.shape[0] // head_dim
    if wk.shape != wv.shape or wk.shape[0] % head_dim or wq.shape[0] % (groups * head_dim):
        raise ValueError("q, k, v rows must be whole heads, with as many key as value heads")
    r = wq.shape[0] // (groups * head_dim)
    K = wq.shape[1]
    q = wq.reshape(groups, r * head_dim, K)
    k = wk.reshape(groups, head_dim, K)
    v = wv.reshape(groups, head_dim, K)
    return torch.cat([q, k, v], dim=1).reshape(-1, K)


# ----------------------------------------------------------------------------- weights chosen row by row

_LOGIT_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_repacked = functools.lru_cache(maxsize=1024)(w4_repacked_bytes)

# A decode step makes these calls with a few microseconds of device work each, so the argument checks read each property
# once, the C ABI's argument structs are packed in one step, and the workspace is sized only when the library finds it
# too small.
_ROUTE_OPTIONS = struct.Struct("@6ifi")   # w4_route_options
_EXPERTS_ARGS = struct.Struct("@6P3q4i")  # w4a16_experts_args
_LORA_ARGS = struct.Struct("@8P6q4i")     # w4_lora_args


_DEVICES = [torch.device("cuda", i) for i in range(64)]


def _rows(t: torch.Tensor, name: str) -> int:
    """Values between the rows of a 2-D CUDA tensor, which are contiguous and do not overlap, but may lie further apart
    than they are long (a single row's stride says nothing)."""
    n, m = t.shape
    if n <= 1:
        if m > 1 and t.stride(1) != 1:
            raise ValueError(f"the rows of {name} must be contiguous")
        return -(-m // 8) * 8
    if t.is_contiguous():
        return m
    if m > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if t.stride(0) < m:
        raise ValueError(f"the rows of {name} must not overlap")
    return t.stride(0)


def _like(t: torch.Tensor, name: str, dtype, shape, device: int) -> int:
    """The address of a contiguous CUDA tensor of this type, shape and device index."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        raise ValueError(f"{name} must be {dtype} {list(shape)} on cuda:{device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _handle(stream, device: int) -> int:
    """The stream's handle. The library launches on the current device, so the tensors and the stream have to be its own."""
    current = torch._C._cuda_getDevice()
    if device != current:
        raise ValueError(f"the tensors are on cuda:{device}, the current device is cuda:{current}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device.index != device:
        raise ValueError(f"the tensors are on cuda:{device}, the stream is of {stream.device}")
    return stream.cuda_stream


def _run_with(call, args, workspace, sized, device: int, stream, what: str):
    """call(args, workspace, its bytes, stream). A Workspace grows, and without one a buffer is made, by sized()."""
    handle = _handle(stream, device)
    if workspace is None:
        if stream is None:
            ws = torch.empty(max(sized(), 1), dtype=torch.uint8, device=_DEVICES[device])
        else:
            with torch.cuda.stream(stream):
                ws = torch.empty(max(sized(), 1), dtype=torch.uint8, device=_DEVICES[device])
    else:
        ws = workspace.scratch if isinstance(workspace, Workspace) else workspace
        if ws.get_device() != device or not ws.is_contiguous():
            raise ValueError(f"workspace must be contiguous on cuda:{device}")
    rc = call(args, ws.data_ptr(), ws.nbytes, handle)
    if rc == 4 and isinstance(workspace, Workspace):
        ws = workspace.get_scratch(sized(), stream)
        rc = call(args, ws.data_ptr(), ws.nbytes, handle)
    if rc != 0:
        raise W4Error(rc, what)


def w4_route(logits: torch.Tensor, k: int, *, sigmoid: bool = False, bias: torch.Tensor | None = None, groups: int = 1,
             top_groups: int | None = None, group_top: int = 1, renormalize: bool = True, scale: float = 1.0,
             weights: torch.Tensor | None = None, ids: torch.Tensor | None = None, stream=None):
    """The k experts of each row of logits [T, E] (fp16, bf16 or fp32) and their weights: (weights fp32 [T, k], ids
    int32 [T, k]), largest first, the lowest index first among equals. Scores are the softmax of the logits, or
    their sigmoid; ``bias`` (fp32 [E]) is added for the choice alone; with ``groups`` > 1 only the ``top_groups``
    groups with the largest sum of their ``group_top`` best scores are chosen from. Weights are the chosen scores,
    divided by their sum (``renormalize``), times ``scale``. -inf masks an expert."""
    dt = _LOGIT_DTYPES.get(logits.dtype)
    if dt is None or logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("logits must be a 2-D fp16, bf16 or fp32 CUDA tensor")
    T, E = logits.shape
    device = logits.get_device()
    ld = _rows(logits, "logits")
    b = None if bias is None else _like(bias, "bias", torch.float32, (E,), device)
    shape = (T, max(k, 0))
    if weights is None:
        weights = _empty(shape, torch.float32, logits.device, stream)
        w_at = weights.data_ptr()
    else:
        w_at = _like(weights, "weights", torch.float32, shape, device)
    if ids is None:
        ids = _empty(shape, torch.int32, logits.device, stream)
        i_at = ids.data_ptr()
    else:
        i_at = _like(ids, "ids", torch.int32, shape, device)
    o = _ROUTE_OPTIONS.pack(k, sigmoid, groups, groups if top_groups is None else top_groups, group_top, renormalize, scale,
                            dt)
    rc = (_lib or load()).w4_route(logits.data_ptr(), T, E, ld, b, o, w_at, i_at, _handle(stream, device))
    if rc != 0:
        raise W4Error(rc, "w4_route")
    return weights, ids


def w4a16_experts_workspace_bytes(T: int, K: int, I: int, experts: int, k: int, g: int) -> int:
    return int(load().w4a16_experts_workspace_bytes(T, K, I, experts, k, g))


def w4a16_experts(x: torch.Tensor, gate_up: torch.Tensor, down: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                  inter: int, g: int, *, y: torch.Tensor | None = None, workspace=None, stream=None, flags: int = 0,
                  wait_limit_cycles: int = 0) -> torch.Tensor:
    """y [T, K] with y[t] = sum_j weights[t, j] * down_e (silu(gate_e x[t]) * up_e x[t]), e = ids[t, j].

    x [T, K] fp16 or bf16; gate_up uint8 [E, w4_repacked_bytes(2 * inter, K, g)], each expert's packed rows
    alternating gate, up (see interleave_gate_up); down uint8 [E, w4_repacked_bytes(K, inter, g)]; ids int32 and
    weights fp32 [T, k] as w4_route gives them (an id outside [0, E) is a dropped choice). A wait that gave up inside a kernel
    (y is then undefined) can be asked for with w4_last_device_error(workspace), so only where one is given.
    ``wait_limit_cycles``: after how many clock cycles a wait gives up (0: about 1.5 s); ``flags``: FLAG_TEST_TIMEOUT,
    in tests."""
    dt = _DTYPES.get(x.dtype)
    if dt is None or x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous fp16 or bf16 CUDA tensor [T, K]")
    if gate_up.dim() != 2 or ids.dim() != 2:
        raise ValueError("gate_up must be [E, bytes] and ids [T, k]")
    T, K = x.shape
    E, k = gate_up.shape[0], ids.shape[1]
    device = x.get_device()
    lib = _lib or load()
    gu_bytes, dn_bytes = _repacked(2 * inter, K, g), _repacked(K, inter, g)
    if not gu_bytes or not dn_bytes:
        raise W4Error(1, "w4a16_experts")
    if K % 8 or inter % 8:
        raise W4Error(2, "w4a16_experts")
    own = y is None
    if own:
        y = _empty(x.shape, x.dtype, x.device, stream)
    a = _EXPERTS_ARGS.pack(
        x.data_ptr(), _like(gate_up, "gate_up", torch.uint8, (E, gu_bytes), device),
        _like(down, "down", torch.uint8, (E, dn_bytes), device), _like(ids, "ids", torch.int32, (T, k), device),
        _like(weights, "weights", torch.float32, (T, k), device),
        y.data_ptr() if own else _like(y, "y", x.dtype, (T, K), device), T, K, inter, E, k, g, dt)
    call = lib.w4a16_experts
    if flags or wait_limit_cycles:
        o = ctypes.byref(Options(flags=flags, wait_limit_cycles=wait_limit_cycles))

        def call(args, ws, nbytes, handle):
            return lib.w4a16_experts_opts(args, ws, nbytes, o, handle)
    _run_with(call, a, workspace, lambda: w4a16_experts_workspace_bytes(T, K, inter, E, k, g), device, stream,
              "w4a16_experts")
    return y


def w4_lora_workspace_bytes(T: int, K: int, N: int, adapters: int, rank: int) -> int:
    return int(load().w4_lora_workspace_bytes(T, K, N, adapters, rank))


def w4_lora_add(base: torch.Tensor | None, x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, adapter: torch.Tensor, *,
                scaling: torch.Tensor | None = None, ranks: torch.Tensor | None = None, y: torch.Tensor | None = None,
                workspace=None, stream=None) -> torch.Tensor:
    """y [T, N] = base + scaling[a] * B[a] . (A[a] . x) with each row's own adapter a (base alone for a row whose index
    is outside [0, R)).

    x [T, K], base [T, N] (or None for zeros) and y fp16 or bf16, rows contiguous, A [R, rank, K], B [R, N, rank] of
    the same type, adapter int32 [T], scaling fp32 [R] (None: 1), ranks int32 [R] (None: rank): an adapter's own
    rank, past which A and B are not used. ``y`` may be ``base`` (in place). There is no gradient: A, B or scaling that
    require one are refused where gradients are recorded."""
    dtype = x.dtype
    dt = _DTYPES.get(dtype)
    if dt is None or x.dim() != 2 or not x.is_cuda or A.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be a fp16 or bf16 CUDA tensor [T, K], A [R, rank, K] and B [R, N, rank]")
    if (A.requires_grad or B.requires_grad or (scaling is not None and scaling.requires_grad)) and torch.is_grad_enabled():
        raise ValueError("w4_lora_add has no gradient: call it under torch.no_grad(), or with A, B and scaling detached")
    T, K = x.shape
    R, rank, _ = A.shape
    N = B.shape[1]
    device = x.get_device()
    shape = (T, N)
    if y is None:
        y = _empty(shape, dtype, x.device, stream)
    elif y.dtype is not dtype or y.shape != shape or y.get_device() != device:
        raise ValueError(f"y must be {dtype} [{T}, {N}] on cuda:{device}")
    if base is None:
        base_at = ldbase = 0
    elif base.dtype is not dtype or base.shape != shape or base.get_device() != device:
        raise ValueError(f"base must be {dtype} [{T}, {N}] on cuda:{device}")
    else:
        base_at, ldbase = base.data_ptr(), _rows(base, "base")
    a = _LORA_ARGS.pack(
        x.data_ptr(), _like(A, "A", dtype, (R, rank, K), device), _like(B, "B", dtype, (R, N, rank), device),
        _like(adapter, "adapter", torch.int32, (T,), device),
        0 if scaling is None else _like(scaling, "scaling", torch.float32, (R,), device),
        0 if ranks is None else _like(ranks, "ranks", torch.int32, (R,), device),
        base_at, y.data_ptr(), T, K, N, _rows(x, "x"), ldbase, _rows(y, "y"), R, rank, dt, 0)
    _run_with((_lib or load()).w4_lora_add, a, workspace, lambda: w4_lora_workspace_bytes(T, K, N, R, rank), device, stream,
              "w4_lora_add")
    return y


# ----------------------------------------------------------------------------- a decoder layer's attention

_ROPE_ARGS = struct.Struct("@8P5q11if")          # w4_rope_args
_KV_APPEND_ARGS = struct.Struct("@9P4q6i")       # w4_kv_append_args
_KV_ATTENTION_ARGS = struct.Struct("@8P3q8if")   # w4_kv_attention_args
_PROMPT_ARGS = struct.Struct("@5P5q5if")         # w4_prompt_attention_args


_F8, _F32, _I32 = torch.float8_e4m3fn, torch.float32, torch.int32


def _heads(t: torch.Tensor, name: str, dtype, shape, device: int):
    """(address, values between rows) of a CUDA tensor [.., heads, head_dim] of this type and shape, whose rows hold their
    heads one after another and lie evenly apart."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        raise ValueError(f"{name} must be {dtype} {list(shape)} on cuda:{device}")
    if t.is_contiguous():
        return t.data_ptr(), shape[-2] * shape[-1]
    return _apart(t, name)


def _apart(t: torch.Tensor, name: str):
    """_heads of a tensor that is not contiguous, its type and shape apart."""
    shape, strides = t.shape, t.stride()
    heads, dim = shape[-2:]
    width = heads * dim
    if (dim > 1 and strides[-1] != 1) or (heads > 1 and strides[-2] != dim):
        raise ValueError(f"the heads of {name} must follow one another in a row")
    if len(shape) == 3:
        ld = strides[0] if shape[0] > 1 else width
    else:
        batch, n = shape[0], shape[1]
        if batch > 1 and n > 1 and strides[0] != n * strides[1]:
            raise ValueError(f"the rows of {name} must lie evenly apart")
        ld = strides[1] if n > 1 else strides[0] if batch > 1 else width
    if ld < width:
        raise ValueError(f"the rows of {name} must not overlap")
    return t.data_ptr(), ld


def _empty_heads(t: torch.Tensor, stream) -> torch.Tensor:
    """_empty of a tensor's type and shape (empty_like takes a third less time, but keeps strides)."""
    if stream is None and t.is_contiguous():
        return torch.empty_like(t)
    return _empty(t.shape, t.dtype, t.device, stream)


def _no_gradient(what: str):
    """For a call whose inputs require a gradient."""
    if torch.is_grad_enabled():
        raise ValueError(f"{what} has no gradient: call it under torch.no_grad(), or with its inputs detached")


def w4_qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor | None, freqs: torch.Tensor | None, *,
                    q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                    sections=None, interleaved: bool = False, q_out: torch.Tensor | None = None,
                    k_out: torch.Tensor | None = None, stream=None):
    """Norm (with ``q_weight``, ``k_weight``: [head_dim]) and rotation by position of each head of q [T, heads, head_dim] and k
    (or None), fp16 or bf16: (q, k) of the same shapes. Rows may lie further apart than they are long (slices of a fused
    projection); ``q_out`` and ``k_out`` may be q and k (in place).

    The first 2 * len(freqs) values of a head are turned by positions * freqs (int32 [T] and fp32): value i with i +
    len(freqs), or neighbours (``interleaved``). With positions [axes, T] (up to 4: time, height, width) ``sections``
    says how many of the frequencies, in order, go by each axis. freqs None: no rotation. There is no gradient."""
    dtype, shape, device = q.dtype, q.shape, q.get_device()
    dt = _DTYPES.get(dtype)
    if dt is None or len(shape) != 3 or device < 0:
        raise ValueError("q must be a fp16 or bf16 CUDA tensor [T, heads, head_dim]")
    if (q.requires_grad or (k is not None and k.requires_grad) or (q_weight is not None and q_weight.requires_grad) or
            (k_weight is not None and k_weight.requires_grad) or (freqs is not None and freqs.requires_grad) or
            (q_out is not None and q_out.requires_grad) or (k_out is not None and k_out.requires_grad)):
        _no_gradient("w4_qk_norm_rope")
    T, hq, dim = shape
    q_at, ldq = (q.data_ptr(), hq * dim) if q.is_contiguous() else _apart(q, "q")
    if q_out is None:
        q_out = _empty_heads(q, stream)
        qo_at, ldqo = q_out.data_ptr(), hq * dim
    else:
        qo_at, ldqo = _heads(q_out, "q_out", dtype, shape, device)
    if k is None:
        if k_out is not None or k_weight is not None:
            raise ValueError("k_out and k_weight go with k")
        hk = k_at = ldk = ko_at = ldko = 0
    else:
        shape = k.shape
        if len(shape) != 3 or shape[0] != T or shape[2] != dim or k.dtype is not dtype or k.get_device() != device:
            raise ValueError(f"k must be {dtype} [{T}, heads, {dim}] on cuda:{device}")
        hk = shape[1]
        k_at, ldk = (k.data_ptr(), hk * dim) if k.is_contiguous() else _apart(k, "k")
        if k_out is None:
            k_out = _empty_heads(k, stream)
            ko_at, ldko = k_out.data_ptr(), hk * dim
        else:
            ko_at, ldko = _heads(k_out, "k_out", dtype, shape, device)
    part = 0, 0, 0, 0
    if freqs is None:
        if positions is not None or sections is not None:
            raise ValueError("positions and sections go with freqs")
        half = axes = p_at = f_at = 0
    else:
        half = freqs.numel()
        f_at = _like(freqs, "freqs", _F32, (half,), device)
        if positions is None:
            raise ValueError("freqs go with positions")
        if sections is None:
            axes, part = 1, (half, 0, 0, 0)
            p_at = _like(positions, "positions", _I32, (T,), device)
        else:
            axes = len(sections)
            if not 1 <= axes <= 4:
                raise ValueError("sections must have an entry for each of up to 4 axes")
            part = (*sections, 0, 0, 0)[:4]
            p_at = _like(positions, "positions", _I32, (axes, T), device)
    a = _ROPE_ARGS.pack(q_at, k_at, qo_at, ko_at, p_at, f_at,
                        0 if q_weight is None else _like(q_weight, "q_weight", dtype, (dim,), device),
                        0 if k_weight is None else _like(k_weight, "k_weight", dtype, (dim,), device),
                        T, ldq, ldk, ldqo, ldko, hq, hk, dim, 2 * half, axes, *part, interleaved, dt, eps)
    rc = (_lib or load()).w4_qk_norm_rope(a, _handle(stream, device))
    if rc != 0:
        raise W4Error(rc, "w4_qk_norm_rope")
    return q_out, k_out


def _cache(k_cache, v_cache, k_scale, v_scale, table, batch: int, heads, dim: int, device: int, what: str):
    """(pages, heads, page, max_pages) of a paged cache (heads None: as many as it has) that goes with a call's other tensors."""
    shape = k_cache.shape
    if k_cache.requires_grad or v_cache.requires_grad or k_scale.requires_grad or v_scale.requires_grad:
        _no_gradient(what)
    if len(shape) != 4 or table.dim() != 2:
        raise ValueError("k_cache must be [pages, heads, page, head_dim] and table [batch, max_pages]")
    pages, hk, page, d = shape
    if (k_cache.dtype is not _F8 or v_cache.dtype is not _F8 or v_cache.shape != shape or d != dim or hk != (heads or hk) or
            k_cache.get_device() != device or v_cache.get_device() != device):
        raise ValueError(f"k_cache and v_cache must be {_F8} [pages, {heads or 'heads'}, page, {dim}] on cuda:{device}")
    if (k_scale.dtype is not _F32 or v_scale.dtype is not _F32 or k_scale.shape != (pages, hk) or v_scale.shape != (pages, hk) or
            k_scale.get_device() != device or v_scale.get_device() != device):
        raise ValueError(f"k_scale and v_scale must be {_F32} [{pages}, {hk}] on cuda:{device}")
    rows, max_pages = table.shape
    if table.dtype is not _I32 or rows != batch or table.get_device() != device:
        raise ValueError(f"table must be {_I32} [{batch}, max_pages] on cuda:{device}")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous() and k_scale.is_contiguous() and v_scale.is_contiguous() and
            table.is_contiguous()):
        raise ValueError("k_cache, v_cache, k_scale, v_scale and table must be contiguous")
    return pages, hk, page, max_pages


def w4_kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor, table: torch.Tensor, cu: torch.Tensor, lens: torch.Tensor, *, stream=None) -> None:
    """Writes rows cu[i] .. cu[i + 1] - 1 of k and v (fp16 or bf16 [T, heads, head_dim]) to positions lens[i], lens[i] + 1, ... of
    sequence i in the paged cache.

    k_cache, v_cache float8_e4m3fn [pages, heads, page, head_dim], k_scale, v_scale fp32 [pages, heads]: a value is
    code * scale. table int32 [batch, max_pages] lists each sequence's pages (-1: none; nothing is written there), cu int32
    [batch + 1] ascends, lens int32 [batch] is what the cache holds before the call (the caller adds the new rows to it). A page that
    gets rows must belong to one sequence only, and stand once in its row of the table. See w4_kv_append in include/w4a16.h for the scales."""
    dtype, shape, device = k.dtype, k.shape, k.get_device()
    dt = _DTYPES.get(dtype)
    if dt is None or len(shape) != 3 or device < 0:
        raise ValueError("k must be a fp16 or bf16 CUDA tensor [T, heads, head_dim]")
    if k.requires_grad or v.requires_grad:
        _no_gradient("w4_kv_append")
    T, heads, dim = shape
    batch = lens.numel()
    pages, _, page, max_pages = _cache(k_cache, v_cache, k_scale, v_scale, table, batch, heads, dim, device, "w4_kv_append")
    k_at, ldk = (k.data_ptr(), heads * dim) if k.is_contiguous() else _apart(k, "k")
    v_at, ldv = _heads(v, "v", dtype, shape, device)
    a = _KV_APPEND_ARGS.pack(k_at, v_at, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                             table.data_ptr(), _like(cu, "cu", _I32, (batch + 1,), device),
                             _like(lens, "lens", _I32, (batch,), device), T, ldk, ldv, pages, batch, max_pages, heads, dim, page, dt)
    rc = (_lib or load()).w4_kv_append(a, _handle(stream, device))
    if rc != 0:
        raise W4Error(rc, "w4_kv_append")


def w4_kv_attention_workspace_bytes(batch: int, n: int, q_heads: int, k_heads: int, head_dim: int) -> int:
    return int(load().w4_kv_attention_workspace_bytes(batch, n, q_heads, k_heads, head_dim))


def w4_kv_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                    table: torch.Tensor, lens: torch.Tensor, *, scale: float | None = None, out: torch.Tensor | None = None,
                    workspace=None, stream=None) -> torch.Tensor:
    """Attention of each sequence's last n positions over its part of the paged cache (w4_kv_append's): q fp16 or bf16
    [batch, n, q_heads, head_dim] or, for n = 1, [batch, q_heads, head_dim]; the result has q's shape. lens int32 [batch] counts
    the n positions in: query j sees positions up to lens[i] - n + j, and gives zeros where there is none. Query head h
    reads key head h // (q_heads // k_heads). ``scale``: of the products (None: 1 / sqrt(head_dim)). There is no gradient."""
    dtype, shape, device = q.dtype, q.shape, q.get_device()
    dt, dims = _DTYPES.get(dtype), len(shape)
    if dt is None or not 3 <= dims <= 4 or device < 0:
        raise ValueError("q must be a fp16 or bf16 CUDA tensor [batch, n, heads, head_dim] or [batch, heads, head_dim]")
    if q.requires_grad or (out is not None and out.requires_grad):
        _no_gradient("w4_kv_attention")
    if dims == 3:
        batch, hq, dim = shape
        n = 1
    else:
        batch, n, hq, dim = shape
    pages, hk, page, max_pages = _cache(k_cache, v_cache, k_scale, v_scale, table, batch, None, dim, device, "w4_kv_attention")
    q_at, ldq = (q.data_ptr(), hq * dim) if q.is_contiguous() else _apart(q, "q")
    if out is None:
        out = _empty_heads(q, stream)
        o_at, ldo = out.data_ptr(), hq * dim
    else:
        o_at, ldo = _heads(out, "out", dtype, shape, device)
    a = _KV_ATTENTION_ARGS.pack(q_at, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), table.data_ptr(),
                                _like(lens, "lens", _I32, (batch,), device), o_at, ldq, ldo, pages, batch, n, max_pages, hq, hk, dim,
                                page, dt, (dim or 1) ** -0.5 if scale is None else scale)
    _run_with((_lib or load()).w4_kv_attention, a, workspace, lambda: w4_kv_attention_workspace_bytes(batch, n, hq, hk, dim),
              device, stream, "w4_kv_attention")
    return out


def w4_prompt_attention_workspace_bytes(T: int, batch: int, q_heads: int) -> int:
    return int(load().w4_prompt_attention_workspace_bytes(T, batch, q_heads))


def w4_prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, *, scale: float | None = None,
                        out: torch.Tensor | None = None, workspace=None, stream=None, flags: int = 0,
                        wait_limit_cycles: int = 0) -> torch.Tensor:
    """Causal attention over packed prompts: rows cu[i] .. cu[i + 1] - 1 of q [T, q_heads, head_dim] and of k and v
    [T, k_heads, head_dim], fp16 or bf16, are sequence i; a row sees its sequence up to itself, and query head h reads key head
    h // (q_heads // k_heads). cu int32 [batch + 1] on the GPU, ascending. Rows outside of all sequences are left as they are in
    ``out``. ``scale``: of the products (None: 1 / sqrt(head_dim)). There is no gradient. A wait that gave up inside the
    kernel (out is then undefined) can be asked for with w4_last_device_error(workspace), so only where one is given;
    ``wait_limit_cycles``: after how many clock cycles it gives up (0: about 1.5 s), for a step of 64 or 128 keys however many a
    prompt has; ``flags``: FLAG_TEST_TIMEOUT, in tests."""
    dtype, shape, device = q.dtype, q.shape, q.get_device()
    dt = _DTYPES.get(dtype)
    k_shape, batch = k.shape, cu.numel() - 1
    if dt is None or len(shape) != 3 or len(k_shape) != 3 or device < 0 or batch < 0:
        raise ValueError("q must be a fp16 or bf16 CUDA tensor [T, heads, head_dim], k alike and cu [batch + 1]")
    if q.requires_grad or k.requires_grad or v.requires_grad or (out is not None and out.requires_grad):
        _no_gradient("w4_prompt_attention")
    T, hq, dim = shape
    hk = k_shape[1]
    if k_shape[0] != T or k_shape[2] != dim or k.dtype is not dtype or k.get_device() != device:
        raise ValueError(f"k must be {dtype} [{T}, heads, {dim}] on cuda:{device}")
    q_at, ldq = (q.data_ptr(), hq * dim) if q.is_contiguous() else _apart(q, "q")
    k_at, ldk = (k.data_ptr(), hk * dim) if k.is_contiguous() else _apart(k, "k")
    v_at, ldv = _heads(v, "v", dtype, k_shape, device)
    if out is None:
        out = _empty_heads(q, stream)
        o_at, ldo = out.data_ptr(), hq * dim
    else:
        o_at, ldo = _heads(out, "out", dtype, shape, device)
    lib = _lib or load()
    a = _PROMPT_ARGS.pack(q_at, k_at, v_at, _like(cu, "cu", _I32, (batch + 1,), device), o_at, T, ldq, ldk, ldv, ldo, batch, hq, hk,
                          dim, dt, (dim or 1) ** -0.5 if scale is None else scale)
    call = lib.w4_prompt_attention
    if flags or wait_limit_cycles:
        o = ctypes.byref(Options(flags=flags, wait_limit_cycles=wait_limit_cycles))

        def call(args, ws, nbytes, handle):
            return lib.w4_prompt_attention_opts(args, ws, nbytes, o, handle)
    _run_with(call, a, workspace, lambda: lib.w4_prompt_attention_workspace_bytes(T, batch, hq), device, stream, "w4_prompt_attention")
    return out
