"""ctypes binding of libmole (include/mole.h): same entry-point names, argument
marshalling only.  Every step of the computation runs in the library's CUDA
kernels; PyTorch supplies device memory and the current stream.

Importing this module loads ``libmole.so`` from this package directory and
raises ``ImportError`` if it is missing -- there is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import itertools
import operator
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmole.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libmole.so not found at {LIB_PATH}; build it with "
        "`python -m mixture_lookup_experts_b200._build` (nvcc, sm_100a)")

lib = ctypes.CDLL(LIB_PATH)

MOLE_OK = 0
STATUS = {0: "MOLE_OK", 1: "MOLE_ERR_ARG", 2: "MOLE_ERR_ALIGN", 3: "MOLE_ERR_UNSUPPORTED",
          4: "MOLE_ERR_WORKSPACE", 5: "MOLE_ERR_INDEX", 6: "MOLE_ERR_CUDA", 7: "MOLE_ERR_TIMEOUT",
          8: "MOLE_ERR_NO_DEVICE"}
F32, BF16 = 0, 1
ACT = {"gelu": 0, "gelu_erf": 0, "gelu_tanh": 1, "relu": 2, "silu": 3, "identity": 4}

# Every function include/mole.h declares, with its ctypes signature.
_P, _I64, _I32, _I, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_size_t
_F = ctypes.c_float
SIGNATURES = {
    "mole_status_str": ([_I], ctypes.c_char_p),
    "mole_version": ([], _I),
    "mole_build_lut_workspace": ([_I64, _I64, _I32, _I64, _I, _I32], _SZ),
    "mole_build_lut": ([_P, _P, _P, _I64, _I64, _I32, _I64, _I, _I, _P, _P, _SZ, _P], _I),
    "mole_build_lut_noalloc": ([_P, _P, _P, _I64, _I64, _I32, _I64, _I, _I, _P, _P], _I),
    "mole_lookup_combine": ([_P, _I64, _P, _P, _P, _I64, _I32, _I64, _I, _P, _P], _I),
    "mole_token_groups_workspace": ([_I64, _I32], _SZ),
    "mole_token_groups_build": ([_P, _I64, _I64, _I32, _P, _SZ, _P], _I),
    "mole_lookup_combine_groups": ([_P, _I64, _P, _SZ, _P, _P, _P, _I64, _I32, _I64, _I, _P, _P], _I),
    "mole_lookup_combine_grouped_workspace": ([_I64, _I32], _SZ),
    "mole_lookup_combine_grouped": ([_P, _I64, _P, _P, _P, _I64, _I32, _I64, _I, _P, _P, _SZ, _P], _I),
    "mole_quantize_lut_nf3": ([_P, _I64, _I32, _I64, _P, _P, _P], _I),
    "mole_lookup_combine_nf3": ([_P, _I64, _P, _P, _P, _P, _I64, _I32, _I64, _I, _P, _P], _I),
    "mole_lookup_combine_nf3_groups": ([_P, _I64, _P, _SZ, _P, _P, _P, _P, _I64, _I32, _I64, _I, _P, _P], _I),
    "mole_offload_staging_bytes": ([_I64, _I64, _I32, _I64, _I, _I32], _SZ),
    "mole_offload_stage": ([_I64, _P, _SZ, _P, _P, _I64, _I32, _I64, _I, _I32, _P, _SZ, _P, _P], _I),
    "mole_lookup_combine_offload": ([_I64, _P, _SZ, _P, _P, _P, _SZ, _I64, _I32, _I64, _I, _I32, _P, _P], _I),
    "mole_shared_ffn_workspace": ([_I64, _I64], _SZ),
    "mole_shared_ffn": ([_P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _P, _P, _SZ, _P], _I),
    "mole_ffn_block_workspace": ([_I64, _I64, _I64], _SZ),
    "mole_ffn_block": ([_P, _I64, _P, _SZ, _P, _P, _P, _I64, _I32, _P, _P, _I64, _I64, _I, _P, _P, _P, _SZ, _P], _I),
    "mole_build_lut_nf3": ([_P, _P, _P, _I64, _I64, _I32, _I64, _I, _P, _P, _P, _SZ, _P], _I),
    "mole_train_cache_bytes": ([_I64, _I64, _I32, _I64, _I64], _SZ),
    "mole_train_forward": ([_P, _I64, _P, _SZ, _P, _P, _P, _P, _P, _I64, _I32, _I64, _I64, _I, _P, _P, _SZ, _P, _P],
                           _I),
    "mole_train_backward": ([_P, _I64, _P, _SZ, _P, _P, _P, _P, _P, _I64, _I32, _I64, _I64, _I, _P, _P, _SZ, _I32,
                             _P, _P, _P, _P, _P, _P], _I),
    "mole_nf3_levels": ([_P], None),
    "mole_nf3_midpoints": ([_P], None),
    "mole_gather_plan": ([_P, _I64, _I64, _P, _P, _P, _P], _I),
    "mole_prefetch_rows": ([_P, _I64, _P, _I32, _I64, _I64, _P], _I),
    "mole_check": ([_P, _I], _I),
    "mole_embed_forward": ([_P, _I64, _P, _I64, _I64, _F, _I, _P, _I, _P], _I),
    "mole_embed_backward_workspace": ([_I64, _I64], _SZ),
    "mole_embed_backward": ([_P, _I64, _P, _I, _I64, _I64, _F, _P, _P, _SZ, _P], _I),
    "mole_block_norm_forward": ([_P, _I, _P, _I, _P, _P, _F, _P, _F, _I64, _I64, _P, _P, _I, _P], _I),
    "mole_block_norm_backward_workspace": ([_I64, _I64], _SZ),
    "mole_block_norm_backward": ([_P, _I, _P, _I, _P, _P, _F, _P, _F, _I64, _I64] + [_P] * 8 + [_SZ, _P], _I),
    "mole_adamw_step": ([_P, _I32, _P, _P], _I),
}
for _name, (_args, _res) in SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


class MoleError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} "
                         f"({lib.mole_status_str(status).decode()})")


def _ok(status: int, where: str) -> None:
    if status != MOLE_OK:
        raise MoleError(status, where)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def mole_version() -> int:
    return lib.mole_version()


def mole_status_str(status: int) -> str:
    return lib.mole_status_str(status).decode()


def mole_build_lut_workspace(V: int, D: int, N: int, Dr: int, dtype=torch.bfloat16,
                             experts_per_launch: int = 0) -> int:
    dt = BF16 if dtype == torch.bfloat16 else F32
    return int(lib.mole_build_lut_workspace(V, D, N, Dr, dt, experts_per_launch))


def mole_build_lut(embed: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor, act: str = "gelu",
                   lut: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """LUT[v, j, :] = act(E[v] . W1[j]) . W2[j] on the device (see mole.h)."""
    _contig(embed, W1, W2, lut, workspace)
    V, D = embed.shape
    N, D2, Dr = W1.shape
    if D2 != D or tuple(W2.shape) != (N, Dr, D):
        raise ValueError("shape mismatch: embed [V,D], W1 [N,D,Dr], W2 [N,Dr,D]")
    dt = _dt(embed)
    if lut is None:
        lut = torch.empty((V, N, D), dtype=embed.dtype, device=embed.device)
    if workspace is None:
        nbytes = mole_build_lut_workspace(V, D, N, Dr, embed.dtype, 0)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=embed.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _ok(lib.mole_build_lut(_ptr(embed), _ptr(W1), _ptr(W2), V, D, N, Dr, ACT[act], dt, _ptr(lut),
                           _ptr(workspace), ws_bytes, _stream(stream)), "mole_build_lut")
    return lut


def mole_build_lut_noalloc(embed: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor, act: str = "gelu",
                           lut: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """mole_build_lut with the scratch in the library's fixed device array
    (no allocation inside the call; see mole.h for the size limit)."""
    _contig(embed, W1, W2, lut)
    V, D = embed.shape
    N, D2, Dr = W1.shape
    if D2 != D or tuple(W2.shape) != (N, Dr, D):
        raise ValueError("shape mismatch: embed [V,D], W1 [N,D,Dr], W2 [N,Dr,D]")
    if lut is None:
        lut = torch.empty((V, N, D), dtype=embed.dtype, device=embed.device)
    _ok(lib.mole_build_lut_noalloc(_ptr(embed), _ptr(W1), _ptr(W2), V, D, N, Dr, ACT[act], _dt(embed), _ptr(lut),
                                   _stream(stream)), "mole_build_lut_noalloc")
    return lut


def mole_lookup_combine(ids: torch.Tensor, h: torch.Tensor, Wr: torch.Tensor, lut: torch.Tensor,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = sum_j softmax(h[t] . Wr)_j LUT[ids[t], j] (fp32 out; see mole.h)."""
    _contig(ids, h, Wr, lut, out)
    V, N, D = lut.shape
    T = ids.numel()
    if out is None:
        out = torch.empty((T, D), dtype=torch.float32, device=h.device)
    _ok(lib.mole_lookup_combine(_ptr(ids), T, _ptr(h), _ptr(Wr), _ptr(lut), V, N, D, _dt(h), _ptr(out),
                                _stream(stream)), "mole_lookup_combine")
    return out


def mole_token_groups_workspace(T: int, N: int) -> int:
    return int(lib.mole_token_groups_workspace(T, N))


def mole_token_groups_build(ids: torch.Tensor, V: int, N: int, groups: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """Groups the batch's tokens by id (once per batch; serves every layer
    with N experts).  Returns the groups buffer (see mole.h)."""
    _contig(ids, groups)
    T = ids.numel()
    if groups is None:
        groups = torch.empty(max(1, mole_token_groups_workspace(T, N)), dtype=torch.uint8, device=ids.device)
    nbytes = groups.numel() * groups.element_size()
    _ok(lib.mole_token_groups_build(_ptr(ids), T, V, N, _ptr(groups), nbytes, _stream(stream)),
        "mole_token_groups_build")
    return groups


def mole_lookup_combine_groups(ids: torch.Tensor, groups: torch.Tensor, h: torch.Tensor, Wr: torch.Tensor,
                               lut: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """mole_lookup_combine over a grouping built from the same ids (each
    distinct row block read once); same result bit for bit (see mole.h)."""
    _contig(ids, groups, h, Wr, lut, out)
    V, N, D = lut.shape
    T = ids.numel()
    if out is None:
        out = torch.empty((T, D), dtype=torch.float32, device=h.device)
    nbytes = groups.numel() * groups.element_size()
    _ok(lib.mole_lookup_combine_groups(_ptr(ids), T, _ptr(groups), nbytes, _ptr(h), _ptr(Wr), _ptr(lut), V, N, D,
                                       _dt(h), _ptr(out), _stream(stream)), "mole_lookup_combine_groups")
    return out


def mole_lookup_combine_grouped_workspace(T: int, N: int) -> int:
    return int(lib.mole_lookup_combine_grouped_workspace(T, N))


def mole_lookup_combine_grouped(ids: torch.Tensor, h: torch.Tensor, Wr: torch.Tensor, lut: torch.Tensor,
                                out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                                stream=None) -> torch.Tensor:
    """mole_lookup_combine with tokens grouped by id (each distinct row block
    fetched once per batch); same result bit for bit (see mole.h)."""
    _contig(ids, h, Wr, lut, out, workspace)
    V, N, D = lut.shape
    T = ids.numel()
    if out is None:
        out = torch.empty((T, D), dtype=torch.float32, device=h.device)
    if workspace is None:
        workspace = torch.empty(max(1, mole_lookup_combine_grouped_workspace(T, N)), dtype=torch.uint8,
                                device=h.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _ok(lib.mole_lookup_combine_grouped(_ptr(ids), T, _ptr(h), _ptr(Wr), _ptr(lut), V, N, D, _dt(h), _ptr(out),
                                        _ptr(workspace), ws_bytes, _stream(stream)), "mole_lookup_combine_grouped")
    return out


def mole_quantize_lut_nf3(lut: torch.Tensor, codes: torch.Tensor | None = None,
                          scales: torch.Tensor | None = None, stream=None):
    """NF3 codes [V, N, D/64, 24] uint8 and fp16 scales [V, N, D/64] (see mole.h)."""
    _contig(lut, codes, scales)
    V, N, D = lut.shape
    if codes is None:
        codes = torch.empty((V, N, D // 64, 24), dtype=torch.uint8, device=lut.device)
    if scales is None:
        scales = torch.empty((V, N, D // 64), dtype=torch.float16, device=lut.device)
    _ok(lib.mole_quantize_lut_nf3(_ptr(lut), V, N, D, _ptr(codes), _ptr(scales), _stream(stream)),
        "mole_quantize_lut_nf3")
    return codes, scales


def mole_build_lut_nf3(embed: torch.Tensor, W1: torch.Tensor, W2: torch.Tensor, act: str = "gelu",
                       codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None):
    """The table build with the NF3 quantiser in its epilogue: codes
    [V, N, D/64, 24] uint8 and fp16 scales [V, N, D/64] (see mole.h)."""
    _contig(embed, W1, W2, codes, scales, workspace)
    V, D = embed.shape
    N, _, Dr = W1.shape
    if codes is None:
        codes = torch.empty((V, N, D // 64, 24), dtype=torch.uint8, device=embed.device)
    if scales is None:
        scales = torch.empty((V, N, D // 64), dtype=torch.float16, device=embed.device)
    if workspace is None:
        workspace = torch.empty(mole_build_lut_workspace(V, D, N, Dr, torch.bfloat16, 0), dtype=torch.uint8,
                                device=embed.device)
    _ok(lib.mole_build_lut_nf3(_ptr(embed), _ptr(W1), _ptr(W2), V, D, N, Dr, ACT[act], _ptr(codes), _ptr(scales),
                               _ptr(workspace), workspace.numel(), _stream(stream)), "mole_build_lut_nf3")
    return codes, scales


def mole_lookup_combine_nf3(ids: torch.Tensor, h: torch.Tensor, Wr: torch.Tensor, codes: torch.Tensor,
                            scales: torch.Tensor, out: torch.Tensor | None = None, stream=None):
    _contig(ids, h, Wr, codes, scales, out)
    V, N, nb, _ = codes.shape
    D = nb * 64
    T = ids.numel()
    if out is None:
        out = torch.empty((T, D), dtype=torch.float32, device=h.device)
    _ok(lib.mole_lookup_combine_nf3(_ptr(ids), T, _ptr(h), _ptr(Wr), _ptr(codes), _ptr(scales), V, N, D,
                                    _dt(h), _ptr(out), _stream(stream)), "mole_lookup_combine_nf3")
    return out


def mole_lookup_combine_nf3_groups(ids: torch.Tensor, groups: torch.Tensor, h: torch.Tensor, Wr: torch.Tensor,
                                   codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor | None = None,
                                   stream=None):
    """mole_lookup_combine_nf3 over a grouping built from the same ids (each
    distinct code block read and decoded once); same result bit for bit."""
    _contig(ids, groups, h, Wr, codes, scales, out)
    V, N, nb, _ = codes.shape
    D = nb * 64
    T = ids.numel()
    if out is None:
        out = torch.empty((T, D), dtype=torch.float32, device=h.device)
    nbytes = groups.numel() * groups.element_size()
    _ok(lib.mole_lookup_combine_nf3_groups(_ptr(ids), T, _ptr(groups), nbytes, _ptr(h), _ptr(Wr), _ptr(codes),
                                           _ptr(scales), V, N, D, _dt(h), _ptr(out), _stream(stream)),
        "mole_lookup_combine_nf3_groups")
    return out


def mole_offload_staging_bytes(T: int, V: int, N: int, D: int, dtype=torch.bfloat16, nf3: bool = False) -> int:
    dt = BF16 if dtype == torch.bfloat16 else F32
    return int(lib.mole_offload_staging_bytes(T, V, N, D, dt, int(nf3)))


def _table_shape(table: torch.Tensor, scales: torch.Tensor | None):
    """(V, N, D, nf3) of a [V, N, D] table or NF3 codes [V, N, D/64, 24]."""
    if scales is None:
        V, N, D = table.shape
        return V, N, D, False
    V, N, nb, _ = table.shape
    return V, N, nb * 64, True


def mole_offload_stage(T: int, groups: torch.Tensor, table: torch.Tensor, scales: torch.Tensor | None = None,
                       staging: torch.Tensor | None = None, n_rows: torch.Tensor | None = None,
                       device=None, stream=None) -> torch.Tensor:
    """Copies the batch's distinct row blocks of `table` (pinned host memory;
    with `scales`, NF3 codes and scales) into a device staging buffer, by
    the dense index the grouping gave each id (see mole.h)."""
    _contig(groups, table, scales, staging, n_rows)
    V, N, D, nf3 = _table_shape(table, scales)
    dtype = torch.bfloat16 if nf3 else table.dtype
    if staging is None:
        nbytes = max(1, mole_offload_staging_bytes(T, V, N, D, dtype, nf3))
        staging = torch.empty(nbytes, dtype=torch.uint8, device=device if device is not None else groups.device)
    _ok(lib.mole_offload_stage(T, _ptr(groups), groups.numel(), _ptr(table), _ptr(scales), V, N, D,
                               BF16 if dtype == torch.bfloat16 else F32, int(nf3), _ptr(staging), staging.numel(),
                               _ptr(n_rows), _stream(stream)), "mole_offload_stage")
    return staging


def mole_lookup_combine_offload(groups: torch.Tensor, h: torch.Tensor, Wr: torch.Tensor, staging: torch.Tensor,
                                V: int, nf3: bool = False, out: torch.Tensor | None = None,
                                stream=None) -> torch.Tensor:
    """mole_lookup_combine (nf3: mole_lookup_combine_nf3) over the rows that
    mole_offload_stage put into `staging`; same result bit for bit."""
    _contig(groups, h, Wr, staging, out)
    T, D = h.shape
    N = Wr.shape[1]
    if out is None:
        out = torch.empty((T, D), dtype=torch.float32, device=h.device)
    _ok(lib.mole_lookup_combine_offload(T, _ptr(groups), groups.numel(), _ptr(h), _ptr(Wr), _ptr(staging),
                                        staging.numel(), V, N, D, _dt(h), int(nf3), _ptr(out), _stream(stream)),
        "mole_lookup_combine_offload")
    return out


def mole_shared_ffn_workspace(T: int, Ds: int) -> int:
    return int(lib.mole_shared_ffn_workspace(T, Ds))


def mole_shared_ffn(h: torch.Tensor, W1s: torch.Tensor, W2s: torch.Tensor, act: str = "gelu",
                    add: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """out = act(h . W1s) . W2s + add + residual (fp32; see mole.h)."""
    _contig(h, W1s, W2s, add, residual, out, workspace)
    T, D = h.shape
    Ds = W1s.shape[1]
    if out is None:
        out = torch.empty((T, D), dtype=torch.float32, device=h.device)
    if workspace is None:
        workspace = torch.empty(max(1, mole_shared_ffn_workspace(T, Ds)), dtype=torch.uint8, device=h.device)
    _ok(lib.mole_shared_ffn(_ptr(h), _ptr(W1s), _ptr(W2s), T, D, Ds, ACT[act], _ptr(add), _ptr(residual), _ptr(out),
                            _ptr(workspace), workspace.numel(), _stream(stream)), "mole_shared_ffn")
    return out


def mole_ffn_block_workspace(T: int, D: int, Ds: int) -> int:
    return int(lib.mole_ffn_block_workspace(T, D, Ds))


def mole_ffn_block(ids: torch.Tensor, groups: torch.Tensor, h: torch.Tensor, Wr: torch.Tensor, lut: torch.Tensor,
                   W1s: torch.Tensor, W2s: torch.Tensor, act: str = "gelu", residual: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """out = residual + act(h . W1s) . W2s + the routed-expert mixture (see mole.h)."""
    _contig(ids, groups, h, Wr, lut, W1s, W2s, residual, out, workspace)
    V, N, D = lut.shape
    T = ids.numel()
    Ds = W1s.shape[1]
    if out is None:
        out = torch.empty((T, D), dtype=torch.float32, device=h.device)
    if workspace is None:
        workspace = torch.empty(max(1, mole_ffn_block_workspace(T, D, Ds)), dtype=torch.uint8, device=h.device)
    _ok(lib.mole_ffn_block(_ptr(ids), T, _ptr(groups), groups.numel(), _ptr(h), _ptr(Wr), _ptr(lut), V, N, _ptr(W1s),
                           _ptr(W2s), D, Ds, ACT[act], _ptr(residual), _ptr(out), _ptr(workspace), workspace.numel(),
                           _stream(stream)), "mole_ffn_block")
    return out


def mole_train_cache_bytes(T: int, V: int, N: int, D: int, Dr: int) -> int:
    return int(lib.mole_train_cache_bytes(T, V, N, D, Dr))


def mole_train_forward(ids: torch.Tensor, groups: torch.Tensor, h: torch.Tensor, Wr: torch.Tensor, E: torch.Tensor,
                       W1: torch.Tensor, W2: torch.Tensor, act: str = "gelu", out: torch.Tensor | None = None,
                       cache: torch.Tensor | None = None, stream=None):
    """(out, cache, n_distinct): one MoLE layer's training forward (see mole.h)."""
    _contig(ids, groups, h, Wr, E, W1, W2, out, cache)
    V, D = E.shape
    N, _, Dr = W1.shape
    T = ids.numel()
    if out is None:
        out = torch.empty((T, D), dtype=torch.float32, device=h.device)
    if cache is None:
        cache = torch.empty(max(1, mole_train_cache_bytes(T, V, N, D, Dr)), dtype=torch.uint8, device=h.device)
    n = ctypes.c_int32(0)
    _ok(lib.mole_train_forward(_ptr(ids), T, _ptr(groups), groups.numel(), _ptr(h), _ptr(Wr), _ptr(E), _ptr(W1),
                               _ptr(W2), V, N, D, Dr, ACT[act], _ptr(out), _ptr(cache), cache.numel(),
                               ctypes.addressof(n), _stream(stream)), "mole_train_forward")
    return out, cache, int(n.value)


def mole_train_backward(ids: torch.Tensor, groups: torch.Tensor, h: torch.Tensor, Wr: torch.Tensor, E: torch.Tensor,
                        W1: torch.Tensor, W2: torch.Tensor, dout: torch.Tensor, cache: torch.Tensor, n_distinct: int,
                        act: str = "gelu", dh=None, dWr=None, dE=None, dW1=None, dW2=None, stream=None):
    """Adds this layer's gradients of sum(out * dout) into the fp32 buffers
    given (see mole.h); returns them."""
    _contig(ids, groups, h, Wr, E, W1, W2, dout, cache, dh, dWr, dE, dW1, dW2)
    V, D = E.shape
    N, _, Dr = W1.shape
    T = ids.numel()
    _ok(lib.mole_train_backward(_ptr(ids), T, _ptr(groups), groups.numel(), _ptr(h), _ptr(Wr), _ptr(E), _ptr(W1),
                                _ptr(W2), V, N, D, Dr, ACT[act], _ptr(dout), _ptr(cache), cache.numel(), n_distinct,
                                _ptr(dh), _ptr(dWr), _ptr(dE), _ptr(dW1), _ptr(dW2), _stream(stream)),
        "mole_train_backward")
    return dh, dWr, dE, dW1, dW2


def mole_nf3_levels():
    buf = (ctypes.c_uint16 * 8)()
    lib.mole_nf3_levels(ctypes.cast(buf, ctypes.c_void_p))
    return list(buf)


def mole_nf3_midpoints():
    buf = (ctypes.c_float * 7)()
    lib.mole_nf3_midpoints(ctypes.cast(buf, ctypes.c_void_p))
    return list(buf)


def mole_gather_plan(ids: torch.Tensor, V: int, stream=None):
    """(uniq[:n], slot) of a batch's ids (see mole.h).  Synchronises to read n."""
    _contig(ids)
    T = ids.numel()
    uniq = torch.empty(max(T, 1), dtype=torch.int32, device=ids.device)
    slot = torch.empty(max(T, 1), dtype=torch.int32, device=ids.device)
    n = torch.zeros(1, dtype=torch.int32, device=ids.device)
    _ok(lib.mole_gather_plan(_ptr(ids), T, V, _ptr(uniq), _ptr(n), _ptr(slot), _stream(stream)),
        "mole_gather_plan")
    k = int(n.item())
    return uniq[:k], slot[:T]


def mole_prefetch_rows(ids: torch.Tensor, tables, stream=None) -> None:
    """L2 prefetch of the rows of `tables` (device tensors of V rows each:
    bf16 [V, N, D] tables, NF3 code [V, N, D/64, 24] and scale [V, N, D/64]
    arrays) that the step's `ids` address (see mole.h)."""
    _contig(ids, *tables)
    tables = list(tables)
    if not tables:
        return
    V = tables[0].shape[0]
    row_bytes = tables[0].numel() // V * tables[0].element_size()
    for t in tables:
        if t.shape[0] != V or t.numel() // V * t.element_size() != row_bytes:
            raise ValueError("mole_prefetch_rows: tables of one call share V and the row size")
    arr = (ctypes.c_void_p * len(tables))(*[t.data_ptr() for t in tables])
    _ok(lib.mole_prefetch_rows(_ptr(ids), ids.numel(), arr, len(tables), V, row_bytes, _stream(stream)),
        "mole_prefetch_rows")


# ---- Around the layer in a training step (see mole.h) ----
# These calls check shapes, types and devices, and run on the device that holds
# their tensors: `stream` (default: that device's current stream) gets the
# kernels, and what the call allocates for itself is allocated for that stream.
# Their checks are written for few Python operations: a small call is bound by
# its host time.

@contextlib.contextmanager
def _on_stream(stream, dev: torch.device):
    """The device and `stream` (if any) made current."""
    with torch.cuda.device(dev):
        if stream is None:
            yield
            return
        if not isinstance(stream, torch.cuda.Stream):
            handle = int(stream)
            if handle == 2:  # cudaStreamPerThread: torch allocates nothing for it
                raise ValueError("the per-thread default stream is not supported, pass a stream")
            # 0 and cudaStreamLegacy (ExternalStream takes 0 for "any stream of the pool")
            stream = (torch.cuda.default_stream(dev) if handle in (0, 1)
                      else torch.cuda.ExternalStream(handle, device=dev))
        if stream.device != dev:
            raise ValueError(f"stream of {stream.device}, tensors on {dev}")
        with torch.cuda.stream(stream):
            yield


def _elsewhere(stream, dev: int) -> bool:
    """Whether a call has to make another stream or device current first."""
    return stream is not None or torch._C._cuda_getDevice() != dev


def _device_of(name: str, t: torch.Tensor) -> int:
    at = t.get_device()
    if at < 0:
        raise ValueError(f"{name} is on {t.device}, expected a CUDA device, the same for all tensors")
    return at


def _expect(name: str, t, dev: int, shape=None, dtypes=None) -> None:
    """A tensor argument's device, layout, shape and type (None passes)."""
    if t is None:
        return
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected a CUDA device, the same for all tensors")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")


_ROWS = (torch.float32, torch.bfloat16)
_FP32 = (torch.float32,)
_INT32 = (torch.int32,)
_DT = {torch.float32: F32, torch.bfloat16: BF16}


def mole_embed_forward(ids: torch.Tensor, E: torch.Tensor, scale: float = 1.0, out: torch.Tensor | None = None,
                       out_dtype=None, stream=None) -> torch.Tensor:
    """out[t] = scale * E[ids[t]] (fp32 or bf16; out in E's type unless asked otherwise)."""
    dev = _device_of("E", E)
    if _elsewhere(stream, dev):
        with _on_stream(stream, E.device):
            return mole_embed_forward(ids, E, scale, out, out_dtype)
    T = ids.numel()
    V, D = E.shape
    _expect("E", E, dev, None, _ROWS)
    _expect("ids", ids, dev, None, _INT32)
    if out is None:
        out = torch.empty((T, D), dtype=out_dtype or E.dtype, device=E.device)
        if out.dtype not in _DT:
            raise TypeError(f"out_dtype is {out_dtype}")
    else:
        _expect("out", out, dev, (T, D), _ROWS if out_dtype is None else (out_dtype,))
    _ok(lib.mole_embed_forward(ids.data_ptr(), T, E.data_ptr(), V, D, scale, _DT[E.dtype], out.data_ptr(),
                               _DT[out.dtype], torch._C._cuda_getCurrentRawStream(dev)), "mole_embed_forward")
    return out


def mole_embed_backward_workspace(T: int, D: int) -> int:
    return int(lib.mole_embed_backward_workspace(T, D))


def mole_embed_backward(ids: torch.Tensor, dout: torch.Tensor, dE: torch.Tensor, scale: float = 1.0,
                        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dE[ids[t]] += scale * dout[t] (dE fp32; the same bits on every run); returns dE."""
    dev = _device_of("dE", dE)
    if _elsewhere(stream, dev):
        with _on_stream(stream, dE.device):
            return mole_embed_backward(ids, dout, dE, scale, workspace)
    T = ids.numel()
    V, D = dE.shape
    _expect("dE", dE, dev, None, _FP32)
    _expect("ids", ids, dev, None, _INT32)
    _expect("dout", dout, dev, (T, D), _ROWS)
    if workspace is None:
        nbytes = lib.mole_embed_backward_workspace(T, D)
        workspace = torch.empty(max(1, nbytes), dtype=torch.uint8, device=dE.device)
    else:
        _expect("workspace", workspace, dev)
        nbytes = workspace.numel() * workspace.element_size()
    _ok(lib.mole_embed_backward(ids.data_ptr(), T, dout.data_ptr(), _DT[dout.dtype], V, D, scale, dE.data_ptr(),
                                workspace.data_ptr(), nbytes, torch._C._cuda_getCurrentRawStream(dev)),
        "mole_embed_backward")
    return dE


def mole_block_norm_forward(x: torch.Tensor, f: torch.Tensor | None = None, w_post: torch.Tensor | None = None,
                            gate: torch.Tensor | None = None, res_scale: float = 1.0,
                            w_pre: torch.Tensor | None = None, eps: float = 1e-6, x_out: torch.Tensor | None = None,
                            h: torch.Tensor | None = None, h_dtype=torch.bfloat16, stream=None):
    """(x', h): x' = res_scale x + gate w_post f / rms(f), h = w_pre x' / rms(x').

    x' is made where f is given or res_scale is not 1 (or x_out is passed;
    x_out may be x), else it is x itself; h is made where w_pre is given, else
    None.
    """
    dev = _device_of("x", x)
    if _elsewhere(stream, dev):
        with _on_stream(stream, x.device):
            return mole_block_norm_forward(x, f, w_post, gate, res_scale, w_pre, eps, x_out, h, h_dtype)
    T, D = shape = x.shape
    _expect("x", x, dev, None, _ROWS)
    _expect("f", f, dev, shape, _ROWS)
    _expect("w_post", w_post, dev, (D,), _FP32)
    _expect("gate", gate, dev, (T,), _FP32)
    _expect("w_pre", w_pre, dev, (D,), _FP32)
    _expect("x_out", x_out, dev, shape, (x.dtype,))
    _expect("h", h, dev, shape, _ROWS)
    if x_out is None and (f is not None or res_scale != 1.0):
        x_out = torch.empty_like(x)
    if h is None and w_pre is not None:
        if h_dtype not in _DT:
            raise TypeError(f"h_dtype is {h_dtype}")
        h = torch.empty_like(x, dtype=h_dtype)
    _ok(lib.mole_block_norm_forward(x.data_ptr(), _DT[x.dtype], _ptr(f), F32 if f is None else _DT[f.dtype],
                                    _ptr(w_post), _ptr(gate), res_scale, _ptr(w_pre), eps, T, D, _ptr(x_out),
                                    _ptr(h), BF16 if h is None else _DT[h.dtype],
                                    torch._C._cuda_getCurrentRawStream(dev)), "mole_block_norm_forward")
    return (x if x_out is None else x_out), h


def mole_block_norm_backward_workspace(T: int, D: int) -> int:
    return int(lib.mole_block_norm_backward_workspace(T, D))


def mole_block_norm_backward(x_out: torch.Tensor, dx_out: torch.Tensor | None, dh: torch.Tensor | None,
                             f: torch.Tensor | None = None, w_post: torch.Tensor | None = None,
                             gate: torch.Tensor | None = None, res_scale: float = 1.0,
                             w_pre: torch.Tensor | None = None, eps: float = 1e-6, dx: torch.Tensor | None = None,
                             df: torch.Tensor | None = None, dgate: torch.Tensor | None = None,
                             dw_post: torch.Tensor | None = None, dw_pre: torch.Tensor | None = None,
                             workspace: torch.Tensor | None = None, stream=None):
    """(dx, df, dgate) of mole_block_norm_forward from the gradients of its two
    outputs; dw_post and dw_pre are added to where given.  df is made where f
    is given, dgate where f and gate are; with a post-norm left out, df needs no
    f and is written where it is passed."""
    dev = _device_of("x_out", x_out)
    if _elsewhere(stream, dev):
        with _on_stream(stream, x_out.device):
            return mole_block_norm_backward(x_out, dx_out, dh, f, w_post, gate, res_scale, w_pre, eps, dx, df, dgate,
                                            dw_post, dw_pre, workspace)
    T, D = shape = x_out.shape
    per_column = (D,)
    _expect("x_out", x_out, dev, None, _ROWS)
    _expect("f", f, dev, shape, _ROWS)
    _expect("dx_out", dx_out, dev, shape, _FP32)
    _expect("dh", dh, dev, shape, _FP32)
    _expect("w_post", w_post, dev, per_column, _FP32)
    _expect("w_pre", w_pre, dev, per_column, _FP32)
    _expect("dw_post", dw_post, dev, per_column, _FP32)
    _expect("dw_pre", dw_pre, dev, per_column, _FP32)
    _expect("gate", gate, dev, (T,), _FP32)
    _expect("dgate", dgate, dev, (T,), _FP32)
    _expect("dx", dx, dev, shape, _FP32)
    _expect("df", df, dev, shape, _FP32)
    _expect("workspace", workspace, dev)
    if dx is None:
        dx = torch.empty_like(x_out, dtype=torch.float32)
    if df is None and f is not None:
        df = torch.empty_like(x_out, dtype=torch.float32)
    if dgate is None and gate is not None and f is not None:
        dgate = torch.empty_like(gate)
    nbytes = 0
    if workspace is not None:
        nbytes = workspace.numel() * workspace.element_size()
    elif dw_post is not None or dw_pre is not None:
        nbytes = lib.mole_block_norm_backward_workspace(T, D)
        workspace = torch.empty(max(1, nbytes), dtype=torch.uint8, device=x_out.device)
    _ok(lib.mole_block_norm_backward(x_out.data_ptr(), _DT[x_out.dtype], _ptr(f), F32 if f is None else _DT[f.dtype],
                                     _ptr(w_post), _ptr(gate), res_scale, _ptr(w_pre), eps, T, D, _ptr(dx_out),
                                     _ptr(dh), dx.data_ptr(), _ptr(df), _ptr(dgate), _ptr(dw_post), _ptr(dw_pre),
                                     _ptr(workspace), nbytes, torch._C._cuda_getCurrentRawStream(dev)),
        "mole_block_norm_backward")
    return dx, df, dgate


class AdamWTensor(ctypes.Structure):
    """mole_adamw_tensor of mole.h."""
    _fields_ = [("param", _P), ("grad", _P), ("master", _P), ("m", _P), ("v", _P), ("m_scale", _P), ("v_scale", _P),
                ("n", _I64), ("weight_decay", _F), ("dt_param", _I32), ("dt_grad", _I32)]


class AdamWConfig(ctypes.Structure):
    """mole_adamw_config of mole.h."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", _I64), ("step_dev", _P), ("lr_dev", _P), ("grad_scale_dev", _P),
                ("state8", _I32)]


ADAMW_BLOCK = 128  # elements per scale of an 8-bit state
_ADAMW_TENSOR = struct.Struct("@7Pqfii4x")  # AdamWTensor's layout
_DTYPE = operator.attrgetter("dtype")
assert _ADAMW_TENSOR.size == ctypes.sizeof(AdamWTensor)


def _addresses(name: str, tensors, sizes, dev: int, dtypes, optional=False):
    """The tensors' addresses (0 for None, where allowed), all of them checked
    at once: a list of small tensors costs its user host time."""
    if optional:
        given = [(t, k) for t, k in zip(tensors, sizes) if t is not None]
        tensors_given, sizes = [t for t, _ in given], [k for _, k in given]
    else:
        tensors_given = tensors
    of = torch.Tensor
    if (list(map(of.numel, tensors_given)) != sizes or not {dev}.issuperset(map(of.get_device, tensors_given))
            or not set(dtypes).issuperset(map(_DTYPE, tensors_given)) or not all(map(of.is_contiguous, tensors_given))):
        for i, (t, k) in enumerate(zip(tensors_given, sizes)):  # which one, and why
            _expect(f"{name}[{i}]", t, dev, None, dtypes)
            if t.numel() != k:
                raise ValueError(f"{name}[{i}] has {t.numel()} elements, expected {k}")
    if optional:
        return [0 if t is None else t.data_ptr() for t in tensors]
    return map(of.data_ptr, tensors)


def mole_adamw_step(params, grads, ms, vs, masters=None, m_scales=None, v_scales=None, weight_decay=0.0,
                    lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, step=1,
                    lr_dev: torch.Tensor | None = None, grad_scale: torch.Tensor | None = None, stream=None) -> None:
    """One AdamW step over the tensors of `params` (fp32 or bf16; lists of
    equal length, tensors of equal numbers of elements; see mole.h).  ms and vs
    are fp32, or torch.float8_e4m3fn with m_scales and v_scales (fp32, one
    value per 128 elements).  masters: fp32 weights of the bf16 params (a list,
    entries may be None).  weight_decay: a number or one per tensor.  step: the step's number from 1, or a device
    int64 tensor that holds it; lr_dev (device fp32) replaces lr, grad_scale
    (device fp32) multiplies every gradient."""
    params, grads, ms, vs = list(params), list(grads), list(ms), list(vs)
    n = len(params)
    none = [0] * n
    masters = none if masters is None else list(masters)
    m_scales = none if m_scales is None else list(m_scales)
    v_scales = none if v_scales is None else list(v_scales)
    decay = [weight_decay] * n if isinstance(weight_decay, (int, float)) else list(weight_decay)
    if any(len(x) != n for x in (grads, ms, vs, masters, m_scales, v_scales, decay)):
        raise ValueError("lists of different lengths")
    if n == 0:
        return
    state8 = ms[0].dtype == torch.float8_e4m3fn
    states = (torch.float8_e4m3fn,) if state8 else _FP32
    if state8 != (m_scales is not none) or state8 != (v_scales is not none):
        raise ValueError("m_scales and v_scales belong to 8-bit states, and 8-bit states need them")
    dev = _device_of("params[0]", params[0])
    if _elsewhere(stream, dev):
        with _on_stream(stream, params[0].device):
            return mole_adamw_step(params, grads, ms, vs, masters if masters is not none else None,
                                   m_scales if m_scales is not none else None,
                                   v_scales if v_scales is not none else None, decay, lr, beta1, beta2, eps, step,
                                   lr_dev, grad_scale)
    sizes = list(map(torch.Tensor.numel, params))
    blocks = [(k + ADAMW_BLOCK - 1) // ADAMW_BLOCK for k in sizes] if state8 else None
    table = zip(_addresses("params", params, sizes, dev, _ROWS), _addresses("grads", grads, sizes, dev, _ROWS),
                masters if masters is none else _addresses("masters", masters, sizes, dev, _FP32, optional=True),
                _addresses("ms", ms, sizes, dev, states), _addresses("vs", vs, sizes, dev, states),
                _addresses("m_scales", m_scales, blocks, dev, _FP32) if state8 else none,
                _addresses("v_scales", v_scales, blocks, dev, _FP32) if state8 else none,
                sizes, decay, map(_DT.__getitem__, map(_DTYPE, params)),
                map(_DT.__getitem__, map(_DTYPE, grads)))
    arr = b"".join(itertools.starmap(_ADAMW_TENSOR.pack, table))
    cfg = AdamWConfig(lr=lr, beta1=beta1, beta2=beta2, eps=eps, state8=int(state8))
    if isinstance(step, torch.Tensor):
        _expect("step", step.view(-1), dev, (1,), (torch.int64,))
        cfg.step_dev = step.data_ptr()
    else:
        cfg.step = step
    for name, t, field in (("lr_dev", lr_dev, "lr_dev"), ("grad_scale", grad_scale, "grad_scale_dev")):
        if t is not None:
            _expect(name, t.view(-1), dev, (1,), _FP32)
            setattr(cfg, field, t.data_ptr())
    _ok(lib.mole_adamw_step(arr, n, ctypes.addressof(cfg), torch._C._cuda_getCurrentRawStream(dev)),
        "mole_adamw_step")


def mole_check(stream=None, timeout_ms: int = 10000) -> int:
    """Drain the stream (bounded) and return the device error status (0 = ok)."""
    return int(lib.mole_check(_stream(stream), timeout_ms))
