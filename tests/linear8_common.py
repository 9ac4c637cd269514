"""ctypes view of include/muon_linear8.h for the tests."""
import ctypes

import torch

from matrix_aware_optimizer_muon_amd._lib import load

EXPORTED = ("muon_rmsnorm_forward", "muon_rmsnorm_backward_workspace", "muon_rmsnorm_backward",
            "muon_q8_quantize", "muon_q8_dequantize", "muon_q8_workspace", "muon_q8_matmul",
            "muon_q8_grad_input", "muon_q8_grad_weight")
MATMUL, GRAD_INPUT, GRAD_WEIGHT = 0, 1, 2
CODE = {torch.float32: 0, torch.bfloat16: 1}


def abi():
    lib = load()
    P, I, L, S, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sig = {
        "muon_rmsnorm_forward": [P, L, P, L, P, I, L, L, F, P, L, P, L, P, L, P, P, P],
        "muon_rmsnorm_backward_workspace": [L, L, P],
        "muon_rmsnorm_backward": [P, L, P, L, P, P, P, P, L, I, L, L, P, L, P, P, S, P],
        "muon_q8_quantize": [P, L, I, L, L, P, L, P, P],
        "muon_q8_dequantize": [P, L, P, L, L, P, L, I, P],
        "muon_q8_workspace": [I, P, L, P, L, L, L, L, P],
        "muon_q8_matmul": [P, L, P, P, L, P, L, L, L, P, L, I, P, S, P],
        "muon_q8_grad_input": [P, L, P, L, P, L, L, L, P, L, I, P, S, P],
        "muon_q8_grad_weight": [P, L, P, L, P, L, L, L, P, L, I, I, P, S, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, ctypes.c_int
    return lib


def workspace(kind, a, lda, b, ldb, t, n, k):
    z = ctypes.c_size_t()
    assert abi().muon_q8_workspace(kind, a, lda, b, ldb, t, n, k, ctypes.addressof(z)) == 0
    return z.value


def back_workspace(rows, cols):
    z = ctypes.c_size_t()
    assert abi().muon_rmsnorm_backward_workspace(rows, cols, ctypes.addressof(z)) == 0
    return z.value


def ld(t):
    return max(t.stride(0), t.shape[1])


def product(kind, a, a_scale, b, b_scale, out, accumulate=False):
    """One product into `out` (any row distance), with a workspace of exactly
    the asked size between guard bytes, which are checked."""
    t = a.shape[0]
    k = b.shape[1]
    n = b.shape[0] if kind == MATMUL else a.shape[1]
    need = workspace(kind, a.data_ptr(), ld(a), b.data_ptr(), ld(b), t, n, k)
    ws = torch.full((need + 512,), 0xa5, dtype=torch.uint8, device=a.device)
    at = ws.data_ptr() + 256
    s = torch.cuda.current_stream().cuda_stream
    f = abi()
    code = CODE[out.dtype]
    if kind == MATMUL:
        st = f.muon_q8_matmul(a.data_ptr(), ld(a), a_scale.data_ptr(), b.data_ptr(), ld(b), b_scale.data_ptr(),
                              t, n, k, out.data_ptr(), ld(out), code, at, need, s)
    elif kind == GRAD_INPUT:
        st = f.muon_q8_grad_input(a.data_ptr(), ld(a), b.data_ptr(), ld(b), b_scale.data_ptr(), t, n, k,
                                  out.data_ptr(), ld(out), code, at, need, s)
    else:
        st = f.muon_q8_grad_weight(a.data_ptr(), ld(a), b.data_ptr(), ld(b), b_scale.data_ptr(), t, n, k,
                                   out.data_ptr(), ld(out), code, int(accumulate), at, need, s)
    assert st == 0
    torch.cuda.synchronize()
    assert bool((ws[:256] == 0xa5).all()) and bool((ws[256 + need:] == 0xa5).all())
