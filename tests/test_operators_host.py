"""Host-only checks of the norm and adapter entry points: every call below is refused
during argument validation, before anything touches a GPU."""
import ctypes

import pytest

from post_quantized_linear_b200 import _lib

L = _lib
FAKE = 1 << 20          # a 16-byte aligned, never dereferenced address


def _seg(bounds):
    s, keep = L.segments(bounds)
    return s, keep


def norm(x=FAKE, xt=L.SQ_BF16, B=2, S=9, C=64, ldx=64, xbs=576, groups=8, gamma=FAKE, beta=FAKE, eps=1e-5,
         act=1, y=FAKE, yt=L.SQ_BF16, ldy=64, ybs=576, ws=None, wn=0, stats=None):
    return L.load().sq_group_norm_act(x, xt, B, S, C, ldx, xbs, groups, gamma, beta, eps, act, y, yt, ldy, ybs,
                                      stats, ws, wn, None)


def test_norm_refusals():
    assert norm(x=None) == L.SQ_ERR_INVALID_ARG
    assert norm(y=None) == L.SQ_ERR_INVALID_ARG
    assert norm(xt=5) == L.SQ_ERR_INVALID_ARG
    assert norm(yt=5) == L.SQ_ERR_INVALID_ARG
    assert norm(B=-1) == L.SQ_ERR_INVALID_ARG
    assert norm(groups=0) == L.SQ_ERR_INVALID_ARG
    assert norm(groups=7) == L.SQ_ERR_INVALID_ARG
    assert norm(act=3) == L.SQ_ERR_INVALID_ARG
    assert norm(act=-1) == L.SQ_ERR_INVALID_ARG
    assert norm(eps=-1.0) == L.SQ_ERR_INVALID_ARG
    assert norm(eps=float("nan")) == L.SQ_ERR_INVALID_ARG
    assert norm(ldx=63) == L.SQ_ERR_INVALID_ARG
    assert norm(ldy=32) == L.SQ_ERR_INVALID_ARG
    assert norm(C=60, groups=4) == L.SQ_ERR_UNSUPPORTED
    assert norm(C=8192, groups=1, ldx=8192, ldy=8192) == L.SQ_ERR_UNSUPPORTED      # a group wider than 8192 bytes
    assert norm(B=70000) == L.SQ_ERR_RANGE
    assert norm(S=(1 << 30) + 1) == L.SQ_ERR_RANGE
    assert norm(C=L.SQ_MAX_K + 8, groups=1) == L.SQ_ERR_RANGE
    assert norm(x=FAKE + 2) == L.SQ_ERR_ALIGNMENT
    assert norm(ldx=68) == L.SQ_ERR_ALIGNMENT
    assert norm(xbs=580) == L.SQ_ERR_ALIGNMENT
    assert norm(ldy=66) == L.SQ_ERR_ALIGNMENT
    assert norm(B=1, S=300000, xbs=0, ybs=0) == L.SQ_ERR_INVALID_ARG               # needs a workspace
    assert norm(B=0) == L.SQ_OK and norm(S=0, x=None, y=None) == L.SQ_OK


def test_norm_workspace_size():
    def size(*a):
        n = ctypes.c_size_t(77)
        return L.load().sq_group_norm_workspace_size(*a, ctypes.byref(n)), n.value
    assert size(2, 64, 1280, 32, L.SQ_BF16, 0) == (L.SQ_OK, 0)
    assert size(0, 64, 1280, 32, L.SQ_BF16, 1) == (L.SQ_OK, 0)
    st, n = size(2, 64, 1280, 32, L.SQ_BF16, 1)
    assert st == L.SQ_OK and n == 2 * 4 * 2 * 1280
    st, n = size(1, 300000, 64, 8, L.SQ_F32, 0)
    assert st == L.SQ_OK and n > 0 and n % (8 * 8) == 0
    assert size(2, 64, 1281, 32, L.SQ_BF16, 0)[0] == L.SQ_ERR_INVALID_ARG
    assert size(2, 64, 1280, 32, 9, 0)[0] == L.SQ_ERR_INVALID_ARG
    assert L.load().sq_group_norm_workspace_size(2, 64, 1280, 32, 0, 0, None) == L.SQ_ERR_INVALID_ARG


def codes(kb=(0, 64), C=64, c=FAKE, n=FAKE, ldc=64, sp=FAKE, sn=FAKE, y=None, ldy=64, groups=8, ldx=64):
    s, keep = _seg(kb)
    return L.load().sq_quantize_activations_norm(FAKE, L.SQ_BF16, 2, 9, C, ldx, 9 * ldx, groups, None, None,
                                                          1e-5, 0, ctypes.byref(s), sp, sn, c, n, ldc, y, ldy, None, 0,
                                                          None)


def test_norm_codes_refusals():
    assert codes(c=None) == L.SQ_ERR_INVALID_ARG
    assert codes(n=None) == L.SQ_ERR_INVALID_ARG
    assert codes(n=FAKE + 8) == L.SQ_ERR_ALIGNMENT
    assert codes(sp=None) == L.SQ_ERR_INVALID_ARG
    assert codes(ldc=48) == L.SQ_ERR_INVALID_ARG
    assert codes(ldc=72) == L.SQ_ERR_ALIGNMENT
    assert codes(c=FAKE + 8) == L.SQ_ERR_ALIGNMENT
    assert codes(kb=(0, 32)) == L.SQ_ERR_INVALID_ARG
    assert codes(kb=(0, 32, 64)) == L.SQ_ERR_UNSUPPORTED
    assert codes(C=72, kb=(0, 72), ldc=80, ldx=72) == L.SQ_ERR_UNSUPPORTED
    assert codes(y=FAKE, ldy=60) == L.SQ_ERR_INVALID_ARG


def norm_bwd(dy=FAKE, x=FAKE, stats=FAKE, dx=FAKE, ws=FAKE, wn=1 << 30, act=2, lddy=64, groups=8, C=64):
    return L.load().sq_group_norm_act_backward(dy, lddy, 9 * lddy, x, L.SQ_F32, 2, 9, C, 64, 576, groups, stats,
                                               None, None, act, dx, 64, 576, None, None, ws, wn, None)


def test_norm_backward_refusals():
    for k in ("dy", "x", "stats", "dx", "ws"):
        assert norm_bwd(**{k: None}) == L.SQ_ERR_INVALID_ARG
    assert norm_bwd(wn=100) == L.SQ_ERR_INVALID_ARG
    assert norm_bwd(act=9) == L.SQ_ERR_INVALID_ARG
    assert norm_bwd(lddy=66) == L.SQ_ERR_ALIGNMENT
    assert norm_bwd(ws=FAKE + 4) == L.SQ_ERR_ALIGNMENT
    assert norm_bwd(dy=FAKE + 8) == L.SQ_ERR_ALIGNMENT
    assert norm_bwd(groups=5) == L.SQ_ERR_INVALID_ARG


def test_misaligned_and_overlapping_norm_arguments():
    # the backward reads the statistics in pairs: eight bytes; every other fp32 array takes four
    assert norm_bwd(stats=FAKE + 4) == L.SQ_ERR_ALIGNMENT
    assert norm(stats=FAKE + 2) == L.SQ_ERR_ALIGNMENT
    assert codes(sp=FAKE + 2) == L.SQ_ERR_ALIGNMENT
    # an input may repeat its image, an output not
    assert norm(ybs=0) == L.SQ_ERR_INVALID_ARG
    assert norm(ybs=32) == L.SQ_ERR_INVALID_ARG


def add(x=FAKE, xt=L.SQ_BF16, M=100, ldx=128, A=2, R=16, K=128, N=64, a=FAKE, b=FAKE, scale=None, bounds=FAKE,
        index=FAKE, Q=3, y=FAKE, yt=L.SQ_BF16, ldy=64, h=None):
    ad = L.SqAdapters(A, R, K, N, a, b, scale)
    return L.load().sq_adapter_add(x, xt, M, ldx, ctypes.byref(ad), bounds, index, Q, y, yt, ldy, h, None)


def test_adapter_refusals():
    for k in ("x", "y", "a", "b", "bounds", "index"):
        assert add(**{k: None}) == L.SQ_ERR_INVALID_ARG
    assert add(M=-1) == L.SQ_ERR_INVALID_ARG
    assert add(Q=-1) == L.SQ_ERR_INVALID_ARG
    assert add(A=0) == L.SQ_ERR_INVALID_ARG
    assert add(R=0) == L.SQ_ERR_INVALID_ARG
    assert add(xt=9) == L.SQ_ERR_INVALID_ARG
    assert add(ldx=120) == L.SQ_ERR_INVALID_ARG
    assert add(R=12) == L.SQ_ERR_UNSUPPORTED
    assert add(R=136) == L.SQ_ERR_UNSUPPORTED
    assert add(K=136, ldx=136) == L.SQ_ERR_UNSUPPORTED
    assert add(N=72, ldy=72) == L.SQ_ERR_UNSUPPORTED
    assert add(M=(1 << 30) + 1) == L.SQ_ERR_RANGE
    assert add(K=L.SQ_MAX_K + 16, ldx=L.SQ_MAX_K + 16) == L.SQ_ERR_RANGE
    assert add(A=65536) == L.SQ_ERR_RANGE
    assert add(Q=(1 << 24) + 1) == L.SQ_ERR_RANGE
    assert add(a=FAKE + 8) == L.SQ_ERR_ALIGNMENT
    assert add(x=FAKE + 8) == L.SQ_ERR_ALIGNMENT
    assert add(ldy=68) == L.SQ_ERR_ALIGNMENT
    assert add(bounds=FAKE + 2) == L.SQ_ERR_ALIGNMENT
    assert add(scale=FAKE + 2) == L.SQ_ERR_ALIGNMENT
    assert add(h=FAKE + 8) == L.SQ_ERR_ALIGNMENT
    assert add(M=0, x=None, y=None) == L.SQ_OK
    assert L.load().sq_adapter_add(FAKE, 1, 1, 128, None, FAKE, FAKE, 1, FAKE, 1, 64, None, None) == L.SQ_ERR_INVALID_ARG


def add_to(y=FAKE, ldy=64, out=FAKE, ldo=64, x=FAKE, M=100, h=None, bounds=FAKE):
    ad = L.SqAdapters(2, 16, 128, 64, FAKE, FAKE, None)
    return L.load().sq_adapter_add_to(x, L.SQ_BF16, M, 128, ctypes.byref(ad), bounds, FAKE, 3, y, ldy, out, ldo, h, None)


def test_adapter_output_of_its_own_refusals():
    for k in ("x", "y", "out", "bounds"):
        assert add_to(**{k: None}) == L.SQ_ERR_INVALID_ARG
    assert add_to(ldo=56) == L.SQ_ERR_INVALID_ARG
    assert add_to(ldo=68) == L.SQ_ERR_ALIGNMENT
    assert add_to(out=FAKE + 8) == L.SQ_ERR_ALIGNMENT
    assert add_to(ldy=66) == L.SQ_ERR_ALIGNMENT
    assert add_to(h=FAKE + 4) == L.SQ_ERR_ALIGNMENT
    assert add_to(M=-1) == L.SQ_ERR_INVALID_ARG
    assert add_to(M=0, out=None, y=None, x=None) == L.SQ_OK


def test_adapter_backward_request_limits():
    """A call that would walk more requests an adapter than this is refused, not run for minutes."""
    def many(Q, A):
        ad = L.SqAdapters(A, 16, 128, 64, FAKE, FAKE, None)
        return L.load().sq_adapter_backward(FAKE, L.SQ_BF16, 100, 64, FAKE, L.SQ_BF16, 128, FAKE, ctypes.byref(ad), FAKE,
                                            FAKE, Q, FAKE, 128, FAKE, FAKE, None, 0, None)
    assert many((1 << 20) + 1, 2) == L.SQ_ERR_RANGE
    assert many((1 << 16) + 1, 1 << 10) == L.SQ_ERR_RANGE
    assert many(1 << 20, 64) == L.SQ_ERR_INVALID_ARG             # accepted; the workspace is missing
    assert many(1 << 16, 1 << 10) == L.SQ_ERR_INVALID_ARG


def bwd(dy=FAKE, x=FAKE, h=FAKE, dx=FAKE, da=FAKE, db=FAKE, ws=FAKE, wn=1 << 30, lddx=128, R=16):
    ad = L.SqAdapters(2, R, 128, 64, FAKE, FAKE, None)
    return L.load().sq_adapter_backward(dy, L.SQ_BF16, 100, 64, x, L.SQ_BF16, 128, h, ctypes.byref(ad), FAKE, FAKE, 3,
                                        dx, lddx, da, db, ws, wn, None)


def test_adapter_backward_refusals():
    for k in ("dy", "x", "h", "dx", "da", "db", "ws"):
        assert bwd(**{k: None}) == L.SQ_ERR_INVALID_ARG
    assert bwd(wn=100 * 16 * 4 - 1) == L.SQ_ERR_INVALID_ARG
    assert bwd(lddx=132) == L.SQ_ERR_ALIGNMENT
    assert bwd(da=FAKE + 4) == L.SQ_ERR_ALIGNMENT
    assert bwd(R=20) == L.SQ_ERR_UNSUPPORTED
    n = ctypes.c_size_t()
    assert L.load().sq_adapter_backward_workspace_size(100, 16, ctypes.byref(n)) == L.SQ_OK and n.value >= 6400
    assert L.load().sq_adapter_backward_workspace_size(-1, 16, ctypes.byref(n)) == L.SQ_ERR_INVALID_ARG


class OtherTensor:
    """What the binding asks of a tensor, for checks that need a second device."""

    def __init__(self, shape, dtype, device):
        import torch
        self.shape, self.dtype, self.index, self.is_cuda, self.device = torch.Size(shape), dtype, device, True, device
        self.strides = [1]
        for n in reversed(shape[1:]):
            self.strides.insert(0, self.strides[0] * n)

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return tuple(self.strides) if i is None else self.strides[i]

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        raise AssertionError("a call went past its checks")


def test_binding_refuses_codes_on_another_device(monkeypatch):
    torch = pytest.importorskip("torch")
    import post_quantized_linear_b200 as pq
    monkeypatch.setattr(pq, "_current_device", lambda: 0)
    x, scale = OtherTensor((2, 9, 64), torch.bfloat16, 0), OtherTensor((1,), torch.float32, 0)
    here, there = (OtherTensor((18, 64), torch.int8, d) for d in (0, 1))
    for out in ((there, there), (here, there), (there, here)):
        with pytest.raises(ValueError, match="current CUDA device"):
            pq.quantize_activations_norm(x, 8, None, None, (0, 64), scale, scale, out=out)
    with pytest.raises(AssertionError, match="past its checks"):
        pq.quantize_activations_norm(x, 8, None, None, (0, 64), scale, scale, out=(here, here))


def test_binding_refuses_wrong_tensors():
    """The binding's own checks, on CPU tensors."""
    torch = pytest.importorskip("torch")
    import post_quantized_linear_b200 as pq
    x = torch.zeros(2, 9, 64)
    with pytest.raises(ValueError, match="CUDA"):
        pq.group_norm_act(x, 8)
    with pytest.raises(ValueError, match="3-D"):
        pq.group_norm_act(x[0], 8)
    with pytest.raises(ValueError, match="unit channel stride"):
        pq.group_norm_act(x.transpose(1, 2), 8)
    with pytest.raises(ValueError, match="bfloat16 CUDA"):
        pq.Adapters(torch.zeros(2, 8, 16), torch.zeros(2, 32, 8))
    with pytest.raises(ValueError, match=r"\[L, R, K\]"):
        pq.Adapters(torch.zeros(2, 8, 16), torch.zeros(2, 32, 16))
