"""GPU tests of the linear head's cross entropy: the few-row forward on rows of
w that end inside a 16-byte access, and on both sides of its limits.

A logit is a sum of D binary32 products, 8 to a lane and step and a tree of 5
(tensor-core path: 16 to a truncating step of 2u, six products for binary32):
(D / 2 + 64) u of the sum of the terms' sizes, u = 2^-24.  lse adds the
exponentials' 2^-21, their arguments' 4u (|l| + |lse|) and 64u.
"""
import ctypes
import json

import pytest
import torch

import broadcast_elementwise_shape_gb300 as zr
from broadcast_elementwise_shape_gb300 import ZrTensor, _i64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    zr.build()
    zr.lib()


def kernel(x, w, y):
    """The kernel that the forward's plan names."""
    L, buf, keep = zr.lib(), ctypes.create_string_buffer(1024), []

    def desc(t):
        keep.append((_i64(t.shape), _i64(t.stride())))
        return ZrTensor(t.data_ptr(), t.dim(), *keep[-1])

    L.zr_test_describe_linear_xent.argtypes = [ctypes.c_int, ZrTensor, ZrTensor, ctypes.c_int, ZrTensor,
                                               ctypes.c_int, ctypes.c_char_p, ctypes.c_size_t]
    dt = 0 if x.dtype == torch.float32 else 1
    assert L.zr_test_describe_linear_xent(dt, desc(x), desc(w), 1, desc(y), 0, buf, 1024) == 0
    return json.loads(buf.value)["kernel"]


def check(x, w, y):
    loss, lse = zr.zr_linear_xent_fwd(x, w, y, "none")
    l = x.double() @ w.double().t()
    lerr = ((x.shape[1] / 2 + 64) * U * (x.double().abs() @ w.double().abs().t())).max(1).values
    want = torch.logsumexp(l, 1)
    at = l.gather(1, y[:, None])[:, 0]
    size = l.abs().max(1).values + want.abs()
    bound = lerr + 2.0 ** -21 + 4 * U * size + 64 * U
    assert bool(((lse.double() - want).abs() <= bound).all())
    assert bool(((loss.double() - (want - at)).abs() <= bound + lerr + 4 * U * size).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [1, 2, 4, 16])
def test_rows_that_end_inside_an_access(N, dtype):
    g = torch.Generator("cuda").manual_seed(N)
    for D, pitch in ((1, 8), (3, 8), (7, 8), (9, 16), (130, 136), (257, 264), (1001, 1024), (2999, 3000)):
        w = torch.randn(77, pitch, generator=g, device="cuda").to(dtype)[:, :D]
        x = torch.randn(N, D, generator=g, device="cuda").to(dtype)
        y = torch.randint(0, 77, (N,), generator=g, device="cuda")
        assert kernel(x, w, y) == ("xent_few" if N <= 4 or dtype == torch.float32 else "xent")
        # What lies past a row's end is not read into it.
        w._base[:, D:] = float("nan")
        check(x, w, y)


@pytest.mark.parametrize("dtype,N,D,few", [(torch.float32, 16, 6144, True), (torch.float32, 16, 6148, False),
                                           (torch.float32, 4, 12288, True), (torch.float32, 4, 12292, False),
                                           (torch.float32, 2, 24576, True), (torch.float32, 2, 24580, False),
                                           (torch.float32, 1, 49152, True), (torch.float32, 1, 49156, False),
                                           (torch.float32, 9, 6144, True), (torch.float32, 17, 64, False),
                                           (torch.bfloat16, 4, 12288, True), (torch.bfloat16, 4, 12296, False),
                                           (torch.bfloat16, 1, 49152, True), (torch.bfloat16, 1, 49160, False)])
def test_around_the_shared_memory_limit(dtype, N, D, few):
    """Widths that w's rows allow on both sides of what x may take in shared memory."""
    g = torch.Generator("cuda").manual_seed(D)
    w = (torch.randn(301, D, generator=g, device="cuda") / D ** 0.5).to(dtype)
    x = torch.randn(N, D, generator=g, device="cuda").to(dtype)
    y = torch.randint(0, 301, (N,), generator=g, device="cuda")
    assert kernel(x, w, y) == ("xent_few" if few else "xent")
    check(x, w, y)
