"""CPU-only checks of the operators around the head: what the C entries and the
binding refuse, before any device is touched."""
import ctypes

import pytest
import torch

import linear_cross_entropy_fwd_gb300 as flce
from linear_cross_entropy_fwd_gb300 import build as flce_build


@pytest.fixture(scope="module")
def lib():
    flce_build.build()
    return flce.load_library()


A = 4096  # a non-null, aligned address; refused calls never read it


@pytest.mark.parametrize("kw,status", [
    (dict(W=None), flce.FLCE_ERR_ARG),
    (dict(ids=None), flce.FLCE_ERR_ARG),
    (dict(Y=None), flce.FLCE_ERR_ARG),
    (dict(N=-1), flce.FLCE_ERR_ARG),
    (dict(N=1 << 31), flce.FLCE_ERR_ARG),
    (dict(H=0), flce.FLCE_ERR_ARG),
    (dict(H=(1 << 20) + 8), flce.FLCE_ERR_ARG),
    (dict(V=0), flce.FLCE_ERR_ARG),
    (dict(V=1 << 31), flce.FLCE_ERR_ARG),
    (dict(scale=float("nan")), flce.FLCE_ERR_ARG),
    (dict(dtype=7), flce.FLCE_ERR_ARG),
    (dict(H=12), flce.FLCE_ERR_ALIGN),          # 24 bytes of bf16
    (dict(W=A + 8), flce.FLCE_ERR_ALIGN),
    (dict(Y=A + 2), flce.FLCE_ERR_ALIGN),
])
def test_embed_refusals(lib, kw, status):
    a = dict(W=A, ids=A, N=4, H=16, V=10, scale=1.0, Y=A, dtype=flce.FLCE_BF16)
    a.update(kw)
    o = flce.make_opts(sync=0)
    o.dtype = a["dtype"]
    assert lib.flce_embed_fwd(a["W"], a["ids"], a["N"], a["H"], a["V"], a["scale"], -100, a["Y"],
                              ctypes.byref(o)) == status
    assert lib.flce_last_error()
    assert lib.flce_embed_bwd(a["Y"], a["ids"], a["N"], a["H"], a["V"], a["scale"], -100, a["W"],
                              0, ctypes.byref(o)) == status


def test_embed_binding_refusals():
    W, ids = torch.zeros(5, 8), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):  # not on a device
        flce.flce_embed_fwd(W, ids)
    with pytest.raises(ValueError):
        flce.flce_embed_bwd(torch.zeros(3, 8), ids, 5)
