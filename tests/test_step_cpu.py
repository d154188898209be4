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


def _attn(**kw):
    """A flce_attn that no check refuses, with some fields replaced."""
    a = flce.FlceAttn()
    f = dict(T=300, batch=2, cu_seqlens=A, heads_q=4, heads_kv=2, head_dim=64, scale=0.125, lse=A)
    for n, h in (("q", 4), ("k", 2), ("v", 2), ("o", 4), ("dO", 4), ("dq", 4), ("dk", 2),
                 ("dv", 2)):
        f.update({n: A, n + "_token": 64 * h, n + "_head": 64})
    f.update(kw)
    for n, x in f.items():
        setattr(a, n, x)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), flce.FLCE_ERR_ARG),
    (dict(T=(1 << 31) - 256), flce.FLCE_ERR_ARG),
    (dict(batch=-1), flce.FLCE_ERR_ARG),
    (dict(batch=1 << 29), flce.FLCE_ERR_ARG),        # too many CTAs
    (dict(cu_seqlens=None), flce.FLCE_ERR_ARG),
    (dict(heads_q=3), flce.FLCE_ERR_ARG),
    (dict(heads_kv=0), flce.FLCE_ERR_ARG),
    (dict(head_dim=0), flce.FLCE_ERR_ARG),
    (dict(head_dim=68), flce.FLCE_ERR_ARG),
    (dict(head_dim=136), flce.FLCE_ERR_ARG),
    (dict(scale=0.0), flce.FLCE_ERR_ARG),
    (dict(scale=float("inf")), flce.FLCE_ERR_ARG),
    (dict(scale=float("nan")), flce.FLCE_ERR_ARG),
    (dict(q=None), flce.FLCE_ERR_ARG),
    (dict(o=None), flce.FLCE_ERR_ARG),
    (dict(lse=None), flce.FLCE_ERR_ARG),
    (dict(k_token=0), flce.FLCE_ERR_ARG),
    (dict(k_head=0), flce.FLCE_ERR_ARG),
    (dict(v_head=-64), flce.FLCE_ERR_ARG),
    (dict(v_token=132), flce.FLCE_ERR_ALIGN),
    (dict(k=A + 8), flce.FLCE_ERR_ALIGN),
])
def test_attention_refusals(lib, kw, status):
    o = flce.make_opts(sync=0)
    for fn in (lib.flce_attn_fwd, lib.flce_attn_bwd):
        assert fn(ctypes.byref(_attn(**kw)), ctypes.byref(o)) == status
        assert lib.flce_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dO=None), flce.FLCE_ERR_ARG),
    (dict(dq=None), flce.FLCE_ERR_ARG),
    (dict(dk_head=0), flce.FLCE_ERR_ARG),
    (dict(dv=A + 4), flce.FLCE_ERR_ALIGN),
])
def test_attention_gradient_refusals(lib, kw, status):
    o = flce.make_opts(sync=0)
    assert lib.flce_attn_bwd(ctypes.byref(_attn(**kw)), ctypes.byref(o)) == status


def test_attention_refuses_other_types(lib):
    o = flce.make_opts(sync=0)
    o.dtype = flce.FLCE_FP32
    assert lib.flce_attn_fwd(ctypes.byref(_attn()), ctypes.byref(o)) == flce.FLCE_ERR_ARG
    assert lib.flce_attn_fwd(None, None) == flce.FLCE_ERR_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(G=None), flce.FLCE_ERR_ARG),
    (dict(out=None), flce.FLCE_ERR_ARG),
    (dict(batch=-1), flce.FLCE_ERR_ARG),
    (dict(batch=65536), flce.FLCE_ERR_ARG),
    (dict(rows=-1), flce.FLCE_ERR_ARG),
    (dict(cols=(1 << 20) + 1), flce.FLCE_ERR_ARG),
    (dict(steps=0), flce.FLCE_ERR_ARG),
    (dict(steps=65), flce.FLCE_ERR_ARG),
    (dict(eps=-1e-3), flce.FLCE_ERR_ARG),
    (dict(eps=float("nan")), flce.FLCE_ERR_ARG),
    (dict(dtype=9), flce.FLCE_ERR_ARG),
    (dict(G=A + 1), flce.FLCE_ERR_ALIGN),
    (dict(out=A + 1), flce.FLCE_ERR_ALIGN),
    (dict(coeffs=(float("nan"), 0, 0)), flce.FLCE_ERR_ARG),
    (dict(coeffs=(4.0, 0.0, 0.0)), flce.FLCE_ERR_ARG),      # s -> 4 s
    (dict(coeffs=(3.0, 0.0, 0.0), steps=2), flce.FLCE_ERR_ARG),
    (dict(coeffs=(1.0, -16.0, 0.0)), flce.FLCE_ERR_ARG),    # B out of range
    (dict(coeffs=(1.0, 0.0, 3.0), steps=2), flce.FLCE_ERR_ARG),
    (dict(coeffs=(3.4445, -4.7750, 2.6)), flce.FLCE_ERR_ARG),  # the standard one, grown
])
def test_orthogonalize_refusals(lib, kw, status):
    a = dict(G=A, batch=1, rows=8, cols=16, steps=5, coeffs=None, eps=1e-7, out=A,
             dtype=flce.FLCE_BF16)
    a.update(kw)
    o = flce.make_opts(sync=0)
    o.dtype = a["dtype"]
    c = None if a["coeffs"] is None else (ctypes.c_float * 3)(*a["coeffs"])
    assert lib.flce_orthogonalize(a["G"], a["batch"], a["rows"], a["cols"], a["steps"], c,
                                  a["eps"], a["out"], ctypes.byref(o)) == status
    assert lib.flce_last_error()


@pytest.mark.parametrize("scale", [float("inf"), -float("inf")])
def test_embed_refuses_an_infinite_scale(lib, scale):
    """0 times it is NaN: ignored tokens would not get their zeros."""
    o = flce.make_opts(sync=0)
    assert lib.flce_embed_fwd(A, A, 4, 16, 10, scale, -100, A, ctypes.byref(o)) == flce.FLCE_ERR_ARG
    assert b"scale" in lib.flce_last_error()
    assert lib.flce_embed_bwd(A, A, 4, 16, 10, scale, -100, A, 0,
                              ctypes.byref(o)) == flce.FLCE_ERR_ARG
    assert b"scale" in lib.flce_last_error()


# Token stride of the operands below: q, k and v as slices of one projection's output,
# and their gradients as slices of another.
QKV = dict(q=A, k=A + 2 * 256, v=A + 2 * 384, o=A + (1 << 30), dO=A + (2 << 30),
           dq=A + (3 << 30), dk=A + (3 << 30) + 2 * 256, dv=A + (3 << 30) + 2 * 384,
           **{n + "_token": 512 for n in ("q", "k", "v", "dq", "dk", "dv")})
HEAD_BY_HEAD = {f: x for i, n in enumerate(("dq", "dk", "dv")) for f, x in (
    (n, A + (3 << 30) + 2 * 64 * i), (n + "_token", 4 * 192), (n + "_head", 192))}


def _attn_statuses(lib, kw):
    """Statuses of both entries; a workspace of 0 bytes keeps an accepted call off the GPU."""
    a = _attn(T=50000, batch=300, **{**QKV, **kw})
    o = flce.make_opts(sync=0)
    o.workspace, o.workspace_bytes = A, 0
    return [fn(ctypes.byref(a), ctypes.byref(o)) for fn in (lib.flce_attn_fwd, lib.flce_attn_bwd)]


@pytest.mark.parametrize("kw", [
    dict(),                                                       # beside each other per token
    {**HEAD_BY_HEAD, "heads_kv": 4, "k_token": 512, "v": A + (4 << 30)},  # per head
    dict(dq=A + (1 << 30)),                                       # a gradient over o
    dict(o=A + 2 * 50000 * 512),                                  # right behind the projection
    dict(dO=A + (3 << 30) - 2 * 50000 * 256),                     # right before the gradients
])
def test_attention_accepts_disjoint_layouts(lib, kw):
    accepted = (flce.FLCE_ERR_ARCH, flce.FLCE_ERR_CUDA, flce.FLCE_ERR_WORKSPACE)
    for status in _attn_statuses(lib, kw):
        assert status in accepted, lib.flce_last_error()


@pytest.mark.parametrize("kw,forward", [
    (dict(o=A, o_token=512), True),                               # o over q
    (dict(o=A + 2 * 256, o_token=512), True),                     # o over k and v
    (dict(o=A + 2 * 48, o_token=512), True),                      # a part of a row
    (dict(o=A + 2 * (512 * 49999 + 256), o_token=512), True),     # the last token of k
    (dict(o=A + 2 * (512 * 50000 - 64), o_token=512), True),      # the end of v
    (dict(dq=A, dq_token=512), False),                            # in place
    (dict(dk=A + 2 * 256, dk_token=512), False),
    (dict(dv=A + 2 * 384, dv_token=512), False),
    (dict(dq=A + (2 << 30)), False),                              # dq over dO
    (dict(dv=A + (3 << 30) + 2 * 256), False),                    # dv over dk
    (dict(dk=A + (3 << 30) + 2 * 200), False),                    # dk into dq's last head
    (dict(dv=A + (3 << 30) + 2 * 512 * 7 + 2 * 128), False),      # dq's heads, tokens later
])
def test_attention_refuses_overlaps(lib, kw, forward):
    fwd, bwd = _attn_statuses(lib, kw)
    assert (fwd if forward else bwd) == flce.FLCE_ERR_ARG
    if not forward:
        assert b"overlaps" in lib.flce_last_error()


def test_orthogonalize_tests_reach_every_tile_shape(lib):
    """The cases of test_orthogonalize_forms take the tile shapes they are there for."""
    from test_gpu_orthogonalize import FORMS, MERGED, PAIR, SINGLE, SPLIT, shapes_of
    for shape, _, forms in FORMS:
        assert shapes_of(lib, shape, 152) == forms, shape
    reached = [set(x) for x in zip(*(forms for _, _, forms in FORMS))]
    assert reached == [{PAIR, SINGLE, SPLIT}, {PAIR, SINGLE, MERGED}, {PAIR, SINGLE, MERGED}]


@pytest.mark.parametrize("a", [(0, 8, 8, 152), (1, 0, 8, 152), (1, 8, (1 << 20) + 1, 152),
                               (65536, 8, 8, 152), (1, 8, 8, 1)])
def test_orthogonalize_shapes_refusals(lib, a):
    out = (ctypes.c_int32 * 3)()
    assert lib.flce_selftest_ortho_shapes(*a, out) == flce.FLCE_ERR_ARG
    assert lib.flce_selftest_ortho_shapes(1, 8, 8, 152, None) == flce.FLCE_ERR_ARG
