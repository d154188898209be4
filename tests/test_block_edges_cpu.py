"""CPU-only checks of edges of the operators between blocks."""
import ctypes

import pytest

from linear_cross_entropy_fwd_gb300 import FLCE_ERR_ALIGN
from test_block_cpu import A, ACCEPTED, M, _join, _opts, lib  # noqa: F401


@pytest.mark.parametrize("norm,names", [("post_norm", ("w_post", "b_post")),
                                        ("pre_norm", ("w_pre", "b_pre"))])
def test_vectors_without_their_norm(lib, norm, names):  # noqa: F811
    """What nothing reads is not checked either: neither its alignment nor what it overlaps."""
    for name in names:
        for at in (A + 4, A + 5 * M):
            for fn in (lib.flce_resnorm_fwd, lib.flce_resnorm_bwd):
                a = _join(**{norm: 0, name: at})
                assert fn(ctypes.byref(a), _opts()) in ACCEPTED, lib.flce_last_error()
        assert lib.flce_resnorm_fwd(ctypes.byref(_join(**{name: A + 4})), _opts()) == FLCE_ERR_ALIGN
