"""Calls of the norms that the C entry points refuse; no GPU is touched."""
import ctypes

import pytest

from shot_allreduce_ranks_gb300 import _lib, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_r_and_y_in_one_place_are_refused(lib):
    n = _lib.ArNorm(0, 0, 4, 8, 0, 1e-6, 1.0, 0.0)

    def forward(r, y):
        return lib.ar_residual_norm(ctypes.byref(n), 16, 8, 16, 8, None, 0, None, None, 32, None, r, 8, y, 8, None)

    assert forward(64, 64) == forward(16, 16) == _lib.AR_ERR_INVALID_ARG
    n.rows = 0
    assert forward(64, 64) == _lib.AR_OK
