"""Calls without a row (an expert-parallel rank, or a batch, that got no token) on a host without a GPU.

The buffers of no rows have no address: a call that has nothing to write is
accepted, as moe_unpermute accepts it, and what is wrong beside that is still
refused.
"""

from test_experts_host import (INVALID, MISALIGNED, OK, gated, gated_back, host_only, lib, linear,  # noqa: F401
                               linear_back, unpermute_back)


@host_only
def test_no_tokens(lib):  # noqa: F811
    empty = dict(n=0, do=None, y=None, wts=None, inv=None)
    assert unpermute_back(lib, dy=None, dw=None, **empty) == OK
    assert unpermute_back(lib, dw=None, **empty) == OK
    assert unpermute_back(lib, dy=None, **empty) == OK
    assert unpermute_back(lib, dy=None, dw=None, n=10) == INVALID
    assert unpermute_back(lib, dy=None, dw=None, **dict(empty, h=60)) == MISALIGNED
    assert unpermute_back(lib, dy=None, dw=None, dt=7, **empty) == INVALID


@host_only
def test_no_rows(lib):  # noqa: F811
    plain = dict(rows=0, act=0, dy=None, pre=None, dz=None, x=None, dx=None, db=None, dw=None)
    assert linear_back(lib, **plain) == OK
    assert linear_back(lib, **dict(plain, w=None)) == OK
    assert linear_back(lib, **dict(plain, rows=1)) == INVALID
    assert linear_back(lib, **dict(plain, k=12)) == MISALIGNED
    assert linear_back(lib, **dict(plain, off=None)) == INVALID
    assert linear_back(lib, **dict(plain, act=2)) == OK
    assert gated_back(lib, rows=0, dh=None, keep=None, dgu=None, x=None, dx=None, dw=None) == OK
    assert linear(lib, rows=0, x=None, y=None, pre=None, r=None) == OK
    assert gated(lib, rows=0, x=None, h=None, keep=None) == OK
