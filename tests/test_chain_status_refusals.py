"""Argument refusals of ddt_chain_status, on the host before any launch (no GPU needed): the pointers below are never
dereferenced."""
import ctypes

from tests.test_serving_refusals import INVALID, lib, pytestmark  # noqa: F401

at = ctypes.c_void_p


def _call(lib, n=3, B=4, st=1 << 40, length=2 << 40, length_out=3 << 40, status_out=4 << 40):  # noqa: F811
    return lib.ddt_chain_status(n, B, *(None if x is None else at(x) for x in (st, length, length_out, status_out)), None)


def test_refusals(lib):  # noqa: F811
    before = lib.ddt_launch_count()
    for kw in (dict(n=0), dict(B=0), dict(st=None), dict(length=None), dict(length_out=None),
               dict(length=None, length_out=None, status_out=None),
               # outputs over one another and over inputs: ends of 4 requests and 3 rows of them
               dict(status_out=3 << 40), dict(status_out=(3 << 40) + 12), dict(length_out=(1 << 40) + 44),
               dict(status_out=(1 << 40) + 44), dict(length_out=2 << 40), dict(status_out=(2 << 40) + 12)):
        assert _call(lib, **kw) == INVALID, kw
    assert lib.ddt_launch_count() == before
