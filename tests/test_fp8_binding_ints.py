"""Host integers beyond 32 bits are refused, not cut off: a window of 2^32 would
be one of 0.  On the CPU, against a stand-in library."""
import pytest

from test_fp8_binding import CALLS, lib  # noqa: F401


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 64, -2 ** 31 - 1, -2 ** 32])
@pytest.mark.parametrize("call,name", [
    (c, n) for c in ("decode", "tree") for n in ("max_seqlen", "window_left", "partition_size")
] + [("tree", "max_seqlen_q")])
def test_refused(lib, call, name, value):  # noqa: F811
    f, make = CALLS[call]
    with pytest.raises(ValueError, match=f"{name} must be within 32 bits"):
        f(**dict(make(), **{name: value}))
    assert not lib.calls


@pytest.mark.parametrize("call", ["decode", "tree"])
def test_the_largest_window_goes_through(lib, call):  # noqa: F811
    f, make = CALLS[call]
    f(**dict(make(), window_left=2 ** 31 - 1))
    name = {"decode": "pkv_paged_decode_fp8", "tree": "pkv_paged_tree_attention"}[call]
    assert lib.last(name)["window_left"] == 2 ** 31 - 1
