"""Host integers beyond 32 bits are refused, not cut off, and a wider window is the
widest (2^32 would be one of 0).  On the CPU, against a stand-in library."""
import pytest

from test_fp8_binding import CALLS, lib  # noqa: F401


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 64, -2 ** 31 - 1, -2 ** 32])
@pytest.mark.parametrize("call,name", [
    (c, n) for c in ("decode", "tree") for n in ("max_seqlen", "partition_size")
] + [("tree", "max_seqlen_q")])
def test_refused(lib, call, name, value):  # noqa: F811
    f, make = CALLS[call]
    with pytest.raises(ValueError, match=f"{name} must be within 32 bits"):
        f(**dict(make(), **{name: value}))
    assert not lib.calls


@pytest.mark.parametrize("call", ["decode", "tree"])
def test_a_window_below_32_bits_is_refused(lib, call):  # noqa: F811
    f, make = CALLS[call]
    with pytest.raises(ValueError, match="window_left must be within 32 bits"):
        f(**dict(make(), window_left=-2 ** 32))


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 63 - 1, 2 ** 70])
@pytest.mark.parametrize("call", ["decode", "tree"])
def test_the_widest_window(lib, call, window):  # noqa: F811
    f, make = CALLS[call]
    f(**dict(make(), window_left=window))
    name = {"decode": "pkv_paged_decode_fp8", "tree": "pkv_paged_tree_attention"}[call]
    assert lib.last(name)["window_left"] == 2 ** 31 - 1
