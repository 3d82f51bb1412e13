"""qk_norm_rope_reshape_and_cache refuses outputs that overlap one another or an
input, and no others.  On the CPU, against a stand-in library."""
import random

import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from test_fp8_binding import BF16, D, HKV, I64, _norm_args, lib  # noqa: F401

HQ, T = 8, 5
ROW = (HQ + 2 * HKV) * D


def fused(tokens=T, heads=HQ + 2 * HKV):
    return torch.zeros(tokens, heads, D, dtype=BF16)


def slices(x):
    return dict(query=x[:, :HQ], key=x[:, HQ:HQ + HKV], value=x[:, HQ + HKV:HQ + 2 * HKV])


def shared(key_value):
    """key and value from one tensor."""
    return dict(key=key_value, value=key_value)


def one_buffer(*parts):
    """[T, heads, D] tensors cut from one buffer at (offset, heads, stride) elements."""
    x = torch.zeros(40 * ROW, dtype=BF16)
    return [x.as_strided((T, h, D), (s, D, 1), o) for o, h, s in parts]


def overlapping():
    x = fused()
    q, ko = one_buffer((0, HQ, ROW), (HQ * D - 16, HKV, ROW))
    yield dict(query=q, query_out=torch.zeros(T, HQ, D, dtype=BF16), key_out=ko)
    kv = torch.zeros(T + 1, HKV, D, dtype=BF16)
    yield dict(key=kv[:-1], value=kv[1:])                         # key in place, over value
    yield dict(slices(x), key=x[:, HQ - 1:HQ + HKV - 1])          # query and key in place
    yield dict(slices(x), value=x[:, HQ + 1:HQ + HKV + 1])
    yield dict(slices(x), query_out=x[:, HKV:HQ + HKV], key_out=torch.zeros(T, HKV, D, dtype=BF16))
    q = torch.zeros(T + 1, HQ, D, dtype=BF16)
    yield dict(query=q[1:], query_out=q[:-1])                     # a token further
    qo, ko = one_buffer((0, HQ, HQ * D), (3 * HQ * D, HKV, HKV * D))
    yield dict(query_out=qo, key_out=ko)                          # other strides


def apart():
    x = fused()
    yield {}
    yield slices(x)                                               # all in place
    yield dict(slices(x), query_out=torch.zeros(T, HQ, D, dtype=BF16))
    yield dict(slices(x), query_out=x[:, :HQ], key_out=x[:, HQ:HQ + HKV])
    kv = torch.zeros(T, HKV, D, dtype=BF16)
    yield dict(shared(kv), key_out=torch.zeros(T, HKV, D, dtype=BF16))
    yield shared(kv)                                              # value's own rows
    yield dict(value=kv, key_out=kv)
    q = fused(2 * T + 1, HQ)
    yield dict(query=q[T:2 * T], query_out=q[:T])
    qo, ko = one_buffer((0, HQ, HQ * D), (T * HQ * D, HKV, HKV * D))
    yield dict(query_out=qo, key_out=ko)
    qo, ko = one_buffer((0, HQ, 2 * ROW), (ROW, HKV, 2 * ROW))    # between the tokens
    yield dict(query_out=qo, key_out=ko)
    yield dict(key=fused(T, HKV), value=fused(T, HKV), query=None, q_weight=None)


@pytest.mark.parametrize("kw", list(overlapping()), ids=range(7))
def test_overlapping_rows_are_refused(lib, kw):  # noqa: F811
    with pytest.raises(ValueError, match="must not overlap"):
        pkv.qk_norm_rope_reshape_and_cache(**dict(_norm_args(), **kw))
    assert not lib.calls


@pytest.mark.parametrize("kw", list(apart()), ids=range(11))
def test_rows_apart_or_in_place_go_through(lib, kw):  # noqa: F811
    pkv.qk_norm_rope_reshape_and_cache(**dict(_norm_args(), **kw))
    assert lib.calls


def test_rows_meet_as_sets_of_bytes():
    rng = random.Random(1)
    seen = set()
    for _ in range(4000):
        n, la, lb = rng.randint(1, 5), rng.randint(1, 6), rng.randint(1, 6)
        sa = la + rng.randint(0, 8)
        sb = sa if rng.random() < 0.5 and sa >= lb else lb + rng.randint(0, 8)
        a, b = rng.randint(0, 40), rng.randint(0, 40)
        rows = [{p + i * s + k for i in range(n) for k in range(m)}
                for p, s, m in ((a, sa, la), (b, sb, lb))]
        want = bool(rows[0] & rows[1])
        assert pkv._rows_meet(n, a, sa, la, b, sb, lb) == want, (n, a, sa, la, b, sb, lb)
        seen.add((want, sa == sb))
    assert len(seen) == 4
