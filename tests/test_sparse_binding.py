"""The binding of the sparse step's calls: every argument reaches the C parameter it
belongs to, and tensors of a wrong type, shape or device, and overlapping ones, are
refused before the library is called.  On the CPU, against a stand-in library that
records the calls."""
import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from test_binding_marshalling import STREAM, _desc_fields, _Recorder

BF16, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
U8, I8, E4M3 = torch.uint8, torch.int8, torch.float8_e4m3fn
NB, BS, HKV, D = 10, 16, 2, 64


@pytest.fixture
def lib(monkeypatch):
    rec = _Recorder(pkv.load_library())
    monkeypatch.setattr(pkv, "load_library", lambda *a, **k: rec)
    monkeypatch.setattr(pkv, "_cuda_index", lambda name, t: t.get_device())  # -1: the CPU
    monkeypatch.setattr(pkv, "_stream_handle", lambda s: STREAM)
    return rec


def z(*shape, dtype=BF16):
    return torch.zeros(*shape).to(dtype)


def _pool(layout="NHD", dtype=BF16):
    return z(*((NB, BS, HKV, D) if layout == "NHD" else (NB, HKV, BS, D)), dtype=dtype)


def _tables_args():
    return dict(block_table=z(3, 4, dtype=I32), old_seqlens=z(3, dtype=I32),
                new_seqlens=z(3, dtype=I32), free_blocks=z(NB, dtype=I32), num_free=z(1, dtype=I32),
                block_size=BS, num_rows=9)


def _bounds_args():
    return dict(k_cache=_pool(), page_bounds=z(NB, HKV, 2, D, dtype=I8),
                bounds_scale=z(NB, HKV, dtype=U8), slot_mapping=z(7, dtype=I64))


def _select_args():
    return dict(q=z(3, 8, D), page_bounds=z(NB, HKV, 2, D, dtype=I8),
                bounds_scale=z(NB, HKV, dtype=U8), block_table=z(3, 4, dtype=I32),
                cache_seqlens=z(3, dtype=I32), max_seqlen=60, top_k=5, block_size=BS)


def _sparse_args():
    return dict(q=z(3, 8, D), k_cache=_pool(), v_cache=_pool(), block_table=z(3, 4, dtype=I32),
                cache_seqlens=z(3, dtype=I32), pages=z(3, HKV, 5, dtype=I32))


CALLS = dict(tables=(pkv.update_block_tables, _tables_args),
             bounds=(pkv.update_page_bounds, _bounds_args),
             select=(pkv.select_pages, _select_args),
             sparse=(pkv.paged_sparse_attention, _sparse_args))
ALL = tuple(CALLS)


def _same(got, tensors):
    for name, t in tensors.items():
        assert got[name] == (None if t is None else t.data_ptr()), name


def test_tables(lib):
    a = _tables_args()
    outs = dict(slot_mapping=z(9, dtype=I64), positions=z(9, dtype=I64),
                cu_seq_lens_q=z(4, dtype=I32), cu_seq_lens_k=z(4, dtype=I32))
    err = z(1, dtype=I32)
    got = pkv.update_block_tables(**a, **outs, dev_error=err)
    assert all(x is y for x, y in zip(got, outs.values()))
    c = lib.last("pkv_update_block_tables")
    _same(c, dict(outs, dev_error=err, **{k: v for k, v in a.items() if torch.is_tensor(v)}))
    assert (c["max_blocks_per_seq"], c["batch"], c["num_blocks"], c["block_size"], c["num_rows"],
            c["stream"]) == (4, 3, NB, BS, 9, STREAM)
    got = pkv.update_block_tables(**a)
    assert [(tuple(x.shape), x.dtype) for x in got] == [((9,), I64), ((9,), I64), ((4,), I32),
                                                        ((4,), I32)]
    _same(lib.last("pkv_update_block_tables"), dict(zip(outs, got), dev_error=None))


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("fp8", [False, True])
def test_bounds(lib, layout, fp8):
    a = dict(_bounds_args(), k_cache=_pool(layout, E4M3 if fp8 else BF16))
    ks = z(NB, HKV, BS, dtype=U8) if fp8 else None
    err = z(1, dtype=I32)
    assert pkv.update_page_bounds(**a, k_scale=ks, dev_error=err, layout=layout) is None
    c = lib.last("pkv_update_page_bounds")
    _same(c, dict(a, k_scale=ks, dev_error=err))
    assert _desc_fields(c["cache"]) == (NB, BS, HKV, D, pkv.PKV_E4M3 if fp8 else pkv.PKV_BF16,
                                        int(layout == "HND"))
    assert c["num_tokens"] == 7 and c["stream"] == STREAM


def test_select(lib):
    a = dict(_select_args(), q=z(11, 8, D))
    cu, pages, err = z(4, dtype=I32), z(11, HKV, 5, dtype=I32), z(1, dtype=I32)
    got = pkv.select_pages(**a, num_first=2, num_recent=3, cu_seq_lens_q=cu, pages=pages,
                           dev_error=err)
    assert got is pages
    c = lib.last("pkv_select_pages")
    _same(c, dict(pages=pages, cu_seq_lens_q=cu, dev_error=err,
                  **{k: v for k, v in a.items() if torch.is_tensor(v)}))
    assert (c["top_k"], c["num_blocks"], c["block_size"], c["num_kv_heads"], c["head_dim"]) == \
        (5, NB, BS, HKV, D)
    assert (c["max_blocks_per_seq"], c["max_seqlen"], c["batch"], c["total_q"]) == (4, 60, 3, 11)
    assert (c["num_qo_heads"], c["num_first"], c["num_recent"], c["stream"]) == (8, 2, 3, STREAM)
    got = pkv.select_pages(**_select_args())
    c = lib.last("pkv_select_pages")
    assert tuple(got.shape) == (3, HKV, 5) and got.dtype == I32 and c["pages"] == got.data_ptr()
    assert (c["num_first"], c["num_recent"], c["total_q"]) == (1, 1, 3)
    assert c["cu_seq_lens_q"] is None and c["dev_error"] is None


@pytest.mark.parametrize("fp8", [False, True])
def test_sparse(lib, fp8):
    a = dict(_sparse_args(), q=z(11, 8, D), pages=z(11, HKV, 5, dtype=I32))
    if fp8:
        a.update(k_cache=_pool("HND", E4M3), v_cache=_pool("HND", E4M3),
                 k_scale=z(NB, HKV, BS, dtype=U8), v_scale=z(NB, HKV, BS, dtype=U8))
    else:
        a.update(k_cache=_pool("HND"), v_cache=_pool("HND"))
    cu, sink, lse = z(4, dtype=I32), z(8, dtype=F32), z(11, 8, dtype=F32)
    out, err = z(11, 8, D), z(1, dtype=I32)
    got = pkv.paged_sparse_attention(**a, cu_seq_lens_q=cu, sink=sink, sm_scale=0.5, out=out,
                                     lse=lse, dev_error=err, layout="HND")
    assert got is out
    c = lib.last("pkv_paged_sparse_attention")
    _same(c, dict(a, cu_seq_lens_q=cu, sink=sink, lse_out=lse, out=out, dev_error=err))
    assert c["k_scale"] == (a["k_scale"].data_ptr() if fp8 else None)
    assert _desc_fields(c["cache"]) == (NB, BS, HKV, D, pkv.PKV_E4M3 if fp8 else pkv.PKV_BF16, 1)
    assert (c["max_blocks_per_seq"], c["batch"], c["total_q"], c["top_k"], c["num_qo_heads"],
            c["sm_scale"], c["stream"]) == (4, 3, 11, 5, 8, 0.5, STREAM)
    got = pkv.paged_sparse_attention(**_sparse_args())
    c = lib.last("pkv_paged_sparse_attention")
    assert c["out"] == got.data_ptr() and c["sm_scale"] == D ** -0.5
    for name in ("cu_seq_lens_q", "sink", "lse_out", "dev_error", "k_scale", "v_scale"):
        assert c[name] is None


# (calls, argument, a value it refuses)
REFUSALS = [
    (ALL, "dev_error", lambda: z(1, dtype=I64)), (ALL, "dev_error", lambda: z(0, dtype=I32)),
    (("tables",), "block_table", lambda: z(3, 4, dtype=I64)),
    (("tables",), "block_table", lambda: z(3, 8, dtype=I32)[:, ::2]),
    (("tables",), "old_seqlens", lambda: z(2, dtype=I32)),
    (("tables",), "new_seqlens", lambda: z(3, dtype=I64)),
    (("tables",), "free_blocks", lambda: z(NB, dtype=I64)),
    (("tables",), "num_free", lambda: z(2, dtype=I32)),
    (("tables",), "num_rows", -1), (("tables",), "num_rows", 2 ** 32),
    (("tables",), "block_size", 2 ** 32 + 16),
    (("tables",), "slot_mapping", lambda: z(9, dtype=I32)),
    (("tables",), "positions", lambda: z(8, dtype=I64)),
    (("tables",), "cu_seq_lens_q", lambda: z(3, dtype=I32)),
    (("tables",), "cu_seq_lens_k", lambda: z(4, dtype=I64)),
    (("bounds", "sparse"), "layout", "NHWC"),
    (("bounds",), "k_cache", lambda: _pool(dtype=F32)),
    (("bounds",), "k_cache", lambda: _pool(dtype=E4M3)),
    (("bounds",), "k_cache", lambda: z(NB + 1, BS, HKV, D)),
    (("bounds",), "k_scale", lambda: z(NB, HKV, BS, dtype=U8)),
    (("bounds", "select"), "page_bounds", lambda: z(NB, HKV, 2, D, dtype=U8)),
    (("bounds", "select"), "page_bounds", lambda: z(NB, HKV, 3, D, dtype=I8)),
    (("bounds", "select"), "page_bounds", lambda: z(NB, HKV, 2 * D, dtype=I8)),
    (("bounds", "select"), "page_bounds", lambda: z(NB, HKV, 2, 2 * D, dtype=I8)),
    (("bounds", "select"), "bounds_scale", lambda: z(NB, HKV + 1, dtype=U8)),
    (("bounds", "select"), "bounds_scale", lambda: z(NB, HKV, dtype=I8)),
    (("bounds",), "slot_mapping", lambda: z(7, dtype=I32)),
    (("bounds",), "slot_mapping", lambda: z(14, dtype=I64)[::2]),
    (("select", "sparse"), "q", lambda: z(3, 8, D, dtype=F32)),
    (("select", "sparse"), "q", lambda: z(3, 8, 128)),
    (("select", "sparse"), "q", lambda: z(4, 8, D)),
    (("select", "sparse"), "q", lambda: z(3, 16, D)[:, ::2]),
    (("select", "sparse"), "block_table", lambda: z(2, 4, dtype=I32)),
    (("select", "sparse"), "block_table", lambda: z(3, 4, dtype=I64)),
    (("select", "sparse"), "cache_seqlens", lambda: z(4, dtype=I32)),
    (("select", "sparse"), "cu_seq_lens_q", lambda: z(3, dtype=I32)),
    (("select", "sparse"), "cu_seq_lens_q", lambda: z(4, dtype=I64)),
    (("select",), "max_seqlen", 2 ** 31), (("select",), "top_k", 0), (("select",), "top_k", 2 ** 33),
    (("select",), "num_first", 2 ** 32), (("select",), "num_recent", 2 ** 32 + 1),
    (("select",), "pages", lambda: z(3, HKV, 4, dtype=I32)),
    (("select",), "pages", lambda: z(3, HKV, 5, dtype=I64)),
    (("sparse",), "pages", lambda: z(3, 8, 5, dtype=I32)),
    (("sparse",), "pages", lambda: z(2, HKV, 5, dtype=I32)),
    (("sparse",), "pages", lambda: z(3, HKV, 5, dtype=I64)),
    (("sparse",), "pages", lambda: z(3, HKV, 10, dtype=I32)[:, :, ::2]),
    (("sparse",), "pages", lambda: z(3, dtype=I32)[0]),
    (("sparse",), "v_cache", lambda: z(NB, BS, HKV, 2 * D)),
    (("sparse",), "k_cache", lambda: _pool(dtype=E4M3)),
    (("sparse",), "k_scale", lambda: z(NB, HKV, BS, dtype=U8)),
    (("sparse",), "sink", lambda: z(7, dtype=F32)), (("sparse",), "lse", lambda: z(3, 7, dtype=F32)),
    (("sparse",), "out", lambda: z(3, 8, D, dtype=F32)),
]


@pytest.mark.parametrize("call,name,value", [
    pytest.param(c, n, v, id=f"{c}-{n}-{i}") for i, (cs, n, v) in enumerate(REFUSALS) for c in cs])
def test_refusals(lib, call, name, value):
    f, make = CALLS[call]
    args = make()
    f(**args)  # as it is, the call goes through
    lib.calls.clear()
    args[name] = value() if callable(value) else value
    with pytest.raises((ValueError, TypeError)):
        f(**args)
    assert not lib.calls


@pytest.mark.parametrize("a,b", [("block_table", "free_blocks"), ("num_free", "free_blocks"),
                                 ("cu_seq_lens_q", "cu_seq_lens_k"), ("old_seqlens", "cu_seq_lens_q"),
                                 ("new_seqlens", "block_table"), ("slot_mapping", "positions")])
def test_tables_that_overlap(lib, a, b):
    """In place is in place; nothing else shares memory (the two lengths may)."""
    store = z(64, dtype=I64)
    args = _tables_args()
    args.update(slot_mapping=z(9, dtype=I64), positions=z(9, dtype=I64),
                cu_seq_lens_q=z(4, dtype=I32), cu_seq_lens_k=z(4, dtype=I32))
    args["new_seqlens"] = args["old_seqlens"]
    pkv.update_block_tables(**args)
    lib.calls.clear()
    args["new_seqlens"] = z(3, dtype=I32)
    for name, at in ((a, 8), (b, 6)):
        t = args[name]
        flat = store if t.dtype is I64 else store.view(I32)
        args[name] = flat[at:at + t.numel()].view(t.shape)
    with pytest.raises(ValueError, match="overlap"):
        pkv.update_block_tables(**args)
    assert not lib.calls


def test_out_over_q(lib):
    args = _sparse_args()
    with pytest.raises(ValueError, match="overlap"):
        pkv.paged_sparse_attention(**args, out=args["q"])
    assert not lib.calls


@pytest.mark.parametrize("call", ALL)
def test_cpu_tensors_are_refused(call):
    f, make = CALLS[call]
    with pytest.raises(ValueError, match="CUDA"):
        f(**make())


@pytest.mark.parametrize("call,name", [("tables", "update_block_tables"),
                                       ("bounds", "update_page_bounds"), ("select", "select_pages"),
                                       ("sparse", "paged_sparse_attention")])
def test_status_codes_become_exceptions(lib, monkeypatch, call, name):
    monkeypatch.setattr(_Recorder, "__getattr__", lambda self, n: (
        getattr(self.real, n) if n == "pkv_status_string" else lambda *a: 2))
    f, make = CALLS[call]
    with pytest.raises(pkv.PkvError, match=f"pkv_{name}"):
        f(**make())
