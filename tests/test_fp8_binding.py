"""The binding of the 8-bit cache, the tree attention and the fused norm: every
argument reaches the C parameter it belongs to, and tensors of a wrong type,
shape, stride or device are refused before the library is called.  On the CPU,
against a stand-in library that records the calls."""
import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from test_binding_marshalling import STREAM, _desc_fields, _Recorder

BF16, F32, I32, I64, U8 = (torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8)
E4M3 = torch.float8_e4m3fn
NB, BS, HKV, D = 10, 16, 2, 64


@pytest.fixture
def lib(monkeypatch):
    rec = _Recorder(pkv.load_library())
    monkeypatch.setattr(pkv, "load_library", lambda *a, **k: rec)
    monkeypatch.setattr(pkv, "_cuda_index", lambda name, t: t.get_device())  # -1: the CPU
    monkeypatch.setattr(pkv, "_stream_handle", lambda s: STREAM)
    for f in (pkv._decode_ws, pkv._tree_ws):  # sizes of the real library, not the stand-in's
        f.cache_clear()
    yield rec
    for f in (pkv._decode_ws, pkv._tree_ws):
        f.cache_clear()


def _pools(layout="NHD", dtype=E4M3):
    shape = (NB, BS, HKV, D) if layout == "NHD" else (NB, HKV, BS, D)
    return torch.zeros(shape).to(dtype), torch.zeros(shape).to(dtype)


def _scales():
    return torch.zeros(NB, HKV, BS, dtype=U8), torch.zeros(NB, HKV, BS, dtype=U8)


def _same(got, tensors):
    for name, t in tensors.items():
        assert got[name] == t.data_ptr(), name


@pytest.mark.parametrize("layout", ["NHD", "HND"])
def test_write(lib, layout):
    (kc, vc), (ks, vs) = _pools(layout), _scales()
    qkv = torch.zeros(5, 3 * HKV, D, dtype=BF16)
    key, value = qkv[:, HKV:2 * HKV], torch.zeros(5, HKV, D, dtype=BF16)
    slots, err = torch.zeros(5, dtype=I64), torch.zeros(1, dtype=I32)
    pkv.reshape_and_cache_fp8(key, value, kc, vc, ks, vs, slots, dev_error=err, layout=layout)
    a = lib.last("pkv_reshape_and_cache_fp8")
    _same(a, dict(key=key, value=value, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs,
                  slot_mapping=slots, dev_error=err))
    assert (a["key_stride"], a["value_stride"]) == (3 * HKV * D, HKV * D)
    assert a["dtype"] == pkv.PKV_BF16 and a["num_tokens"] == 5 and a["stream"] == STREAM
    assert _desc_fields(a["cache"]) == (NB, BS, HKV, D, pkv.PKV_E4M3, int(layout == "HND"))
    pkv.reshape_and_cache_fp8(key.float(), value.float(), kc, vc, ks, vs, slots, layout=layout)
    a = lib.last("pkv_reshape_and_cache_fp8")
    assert a["dtype"] == pkv.PKV_F32 and a["dev_error"] is None


def test_gather(lib):
    (kc, vc), (ks, vs) = _pools("HND"), _scales()
    bt, cu = torch.zeros(3, 4, dtype=I32), torch.zeros(4, dtype=I32)
    k, v = torch.zeros(9, HKV, D, dtype=BF16), torch.zeros(9, HKV, D, dtype=BF16)
    err = torch.zeros(1, dtype=I32)
    got = pkv.gather_cache_fp8(kc, vc, ks, vs, bt, cu, 9, key=k, value=v, dev_error=err,
                               layout="HND")
    assert got[0] is k and got[1] is v
    a = lib.last("pkv_gather_cache_fp8")
    _same(a, dict(key=k, value=v, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, block_table=bt,
                  cu_seq_lens_k=cu, dev_error=err))
    assert (a["max_blocks_per_seq"], a["batch"], a["total_k"]) == (4, 3, 9)
    assert _desc_fields(a["cache"]) == (NB, BS, HKV, D, pkv.PKV_E4M3, 1)
    k, v = pkv.gather_cache_fp8(kc, vc, ks, vs, bt, cu, 7, layout="HND")
    assert k.shape == v.shape == (7, HKV, D) and k.dtype == v.dtype == BF16
    _same(lib.last("pkv_gather_cache_fp8"), dict(key=k, value=v))


def test_decode(lib):
    (kc, vc), (ks, vs) = _pools(), _scales()
    q, out = torch.zeros(3, 8, D, dtype=BF16), torch.zeros(3, 8, D, dtype=BF16)
    bt, sl = torch.zeros(3, 70, dtype=I32), torch.zeros(3, dtype=I32)
    sink, alibi = torch.zeros(8), torch.zeros(8)
    lse, err = torch.zeros(3, 8), torch.zeros(1, dtype=I32)
    ws = torch.zeros(8192, dtype=U8)
    got = pkv.paged_decode_fp8(q, kc, vc, ks, vs, bt, sl, 999, sink=sink, window_left=700,
                               sm_scale=0.25, partition_size=256, out=out, lse=lse, workspace=ws,
                               dev_error=err, alibi_slopes=alibi)
    assert got is out
    a = lib.last("pkv_paged_decode_fp8")
    _same(a, dict(out=out, q=q, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, block_table=bt,
                  cache_seqlens=sl, sink=sink, alibi_slopes=alibi, lse_out=lse, workspace=ws,
                  dev_error=err))
    assert (a["max_blocks_per_seq"], a["max_seqlen"], a["batch"], a["num_qo_heads"]) == \
        (70, 999, 3, 8)
    assert (a["window_left"], a["sm_scale"], a["partition_size"]) == (700, 0.25, 256)
    assert a["workspace_bytes"] == 8192 and a["stream"] == STREAM
    assert list(lib.last("pkv_paged_decode_workspace_size").values()) == [3, 8, D, 999, 256, 700]


def test_decode_defaults(lib):
    (kc, vc), (ks, vs) = _pools(), _scales()
    q = torch.zeros(1, 2, D, dtype=BF16)
    bt, sl = torch.zeros(1, 80, dtype=I32), torch.zeros(1, dtype=I32)
    out = pkv.paged_decode_fp8(q, kc, vc, ks, vs, bt, sl, 512)
    a = lib.last("pkv_paged_decode_fp8")
    assert out.shape == q.shape and a["out"] == out.data_ptr()
    assert a["sm_scale"] == D ** -0.5 and a["partition_size"] == 0 and a["window_left"] == -1
    assert a["workspace"] is None and a["workspace_bytes"] == 0  # one partition
    for name in ("sink", "alibi_slopes", "lse_out", "dev_error"):
        assert a[name] is None
    pkv.paged_decode_fp8(q, kc, vc, ks, vs, bt, sl, 513)
    a = lib.last("pkv_paged_decode_fp8")
    assert a["workspace"] is not None and a["workspace_bytes"] == 4096


@pytest.mark.parametrize("fp8", [False, True])
def test_norm(lib, fp8):
    (kc, vc), (ks, vs) = _pools(dtype=E4M3 if fp8 else BF16), _scales()
    sc = dict(k_scale=ks, v_scale=vs) if fp8 else {}
    qkv = torch.zeros(6, 8 + 2 * HKV, D, dtype=BF16)
    q, k, v = qkv[:, :8], qkv[:, 8:8 + HKV], qkv[:, 8 + HKV:]
    qo, ko = torch.zeros(6, 8, D, dtype=BF16), torch.zeros(6, 2 * HKV, D, dtype=BF16)[:, HKV:]
    pos, slots = torch.zeros(6, dtype=I64), torch.zeros(6, dtype=I64)
    table, err = torch.zeros(99, 16, 2), torch.zeros(1, dtype=I32)
    qw, kw = torch.zeros(D), torch.zeros(D)
    pkv.qk_norm_rope_reshape_and_cache(q, k, v, kc, vc, pos, slots, table, qw, kw, eps=1e-5,
                                       is_neox_style=False, query_out=qo, key_out=ko,
                                       dev_error=err, **sc)
    a = lib.last("pkv_qk_norm_rope_reshape_and_cache")
    _same(a, dict(query=q, key=k, value=v, query_out=qo, key_out=ko, k_cache=kc, v_cache=vc,
                  positions=pos, slot_mapping=slots, q_weight=qw, k_weight=kw, cos_sin=table,
                  dev_error=err))
    row = (8 + 2 * HKV) * D
    assert [a[n + "_stride"] for n in ("query", "key", "value", "query_out", "key_out")] == \
        [row, row, row, 8 * D, 2 * HKV * D]
    assert a["k_scale"] == (ks.data_ptr() if fp8 else None)
    assert a["v_scale"] == (vs.data_ptr() if fp8 else None)
    assert (a["dtype"], a["num_tokens"], a["num_qo_heads"]) == (pkv.PKV_BF16, 6, 8)
    assert (a["max_position"], a["rotary_dim"]) == (99, 32)
    assert (bool(a["weight_f32"]), bool(a["is_neox_style"]), a["eps"]) == (True, False, 1e-5)
    assert _desc_fields(a["cache"])[4] == (pkv.PKV_E4M3 if fp8 else pkv.PKV_BF16)
    # in place, weights of the rows' dtype
    pkv.qk_norm_rope_reshape_and_cache(q, k, v, kc, vc, pos, slots, table, qw.bfloat16(),
                                       kw.bfloat16(), **sc)
    a = lib.last("pkv_qk_norm_rope_reshape_and_cache")
    assert (a["query_out"], a["key_out"]) == (q.data_ptr(), k.data_ptr())
    assert (a["query_out_stride"], a["key_out_stride"]) == (row, row)
    assert not a["weight_f32"] and a["is_neox_style"] and a["eps"] == 1e-6
    # no query
    pkv.qk_norm_rope_reshape_and_cache(None, k, v, kc, vc, pos, slots, table, None, kw, **sc)
    a = lib.last("pkv_qk_norm_rope_reshape_and_cache")
    assert a["query"] is None and a["query_out"] is None and a["num_qo_heads"] == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_tree(lib, fp8):
    (kc, vc), (ks, vs) = _pools("HND", E4M3 if fp8 else BF16), _scales()
    sc = dict(k_scale=ks, v_scale=vs) if fp8 else {}
    q, out = torch.zeros(11, 8, D, dtype=BF16), torch.zeros(11, 8, D, dtype=BF16)
    bt, cu, sl = torch.zeros(3, 9, dtype=I32), torch.zeros(4, dtype=I32), torch.zeros(3, dtype=I32)
    mask, depth = torch.zeros(11, 2, dtype=I64), torch.zeros(11, dtype=I32)
    sink, alibi, lse = torch.zeros(8), torch.zeros(8), torch.zeros(11, 8)
    ws, err = torch.zeros(8192, dtype=U8), torch.zeros(1, dtype=I32)
    got = pkv.paged_tree_attention(q, kc, vc, bt, cu, sl, 100, 144, mask, tree_depth=depth,
                                   sink=sink, window_left=77, sm_scale=0.5, partition_size=256,
                                   out=out, lse=lse, workspace=ws, dev_error=err,
                                   alibi_slopes=alibi, layout="HND", **sc)
    assert got is out
    a = lib.last("pkv_paged_tree_attention")
    _same(a, dict(out=out, q=q, k_cache=kc, v_cache=vc, block_table=bt, cu_seq_lens_q=cu,
                  cache_seqlens=sl, tree_mask=mask, tree_depth=depth, sink=sink,
                  alibi_slopes=alibi, lse_out=lse, workspace=ws, dev_error=err))
    assert a["k_scale"] == (ks.data_ptr() if fp8 else None)
    assert a["v_scale"] == (vs.data_ptr() if fp8 else None)
    assert (a["max_blocks_per_seq"], a["max_seqlen_q"], a["max_seqlen"], a["total_q"]) == \
        (9, 100, 144, 11)
    assert (a["mask_words"], a["batch"], a["num_qo_heads"]) == (2, 3, 8)
    assert (a["window_left"], a["sm_scale"], a["partition_size"]) == (77, 0.5, 256)
    assert a["workspace_bytes"] == 8192 and a["stream"] == STREAM
    assert _desc_fields(a["cache"]) == (NB, BS, HKV, D, pkv.PKV_E4M3 if fp8 else pkv.PKV_BF16, 1)
    assert list(lib.last("pkv_paged_tree_attention_workspace_size").values()) == \
        [3, 8, HKV, D, 100]
    out = pkv.paged_tree_attention(q, kc, vc, bt, cu, sl, 100, 144, mask, layout="HND", **sc)
    a = lib.last("pkv_paged_tree_attention")
    assert a["out"] == out.data_ptr() and a["sm_scale"] == D ** -0.5
    assert a["workspace_bytes"] == 4096 and a["window_left"] == -1 and a["partition_size"] == 0
    for name in ("tree_depth", "sink", "alibi_slopes", "lse_out", "dev_error"):
        assert a[name] is None


# ---------------------------------------------------------------- refusals
def _write_args():
    (kc, vc), (ks, vs) = _pools(), _scales()
    return dict(key=torch.zeros(5, HKV, D, dtype=BF16), value=torch.zeros(5, HKV, D, dtype=BF16),
                k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs,
                slot_mapping=torch.zeros(5, dtype=I64))


def _gather_args():
    (kc, vc), (ks, vs) = _pools(), _scales()
    return dict(k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs,
                block_table=torch.zeros(3, 4, dtype=I32), cu_seq_lens_k=torch.zeros(4, dtype=I32),
                total_k=9)


def _decode_args():
    (kc, vc), (ks, vs) = _pools(), _scales()
    return dict(q=torch.zeros(3, 8, D, dtype=BF16), k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs,
                block_table=torch.zeros(3, 4, dtype=I32), cache_seqlens=torch.zeros(3, dtype=I32),
                max_seqlen=64)


def _norm_args():
    (kc, vc), (ks, vs) = _pools(), _scales()
    return dict(query=torch.zeros(5, 8, D, dtype=BF16), key=torch.zeros(5, HKV, D, dtype=BF16),
                value=torch.zeros(5, HKV, D, dtype=BF16), k_cache=kc, v_cache=vc, k_scale=ks,
                v_scale=vs, positions=torch.zeros(5, dtype=I64),
                slot_mapping=torch.zeros(5, dtype=I64), cos_sin=torch.zeros(99, D // 2, 2),
                q_weight=torch.zeros(D), k_weight=torch.zeros(D))


def _tree_args():
    (kc, vc), (ks, vs) = _pools(), _scales()
    return dict(q=torch.zeros(11, 8, D, dtype=BF16), k_cache=kc, v_cache=vc, k_scale=ks,
                v_scale=vs, block_table=torch.zeros(3, 4, dtype=I32),
                cu_seq_lens_q=torch.zeros(4, dtype=I32), cache_seqlens=torch.zeros(3, dtype=I32),
                max_seqlen_q=8, max_seqlen=64, tree_mask=torch.zeros(11, 1, dtype=I64),
                tree_depth=torch.zeros(11, dtype=I32))


CALLS = dict(write=(pkv.reshape_and_cache_fp8, _write_args),
             gather=(pkv.gather_cache_fp8, _gather_args),
             decode=(pkv.paged_decode_fp8, _decode_args),
             norm=(pkv.qk_norm_rope_reshape_and_cache, _norm_args),
             tree=(pkv.paged_tree_attention, _tree_args))
ALL = tuple(CALLS)


def z(*shape, dtype=BF16):
    return torch.zeros(*shape).to(dtype)


# (calls, argument, a value it refuses)
REFUSALS = [
    (ALL, "k_scale", None), (ALL, "v_scale", None),
    (ALL, "k_scale", lambda: z(NB, HKV, BS, dtype=torch.int8)),
    (ALL, "k_scale", lambda: z(NB, BS, HKV, dtype=U8)),
    (ALL, "v_scale", lambda: z(NB, HKV, BS + 1, dtype=U8)[:, :, :BS]),
    (ALL, "k_cache", lambda: z(NB, BS, HKV, D)),
    (ALL, "v_cache", lambda: z(NB, BS, HKV, 2 * D, dtype=E4M3)),
    (ALL, "v_cache", lambda: z(NB, BS, 2 * HKV, D, dtype=E4M3)[:, :, ::2]),
    (ALL, "layout", "NHWC"),
    (ALL, "dev_error", lambda: z(1, dtype=I64)), (ALL, "dev_error", lambda: z(0, dtype=I32)),
    (("write", "norm"), "slot_mapping", lambda: z(5, dtype=I32)),
    (("write", "norm"), "slot_mapping", lambda: z(4, dtype=I64)),
    (("write", "norm"), "value", lambda: z(5, HKV, D, dtype=F32)),
    (("write", "norm"), "value", lambda: z(4, HKV, D)),
    (("write", "norm"), "value", lambda: z(5, HKV, 2 * D)[:, :, ::2]),
    (("write", "norm"), "key", lambda: z(5, 2 * HKV, D)[:, ::2]),
    (("write", "norm"), "key", lambda: z(5, HKV, D, dtype=torch.float16)),
    (("gather",), "total_k", -1), (("gather",), "key", lambda: z(8, HKV, D)),
    (("gather",), "value", lambda: z(9, HKV, D, dtype=F32)),
    (("gather",), "cu_seq_lens_k", lambda: z(5, dtype=I32)),
    (("gather",), "cu_seq_lens_k", lambda: z(0, dtype=I32)),
    (("gather", "decode", "tree"), "block_table", lambda: z(3, 4, dtype=I64)),
    (("gather", "decode", "tree"), "block_table", lambda: z(2, 4, dtype=I32)),
    (("gather", "decode", "tree"), "block_table", lambda: z(3, 8, dtype=I32)[:, ::2]),
    (("decode", "tree"), "q", lambda: z(3, 8, D, dtype=F32)),
    (("decode", "tree"), "q", lambda: z(3, 8, 128)),
    (("decode", "tree"), "q", lambda: z(11, 16, D)[:, ::2]),
    (("decode", "tree"), "out", lambda: z(3, 4, D)), (("decode", "tree"), "lse", lambda: z(3, 8)),
    (("decode", "tree"), "sink", lambda: z(7, dtype=F32)),
    (("decode", "tree"), "alibi_slopes", lambda: z(8)),
    (("decode", "tree"), "cache_seqlens", lambda: z(4, dtype=I32)),
    (("decode", "tree"), "cache_seqlens", lambda: z(3, dtype=I64)),
    (("tree",), "workspace", lambda: z(16, dtype=U8)),
    (("tree",), "cu_seq_lens_q", lambda: z(3, dtype=I32)),
    (("tree",), "tree_mask", lambda: z(11, 1, dtype=I32)),
    (("tree",), "tree_mask", lambda: z(10, 1, dtype=I64)),
    (("tree",), "max_seqlen_q", 65),
    (("tree",), "tree_depth", lambda: z(11, dtype=I64)),
    (("tree",), "tree_depth", lambda: z(10, dtype=I32)),
    (("norm",), "positions", lambda: z(5, dtype=I32)),
    (("norm",), "cos_sin", lambda: z(99, D // 2, 2)),
    (("norm",), "cos_sin", lambda: z(99, D, dtype=F32)),
    (("norm",), "rotary_dim", 32), (("norm",), "q_weight", None), (("norm",), "k_weight", None),
    (("norm",), "q_weight", lambda: z(D)), (("norm",), "k_weight", lambda: z(D + 1, dtype=F32)),
    (("norm",), "query", lambda: z(5, 8 * D)), (("norm",), "query_out", lambda: z(5, 4, D)),
    (("norm",), "key_out", lambda: z(5, HKV, D, dtype=F32)),
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
    assert not [n for n, _ in lib.calls if not n.endswith("_workspace_size")]


@pytest.mark.parametrize("kw", [dict(window_left=5), dict(alibi_slopes=torch.zeros(8))])
def test_tree_needs_depths_for_positions(lib, kw):
    args = _tree_args()
    args["tree_depth"] = None
    pkv.paged_tree_attention(**args)
    with pytest.raises(ValueError, match="tree_depth"):
        pkv.paged_tree_attention(**args, **kw)


def test_decode_refuses_a_short_workspace(lib):
    args = _decode_args()
    args.update(max_seqlen=600, workspace=torch.zeros(16, dtype=U8))
    with pytest.raises(ValueError, match="workspace"):
        pkv.paged_decode_fp8(**args)


@pytest.mark.parametrize("call", ALL)
def test_cpu_tensors_are_refused(call):
    f, make = CALLS[call]
    with pytest.raises(ValueError, match="CUDA"):
        f(**make())


def test_status_codes_become_exceptions(lib, monkeypatch):
    monkeypatch.setattr(_Recorder, "__getattr__", lambda self, n: (
        getattr(self.real, n) if n == "pkv_status_string" else lambda *a: 2))
    for call, name in (("write", "reshape_and_cache_fp8"), ("gather", "gather_cache_fp8"),
                       ("decode", "paged_decode_fp8"), ("tree", "paged_tree_attention"),
                       ("norm", "qk_norm_rope_reshape_and_cache")):
        f, make = CALLS[call]
        with pytest.raises(pkv.PkvError, match=f"pkv_{name}"):
            f(**make())
