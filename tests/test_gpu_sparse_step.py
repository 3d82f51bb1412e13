"""A serving loop of the sparse step, as it is used: block tables and slots from
lengths, the fused norm, rotation and cache write, the pages' bounds, the choice of
pages and the attention over them; eagerly and captured in one graph."""
import pytest
import torch

import paged_kv_cache_attention_gb300 as pkv
from tests import _fp8 as R
from tests import _sparse as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, I32, I64, U8, I8 = torch.bfloat16, torch.int32, torch.int64, torch.uint8, torch.int8
HQ, HKV, D, BS, NB, B, TOP = 8, 2, 64, 16, 200, 4, 6


class Server:
    def __init__(self, fp8, seed):
        g = torch.Generator().manual_seed(seed)
        self.fp8 = fp8
        kv = torch.zeros(2, NB, BS, HKV, D, device=DEV)
        self.kc, self.vc = kv.to(R.E4M3 if fp8 else BF16)
        self.ks, self.vs = torch.zeros(2, NB, HKV, BS, dtype=U8, device=DEV) if fp8 else (None, None)
        self.bounds = torch.zeros(NB, HKV, 2, D, dtype=I8, device=DEV)
        self.bscale = torch.zeros(NB, HKV, dtype=U8, device=DEV)
        self.table = torch.full((B, 40), -1, dtype=I32, device=DEV)
        self.free = torch.randperm(NB, generator=g).to(I32).to(DEV)
        self.num_free = torch.tensor([NB], dtype=I32, device=DEV)
        self.cos_sin = pkv.rope_cos_sin_table(1024, D)
        self.one = torch.ones(D, device=DEV)
        self.err = torch.zeros(1, dtype=I32, device=DEV)

    def step(self, qkv, old, new):
        rows = qkv.shape[0]
        slots, pos, cu_q, _ = pkv.update_block_tables(self.table, old, new, self.free, self.num_free,
                                                      BS, rows, dev_error=self.err)
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        out_q = torch.zeros(rows, HQ, D, dtype=BF16, device=DEV)
        out_k = torch.zeros(rows, HKV, D, dtype=BF16, device=DEV)
        pkv.qk_norm_rope_reshape_and_cache(q, k, v, self.kc, self.vc, pos, slots, self.cos_sin,
                                           self.one, self.one, query_out=out_q, key_out=out_k,
                                           k_scale=self.ks, v_scale=self.vs, dev_error=self.err)
        pkv.update_page_bounds(self.kc, self.bounds, self.bscale, slots, k_scale=self.ks,
                               dev_error=self.err)
        pages = pkv.select_pages(out_q, self.bounds, self.bscale, self.table, new, 640, TOP, BS,
                                 cu_seq_lens_q=cu_q, dev_error=self.err)
        lse = torch.zeros(rows, HQ, device=DEV)
        out = torch.zeros(rows, HQ, D, dtype=BF16, device=DEV)
        pkv.paged_sparse_attention(out_q, self.kc, self.vc, self.table, new, pages,
                                   cu_seq_lens_q=cu_q, k_scale=self.ks, v_scale=self.vs, out=out,
                                   lse=lse, dev_error=self.err)
        return out_q, pages, out, lse


class Held:
    """What the pools hold, read back, in place of tests._fp8.Pools."""

    def __init__(self, server):
        self.rows = []
        for c, s in ((server.kc, server.ks), (server.vc, server.vs)):
            if s is None:
                x = c.cpu().to(torch.float64)
            else:
                x = R.CODE_VALUES[c.view(U8).cpu().long()] * \
                    R.scales(s.cpu()).transpose(1, 2)[..., None]
            self.rows.append(x.reshape(NB * BS, HKV, D))

    def at(self, slots):
        return [x[slots] for x in self.rows]


def check(server, outs, old, new):
    """The selection and the attention of the step from what the pools hold now."""
    q, pages, out, lse = (x.cpu() for x in outs)
    table = server.table.cpu().long()
    pools = Held(server)
    slots, want = [], []
    for r, n in enumerate(new):
        p = torch.arange(n)
        slots.append(table[r, p // BS] * BS + p % BS)
    queries = [max(0, b - a) for a, b in zip(old, new)]
    rows = S.rows_of(queries, new)
    for t, (r, n) in enumerate(rows):
        codes, byte = [], []
        for p in range(S.pages_of(n, BS)):   # a page's keys as of its last write
            k, _ = pools.at(slots[r][p * BS:(p + 1) * BS])
            c, b = S.bounds(k.transpose(0, 1))
            codes.append(c)
            byte.append(b)
        want.append(S.choose(S.scores(q[t], torch.stack(codes), torch.stack(byte)), TOP, 1, 1))
    m = len(rows)
    if m:
        assert torch.equal(pages[:m], torch.stack(want))
        ref, rl, absv, smax, floor = S.attend_lists(q[:m], pools, slots, rows, pages[:m], BS,
                                                    D ** -0.5, None)
        bound = R.out_bound(ref, absv, smax, D, 2.0 ** -11, floor) if server.fp8 else \
            R.out_bound(ref, absv, smax, D, 2.0 ** -8)
        R.assert_within(out[:m], ref, bound, "out")
        R.assert_within(lse[:m], rl, R.lse_bound(rl, smax, D), "lse")
    assert bool((out[m:] == 0).all())
    assert pkv.get_device_error(server.err) == 0


def qkv(rows, g):
    return torch.randn(rows, HQ + 2 * HKV, D, generator=g).to(BF16).to(DEV)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_serving_loop(fp8):
    """Prompts, a chunk, decode steps, drafts taken back, a request done and another
    in its place, padded rows."""
    s, g = Server(fp8, 1), torch.Generator().manual_seed(2)
    plan = [[0, 0, 0, 0], [300, 17, 0, 150], [301, 18, 64, 151], [305, 22, 65, 160],
            [302, 22, 66, 155], [303, 0, 67, 156], [304, 200, 68, 157], [305, 201, 100, 158]]
    for old, new in zip(plan, plan[1:]):
        rows = sum(max(0, b - a) for a, b in zip(old, new)) + 3
        outs = s.step(qkv(rows, g), torch.tensor(old, dtype=I32, device=DEV),
                      torch.tensor(new, dtype=I32, device=DEV))
        check(s, outs, old, new)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_captured_step(fp8):
    """One graph for every step of up to 8 tokens: only lengths and rows are copied in."""
    s, g = Server(fp8, 3), torch.Generator().manual_seed(4)
    old, new = [0] * 4, [290, 33, 0, 120]
    s.step(qkv(sum(new), g), torch.tensor(old, dtype=I32, device=DEV),
           torch.tensor(new, dtype=I32, device=DEV))
    rows = torch.zeros(8, HQ + 2 * HKV, D, dtype=BF16, device=DEV)
    do, dn = (torch.tensor(new, dtype=I32, device=DEV) for _ in range(2))
    s.step(rows, do, dn)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = s.step(rows, do, dn)
    for to in ([291, 34, 2, 121], [294, 35, 2, 119], [295, 36, 5, 120], [296, 0, 6, 125], [297, 4, 7, 126]):
        old, new = new, to
        rows.copy_(qkv(8, g))
        do.copy_(torch.tensor(old))
        dn.copy_(torch.tensor(new))
        graph.replay()
        check(s, outs, old, new)


def test_a_step_without_free_pages_does_nothing():
    """Too few pages: an error word, empty outputs, the cache and its bounds untouched,
    and the same step goes through once there are pages again."""
    s, g = Server(False, 5), torch.Generator().manual_seed(6)
    old, new = [0] * 4, [300, 17, 40, 150]
    d = [torch.tensor(x, dtype=I32, device=DEV) for x in (old, new)]
    s.step(qkv(sum(new), g), *d)
    s.num_free.fill_(1)
    state = [x.clone() for x in (s.kc, s.vc, s.bounds, s.bscale, s.table, s.free, s.num_free)]
    more = [320, 60, 41, 151]
    x = qkv(20 + 43 + 2, g)
    dm = torch.tensor(more, dtype=I32, device=DEV)
    outs = s.step(x, d[1], dm)
    assert pkv.get_device_error(s.err, clear=True) & pkv.DEVERR_NO_BLOCKS
    assert bool((outs[2] == 0).all())
    for a, b in zip(state, (s.kc, s.vc, s.bounds, s.bscale, s.table, s.free, s.num_free)):
        assert torch.equal(a, b)
    s.num_free.fill_(NB - 34)
    check(s, s.step(x, d[1], dm), new, more)
