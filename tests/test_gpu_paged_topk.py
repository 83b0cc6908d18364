"""The indexer's selection over the 8-bit paged cache against the choice in 64 bits, and a server's
steps: plan, rotated writes of rows and index keys, selection, attention, release."""
import math

import pytest
import torch

from bwd_sparse_mqa_gb300 import (_lib, paged_indexer_topk, paged_indexer_topk_workspace_bytes, paged_kv_append, paged_plan,
                                  paged_release, sparse_mqa_paged_fwd)
from bwd_sparse_mqa_gb300.api import device_status
from tests import _paged, _topk as ref

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _case(lens, new, H, D, page, seed, spread=1, W=None, extra=3):
    """(q, w, cache, scales, table, seq, req, pos) of requests with `lens` positions of which the
    last `new` are this call's tokens."""
    g = torch.Generator().manual_seed(seed)
    W = W or max(-(-n // page) for n in lens)
    n_pages = sum(-(-n // page) for n in lens) + extra
    cache, scale = _paged.fill_cache(n_pages, page, D, seed, spread=spread)
    table, _ = _paged.deal(lens, page, W, n_pages, seed)
    req = [r for r, q in enumerate(new) for _ in range(q)]
    pos = [n - q + i for n, q in zip(lens, new) for i in range(q)]
    T = len(req)
    q = torch.randn(T, H, D, generator=g).bfloat16()
    w = torch.randn(T, H, generator=g) * (H * D) ** -0.5
    return [q.cuda(), w.cuda(), cache.cuda(), scale.cuda(), table.cuda(), _i32(lens), _i32(req), _i32(pos)]


def _check(c, topk, block=1, recent=0, pos=True, **kw):
    q, w, cache, scale, table, seq, req, p = c
    p = p if pos else None
    got = paged_indexer_topk(q, w, cache, scale, table, seq, req, p, topk, block, recent, check_status=True, **kw)
    val = cache.view(torch.uint8).view(torch.float8_e4m3fn).double()
    want = ref.paged(q, w, val, scale.double(), table, seq, req, p, topk, block, recent)
    bad = (got.long() != want).any(1)
    assert not bad.any(), f"{int(bad.sum())} tokens differ, the first: {int(bad.nonzero()[0])}"
    return got


CASES = [  # lens, new, H, D, page, topk
    ([1], [1], 1, 64, 16, 1), ([300], [1], 64, 128, 64, 32), ([1000, 17, 400], [1, 1, 1], 64, 128, 64, 128),
    ([333, 1000, 50, 129], [5, 3, 50, 1], 24, 64, 16, 100), ([2000, 700], [40, 9], 128, 128, 128, 256), ([500] * 20, [1] * 20, 16, 64, 32, 64),
    ([900, 900], [7, 30], 65, 128, 64, 77), ([4000], [3], 33, 128, 32, 2048), ([20, 30], [20, 30], 16, 64, 16, 8),
    ([9000, 100], [1, 1], 8, 64, 16, 1000),
]


@pytest.mark.parametrize("case", CASES)
def test_sizes(case):
    lens, new, H, D, page, topk = case
    c = _case(lens, new, H, D, page, sum(lens))
    _check(c, topk)
    _check(c, topk, pos=False)


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("block", [2, 16, 32, 64, 128])
def test_blocks(page, block):
    c = _case([1500, 700, 130], [2, 6, 3], 16, 64, page, block)
    _check(c, 256, block)
    _check(c, 512, block, recent=100)


@pytest.mark.parametrize("spread", [0, 6, 20])
def test_page_scales_far_apart(spread):
    _check(_case([1500, 800], [3, 4], 48, 128, 16, spread, spread=spread), 200)


def test_holes_padding_and_lengths():
    """Pages that are not there, tokens of no request, lengths past the table, of 0 and below."""
    c = _case([700, 400, 320, 64], [6, 5, 3, 2], 16, 64, 16, 1)
    table, seq, req = c[4], c[5], c[6]
    table[0, 3], table[0, 20:25], table[1, 0] = -1, 10 ** 6, -5
    table[2] = -1
    seq[3] = 10 ** 6
    req[1], req[9] = -1, 77
    for topk, block, recent in ((64, 1, 0), (64, 64, 0), (256, 128, 30), (600, 1, 5), (1024, 16, 0)):
        _check(c, topk, block, recent)
    seq[0], seq[1] = 0, -4
    _check(c, 64)
    _check(c, 64, pos=False)


def test_rows_of_padding_tokens_are_left_alone():
    c = _case([300, 200], [3, 3], 16, 64, 16, 2)
    c[6][2] = -1
    q, w, cache, scale, table, seq, req, p = c
    out = torch.full((6, 40), 123, dtype=torch.int32, device="cuda")
    ws = torch.full((paged_indexer_topk_workspace_bytes(_lib.PagedShape(6, 2, 16, 64, 40, 16, table.shape[1], cache.shape[0])),), 255,
                    dtype=torch.uint8, device="cuda")
    assert paged_indexer_topk(*c, 40, out=out, workspace=ws) is out
    assert out[2].eq(123).all()
    fresh = paged_indexer_topk(*c, 40)
    assert fresh[2].eq(-1).all() and torch.equal(fresh[[0, 1, 3, 4, 5]], out[[0, 1, 3, 4, 5]])
    assert paged_indexer_topk(q[:0], w[:0], cache, scale, table, seq, req[:0], p[:0], 40).shape == (0, 40)


def test_garbage_behind_a_length_and_nan_codes():
    """Codes behind a request's length do not matter; NaN codes within it rank last."""
    c = _case([500, 300], [4, 4], 16, 64, 64, 3)
    want = _check(c, 100)
    cache, table = c[2], c[4]
    codes = cache.view(torch.uint8)
    codes[table[0, 7].long(), 500 - 448:] = 0x7f
    codes[table[1, 4].long(), 300 - 256:] = 0xff
    assert torch.equal(paged_indexer_topk(*c, 100), want)
    codes[table[0, 1].long(), 10:20, 5] = 0x7f
    _check(c, 100)
    _check(c, 492)
    _check(c, 128, 32)


def test_queries_beyond_two_pieces():
    """Query elements far below the row's largest are rounded in the tensor core's pieces; the
    choice is still that of the exact values."""
    c = _case([3000], [6], 32, 128, 64, 5)
    c[0] *= torch.exp2(torch.randint(-24, 1, c[0].shape, generator=torch.Generator().manual_seed(2)).float()).cuda().bfloat16()
    _check(c, 700)
    c[0][:, :, 0] = 2.0 ** 20
    _check(c, 700)
    c[0] *= 2.0 ** -100
    _check(c, 512, 8)


def test_ties():
    c = _case([4000], [3], 4, 64, 64, 6)
    codes = c[2].view(torch.uint8)
    codes[5:40] = codes[4]
    c[3].fill_(0.25)
    for topk in (100, 1500, 3000):
        _check(c, topk)
    codes.zero_()
    _check(c, 77)


@pytest.mark.parametrize("n,topk,block", [(8200, 2048, 1), (66000, 2048, 1), (66000, 2048, 64)])
def test_long_contexts(n, topk, block):
    _check(_case([n, 500], [1, 2], 16, 64, 128, 7), topk, block, recent=1)


def test_chunks():
    """More scores than a call keeps at once (a wide table)."""
    c = _case([900, 1300], [300, 300], 16, 64, 16, 8, W=4000)
    shp = _lib.PagedShape(600, 2, 16, 64, 64, 16, 4000, c[2].shape[0])
    assert paged_indexer_topk_workspace_bytes(shp) < 600 * 64000 * 4
    _check(c, 64)


@pytest.mark.parametrize("D", [64, 128])
def test_many_calls_in_a_row(D):
    """Key tiles that come early and late (another stream copies meanwhile): a warp that took one
    round of the ring for another would give other positions or run out of its wait."""
    c = _case([9000 + 37 * i for i in range(100)], [1] * 100, 64, D, 64, 11)
    q, w, cache, scale, table, seq, req, pos = c
    first = paged_indexer_topk(q, w, cache, scale, table, seq, req, pos, 256, check_status=True)
    for t in (0, 41, 99):
        one = [q[t:t + 1], w[t:t + 1], cache, scale, table, seq, req[t:t + 1], pos[t:t + 1]]
        assert torch.equal(_check(one, 256)[0], first[t])
    side = torch.cuda.Stream()
    a = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    b = torch.empty_like(a)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(400):
        if i % 4 == 0:
            with torch.cuda.stream(side):
                b.copy_(a)
        got = paged_indexer_topk(q, w, cache, scale, table, seq, req, pos, 256)
        wrong += (got != first).sum()
    torch.cuda.synchronize()
    assert int(wrong) == 0 and device_status() == 0


def test_server_steps():
    """Prompts, then decoding with one graph: rows and index keys written rotated, positions
    chosen, attention over them, a request finished and its pages used again."""
    R, page, n_pages, W, H, D, HI, DI, topk = 3, 16, 40, 12, 16, 64, 8, 128, 24
    g = torch.Generator().manual_seed(3)
    ang = torch.arange(256, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, 64, 2).double() / 64)
    cs = torch.cat([torch.cos(ang), torch.sin(ang)], 1).float().cuda()
    zero = lambda d: torch.zeros(n_pages, page, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # noqa: E731
    kvc, kvs, ic, isc = zero(D), torch.ones(n_pages, device="cuda"), zero(DI), torch.ones(n_pages, device="cuda")
    table = torch.full((R, W), -1, dtype=torch.int32, device="cuda")
    free, count = torch.randperm(n_pages, generator=g).int().cuda(), _i32([n_pages])
    ctx = _i32([0, 0, 0])
    sink = torch.randn(H, generator=g).cuda()
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731

    def step(query, N, kv, ki, qi, wi, q):
        plan = paged_plan(ctx, query, table, free, count, page, N, n_pages, inplace=True)
        paged_kv_append(kv, plan.slot_mapping, kvc, kvs, plan.positions, cs)
        paged_kv_append(ki, plan.slot_mapping, ic, isc, plan.positions, cs, rope_offset=0)
        idx = paged_indexer_topk(qi, wi, ic, isc, plan.block_table, plan.seq_lens, plan.token_req, plan.positions, topk, recent=4)
        o, lse = sparse_mqa_paged_fwd(q, kvc, kvs, sink, plan.block_table, plan.seq_lens, plan.token_req, plan.positions, idx)
        ctx.copy_(plan.seq_lens)
        return plan, idx, o, lse

    def verify(plan, idx, o, lse, qi, wi, q):
        val = ic.view(torch.uint8).view(torch.float8_e4m3fn).double()
        want = ref.paged(qi, wi, val, isc.double(), table, plan.seq_lens, plan.token_req, plan.positions, topk, 1, 4)
        assert torch.equal(idx.long(), want)
        a = _paged.attn(q.cpu(), _paged.codes(kvc), kvs.cpu().double(), sink.cpu(), table.cpu(), plan.seq_lens.tolist(),
                        plan.token_req.tolist(), plan.positions.tolist(), idx.cpu())
        live = (plan.token_req >= 0).cpu()
        _paged.check_attn((o.cpu()[live], lse.cpu()[live]), tuple(x[live] for x in a))

    def inputs(N):
        return r(N, D).bfloat16(), r(N, DI).bfloat16(), r(N, HI, DI).bfloat16(), r(N, HI) * 0.05, r(N, H, D).bfloat16()
    x = inputs(120)
    verify(*step(_i32([50, 7, 60]), 120, *x), x[2], x[3], x[4])
    buf = [v.clone() for v in inputs(4)]
    one = _i32([1, 1, 1])
    step(one, 4, *buf)                                   # (warm-up; also a step)
    graph = torch.cuda.CUDAGraph()
    saved = [t.clone() for t in (kvc.view(torch.uint8), kvs, ic.view(torch.uint8), isc, table, free, count, ctx)]
    with torch.cuda.graph(graph):
        out = step(one, 4, *buf)
    for t, s in zip((kvc.view(torch.uint8), kvs, ic.view(torch.uint8), isc, table, free, count, ctx), saved):
        t.copy_(s)
    for i in range(20):
        for d, s in zip(buf, inputs(4)):
            d.copy_(s)
        graph.replay()
        verify(*out, buf[2], buf[3], buf[4])
        if i == 9:
            paged_release(table, torch.tensor([False, True, False], device="cuda"), free, count, n_pages, ctx)
    assert device_status() == 0


def test_bounded_wait_runs_out():
    lib = _lib.load()
    c = _case([2000, 1500], [1, 1], 64, 128, 64, 9)
    want = paged_indexer_topk(*c, 100)
    lib.smqa_set_wait_limit_ns(50_000_000)
    try:
        for cta in (0, 20):
            lib.smqa_debug_stall(cta)
            with pytest.raises(_lib.SMQAError):
                paged_indexer_topk(*c, 100, check_status=True)
            lib.smqa_debug_stall(-1)
            assert device_status(clear=True) == _lib.SMQA_ERR_DEVICE_TIMEOUT
            assert torch.equal(paged_indexer_topk(*c, 100, check_status=True), want)
    finally:
        lib.smqa_debug_stall(-1)
        lib.smqa_set_wait_limit_ns(0)
        device_status(clear=True)


def test_refusals():
    c = _case([100, 90], [1, 1], 16, 64, 16, 1)
    names = ["index_q", "weights", "k_cache", "k_scales", "block_table", "seq_lens", "token_req", "positions"]
    call = lambda topk=8, block_size=1, recent=0, **k: paged_indexer_topk(**{**dict(zip(names, c)), **k}, topk=topk, block_size=block_size, recent=recent)  # noqa: E731,E501
    call()
    for bad in ({"index_q": c[0][:, :, :32].contiguous()}, {"weights": c[1][:1]}, {"k_scales": c[3][:2]}, {"seq_lens": c[5][:1]},
                {"token_req": c[6][:1]}, {"positions": c[7][:1]}, {"index_q": c[0].transpose(0, 1)}, {"block_table": c[4].t()},
                {"k_cache": c[2].cpu()}, {"topk": 2 ** 31}):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in ({"index_q": c[0].half()}, {"k_cache": c[2].view(torch.uint8)}, {"token_req": c[6].long()}, {"positions": c[7].float()}):
        with pytest.raises(TypeError):
            call(**bad)
    for kw in ({"topk": 0}, {"topk": 6, "block_size": 4}, {"block_size": 256, "topk": 256}, {"recent": 9}):
        with pytest.raises(_lib.SMQAError):
            call(**kw)
    with pytest.raises(_lib.SMQAError):
        call(index_q=torch.zeros(2, 16, 512, dtype=torch.bfloat16, device="cuda"),
             k_cache=torch.zeros(9, 16, 512, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), k_scales=torch.ones(9, device="cuda"))
