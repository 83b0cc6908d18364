"""The indexer's selection over contiguous keys against the choice in 64 bits, position by
position: sizes, blocks, ties, borders closer than the tensor core's sums can tell, values that are
no numbers, long rows, chunks, streams and captures."""
import math

import pytest
import torch

from bwd_sparse_mqa_gb300 import _lib, indexer_topk, indexer_topk_workspace_bytes, sparse_mqa, sparse_mqa_fwd_interface
from bwd_sparse_mqa_gb300.api import device_status
from tests import _topk as ref

pytestmark = pytest.mark.gpu


def _inputs(B, S, S_kv, H, D, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return r(B, S, H, D).bfloat16(), r(B, S, H) * (H * D) ** -0.5, r(B, S_kv, D).bfloat16()


def _check(q, w, k, topk, block=1, recent=0, first=None, **kw):
    got = indexer_topk(q, w, k, topk, block, recent, first, check_status=True, **kw)
    assert got.dtype == torch.int32
    want = ref.flat(q, w, k, topk, block, recent, first)
    bad = (got.long() != want).any(2)
    assert not bad.any(), f"{int(bad.sum())} tokens differ, the first at {bad.nonzero()[0].tolist()}"
    return got


SIZES = [  # B, S, S_kv, H, D, topk
    (1, 1, 1, 1, 64, 1), (1, 1, 2, 1, 64, 1), (2, 5, 5, 16, 64, 3), (1, 128, 128, 16, 64, 32), (3, 33, 700, 64, 128, 128),
    (1, 17, 129, 128, 128, 127), (2, 9, 1000, 65, 64, 100), (1, 40, 513, 24, 128, 512), (1, 37, 300, 33, 128, 7), (1, 3, 8192, 8, 64, 2048),
    (1, 20, 3000, 48, 128, 1500), (1, 200, 200, 100, 64, 64), (1, 50, 4000, 2, 128, 1), (1, 16, 257, 16, 128, 256),
]


@pytest.mark.parametrize("size", SIZES)
def test_sizes(size):
    B, S, S_kv, H, D, topk = size
    _check(*_inputs(B, S, S_kv, H, D, S_kv), topk)


@pytest.mark.parametrize("H", [5, 16, 20, 32, 50, 64, 90])
def test_every_size_of_a_group_of_tokens(H):
    """Groups of 1 to 16 tokens: their columns go to one, two or all of the warps that sum them;
    the last group of a batch element is followed by another element's tokens, or by none."""
    for S in range(1, 18):
        _check(*_inputs(2, S, 300 + 40 * S, H, 64 if S & 1 else 128, S), 40)


@pytest.mark.parametrize("block", [2, 4, 8, 16, 32, 64, 128])
@pytest.mark.parametrize("recent", [0, 1, 100])
def test_blocks_and_recent_positions(block, recent):
    q, w, k = _inputs(2, 30, 1501, 16, 64, block)
    _check(q, w, k, 4 * 128, block, recent)
    _check(q, w, k, 4 * 128, block, recent, first=700)


@pytest.mark.parametrize("first", [0, -7, -1000, 10, 499, 10 ** 6, 2 ** 40, -2 ** 40])
def test_positions_of_the_queries(first):
    """Tokens that see nothing, some or all of the keys; positions beyond 32 bits."""
    q, w, k = _inputs(2, 12, 500, 16, 64, 3)
    got = _check(q, w, k, 64, first=first)
    if first < -12:
        assert got.eq(-1).all()


def test_ties_go_to_the_lowest_position():
    """Repeated keys, weights of 0, keys of 0, all scores 0: more ties than the border's list holds."""
    q, w, k = _inputs(1, 6, 5000, 16, 64, 5)
    k[:, 1000:2000] = k[:, :1000]
    k[:, 2000:3000] = k[:, 500:501]
    k[:, 3000:4000] = 0
    w[:, 1] = 0
    q[:, 2] = 0
    w[:, 3] = w[:, 3].abs()
    w[:, 4] = -w[:, 4].abs()
    for topk in (1, 700, 1500, 3500):
        _check(q, w, k, topk)
    _check(q, w, k, 1504, block=16)
    _check(q[:, :, :1].contiguous(), w[:, :, :1].contiguous(), k, 1200)


@pytest.mark.parametrize("H,D", [(1, 64), (2, 128), (4, 64)])
def test_few_heads(H, D):
    """Half, a quarter, a sixteenth of the scores are exactly 0."""
    for topk in (10, 900, 1800):
        _check(*_inputs(1, 24, 3000, H, D, topk), topk)


@pytest.mark.parametrize("H,D", [(1, 128), (16, 64), (64, 128)])
@pytest.mark.parametrize("ulps", [1, 3])
def test_borders_closer_than_the_sums(H, D, ulps):
    """Keys that differ in a few last bits: thousands of scores within the tensor core's error, of
    one sign and size (a large product beside many small ones among them)."""
    g = torch.Generator(device="cuda").manual_seed(H + ulps)
    n = 2600
    q = (torch.rand(1, 3, H, D, generator=g, device="cuda") + 0.5).bfloat16()
    base = (torch.rand(D, generator=g, device="cuda") + 1.0).bfloat16()
    k = base.expand(1, n, D).clone()
    for _ in range(ulps):
        at = torch.randint(0, D, (n,), generator=g, device="cuda")
        up = torch.randint(-1, 2, (n,), generator=g, device="cuda", dtype=torch.int16)
        rows = torch.arange(n, device="cuda")
        bits = k.view(torch.int16)
        bits[0, rows, at] += up
    w = torch.rand(1, 3, H, generator=g, device="cuda") + 0.5
    q[:, 1, :, 1:] *= 2.0 ** -9
    k2 = k.clone()
    k2[..., 1:] *= 2.0 ** -9
    for kk in (k, k2):
        _check(q, w, kk, 1000)
        _check(q, -w, kk, 17)
        _check(q, w, kk, 640, block=8)


def test_sums_that_cancel():
    """Logits far smaller than their terms: the error bound, not the score, sets the border's width."""
    g = torch.Generator(device="cuda").manual_seed(4)
    S, n, H, D = 8, 4000, 32, 128
    q = torch.randn(1, S, H, D, generator=g, device="cuda").bfloat16()
    q[..., 1::2] = -q[..., ::2]
    k = torch.randn(1, n, D, generator=g, device="cuda").bfloat16()
    k[..., 1::2] = k[..., ::2]
    k[..., 7] += torch.randn(1, n, generator=g, device="cuda").bfloat16() * 2.0 ** -6
    w = torch.randn(1, S, H, generator=g, device="cuda")
    _check(q, w, k, 1000)
    _check(q, w, k, 128, block=32)


@pytest.mark.parametrize("shift", [-60, -30, 30, 40])
def test_magnitudes(shift):
    """Keys and queries of 2^shift, one key row far larger than the others, weights far apart."""
    q, w, k = _inputs(1, 10, 2000, 16, 128, 6)
    q, k = q * 2.0 ** (shift // 2), k * 2.0 ** (shift // 2)
    k[:, 77] *= 2.0 ** 12
    w = w * torch.exp2(torch.randint(-20, 20, w.shape, generator=torch.Generator().manual_seed(1)).float()).cuda()
    _check(q, w, k, 500)
    _check(q, w, k, 512, block=64)


def test_values_that_are_no_numbers():
    """NaN ranks below every number, infinities where they belong; what a token does not see is
    never looked at."""
    q, w, k = _inputs(1, 40, 600, 16, 64, 8)
    k[0, 10], k[0, 20, 5], k[0, 30, 3], k[0, 40, 60] = math.nan, math.nan, math.inf, -math.inf
    k[0, 100:130, 7] = math.inf
    _check(q, w, k, 50)
    _check(q, w, k, 590)
    _check(q, w, k, 96, block=32)
    k2 = k.clone()
    k2[0, :300] = math.nan
    _check(q, w, k2, 320)
    _check(q, w, k2, 290)
    a = _inputs(1, 30, 400, 16, 64, 9)
    seen = indexer_topk(*a, 64, first_position=100)
    dirty = a[2].clone()
    dirty[0, 200:], dirty[0, 131:140] = math.nan, math.inf
    assert torch.equal(indexer_topk(a[0], a[1], dirty, 64, first_position=100), seen)


def test_queries_and_weights_that_are_no_numbers():
    """The choice is then unspecified, but it is one: distinct positions that the token sees,
    ascending, as many as it may have."""
    q, w, k = _inputs(1, 40, 700, 16, 64, 12)
    q[0, 1, 3, 5], q[0, 2, 0, 0], q[0, 3] = math.nan, math.inf, math.inf
    w[0, 4, 2], w[0, 5, 1], w[0, 6] = math.nan, math.inf, -math.inf
    q[0, 7], w[0, 8] = 3e38, 3e38
    for topk, block in ((100, 1), (600, 1), (128, 32)):
        got = indexer_topk(q, w, k, topk, block, check_status=True)
        good = ref.flat(q, w, k, topk, block)
        for t in range(40):
            n = 660 + t + 1
            mine = got[0, t][got[0, t] >= 0].tolist()
            assert mine == sorted(set(mine)) and mine[-1] < n and got[0, t, len(mine):].eq(-1).all()
            if block == 1:
                assert len(mine) == min(topk, n)
            if t == 0 or t > 8:
                assert torch.equal(got[0, t].long(), good[0, t])


@pytest.mark.parametrize("S_kv,topk,block", [(8193, 2048, 1), (20000, 2048, 1), (65536, 1000, 1), (70001, 2048, 1), (70001, 4096, 128)])
def test_long_rows(S_kv, topk, block):
    q, w, k = _inputs(1, 3, S_kv, 16, 64, 2)
    _check(q, w, k, topk, block, recent=5)


def test_chunks():
    """More scores than a call keeps at once; the batch elements' last groups are short."""
    q, w, k = _inputs(2, 1003, 9000, 24, 64, 3)
    shp = _lib.Shape(2, 1003, 9000, 24, 64, 96)
    assert indexer_topk_workspace_bytes(shp) < 2 * 1003 * 9000 * 4
    got = indexer_topk(q, w, k, 96, check_status=True)
    for b, t in ((0, 0), (0, 517), (0, 1002), (1, 0), (1, 511), (1, 860), (1, 1002)):
        s = ref.scores(q[b, t], w[b, t], k[b, :9000 - 1003 + t + 1])
        assert torch.equal(got[b, t].long(), ref.choose(s, 96)), (b, t)
    one = torch.cat([indexer_topk(q[b:b + 1], w[b:b + 1], k[b:b + 1], 96) for b in range(2)])
    assert torch.equal(got, one)


def test_out_workspace_streams_and_capture():
    xs = [_inputs(1, 50, 800, 64, 128, i) for i in range(3)]
    want = [indexer_topk(*x, 100) for x in xs]
    shp = _lib.Shape(1, 50, 800, 64, 128, 100)
    ws = [torch.full((indexer_topk_workspace_bytes(shp),), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    outs = [torch.empty_like(want[0]) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(30):
        for x, s, o, v in zip(xs, streams, outs, ws):
            with torch.cuda.stream(s):
                assert indexer_topk(*x, 100, out=o, workspace=v) is o
    torch.cuda.synchronize()
    for o, r in zip(outs, want):
        assert torch.equal(o, r)
    buf = [v.clone() for v in xs[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        idx = indexer_topk(*buf, 100)
    for x, r in zip(xs, want):
        for d, s in zip(buf, x):
            d.copy_(s)
        graph.replay()
        assert torch.equal(idx, r)
    assert device_status() == 0


def test_same_result_in_any_batch():
    """The choice of a token does not depend on what stands beside it."""
    q, w, k = _inputs(2, 60, 900, 64, 128, 4)
    whole = indexer_topk(q, w, k, 128)
    for t in (0, 1, 31, 59):
        one = indexer_topk(q[:, t:t + 1].contiguous(), w[:, t:t + 1].contiguous(), k, 128, first_position=840 + t)
        assert torch.equal(one[:, 0], whole[:, t])


def test_many_calls_in_a_row():
    q, w, k = _inputs(1, 300, 1200, 64, 128, 7)
    want = indexer_topk(q, w, k, 200)
    out = torch.empty_like(want)
    for _ in range(1500):
        indexer_topk(q, w, k, 200, out=out)
    assert torch.equal(out, want) and device_status() == 0


def test_bounded_wait_runs_out():
    lib = _lib.load()
    q, w, k = _inputs(1, 20, 900, 64, 128, 7)
    want = indexer_topk(q, w, k, 100)
    lib.smqa_set_wait_limit_ns(50_000_000)
    try:
        for cta in (0, 3):
            lib.smqa_debug_stall(cta)
            with pytest.raises(_lib.SMQAError):
                indexer_topk(q, w, k, 100, check_status=True)
            lib.smqa_debug_stall(-1)
            assert device_status(clear=True) == _lib.SMQA_ERR_DEVICE_TIMEOUT
            assert torch.equal(indexer_topk(q, w, k, 100, check_status=True), want)
    finally:
        lib.smqa_debug_stall(-1)
        lib.smqa_set_wait_limit_ns(0)
        device_status(clear=True)


def test_refusals():
    q, w, k = _inputs(1, 3, 20, 16, 64)
    for bad in ((q[:, :2].contiguous(), w, k), (q, w[:, :, :3].contiguous(), k), (q, w, k[:, :, :32].contiguous()), (q.transpose(1, 2), w, k),
                (q.cpu(), w, k), (q[0], w, k)):
        with pytest.raises(ValueError):
            indexer_topk(*bad, 4)
    for bad in ((q.float(), w, k), (q, w.double(), k), (q, w, k.float())):
        with pytest.raises(TypeError):
            indexer_topk(*bad, 4)
    for kw in ({"topk": 0}, {"topk": -4}, {"topk": 6, "block_size": 4}, {"topk": 256, "block_size": 256}, {"topk": 6, "block_size": 3},
               {"topk": 4, "block_size": 0}, {"topk": 4, "recent": -1}, {"topk": 4, "recent": 5}, {"topk": 16, "block_size": 8, "recent": 10}):
        with pytest.raises(_lib.SMQAError):
            indexer_topk(q, w, k, **kw)
    indexer_topk(q, w, k, 16, block_size=8, recent=9)
    for kw in ({"topk": 2 ** 31}, {"topk": 4, "block_size": 2 ** 32 + 1}, {"topk": 4, "out": torch.empty(1, 3, 5, dtype=torch.int32, device="cuda")},
               {"topk": 4, "workspace": torch.empty(10, dtype=torch.uint8)}):
        with pytest.raises(ValueError):
            indexer_topk(q, w, k, **kw)
    with pytest.raises(TypeError):
        indexer_topk(q, w, k, 4, out=torch.empty(1, 3, 4, device="cuda"))
    with pytest.raises(_lib.SMQAError):
        indexer_topk(q[..., :32].contiguous(), w, k[..., :32].contiguous(), 4)


def test_attention_over_the_choice():
    """The list goes straight into sparse_mqa, forward and backward; a token that sees fewer
    positions than it may choose attends to all of them."""
    q, w, k = _inputs(1, 40, 40, 16, 64, 11)
    idx = indexer_topk(q, w, k, 12, block_size=4, recent=3)
    g = torch.Generator(device="cuda").manual_seed(1)
    qa = torch.randn(1, 40, 16, 64, generator=g, device="cuda").bfloat16().requires_grad_()
    kv = torch.randn(1, 40, 64, generator=g, device="cuda").bfloat16().requires_grad_()
    sink = torch.zeros(16, device="cuda", requires_grad=True)
    o, lse = sparse_mqa(qa, kv, sink, idx, check_status=True)
    o.float().sum().backward()
    assert torch.isfinite(qa.grad).all() and torch.isfinite(kv.grad).all()
    every = torch.arange(40, device="cuda", dtype=torch.int32)
    dense = torch.where(every[None, None] <= every[None, :, None], every, -1).contiguous()
    o2, _ = sparse_mqa_fwd_interface(qa.detach(), kv.detach(), sink.detach(), dense)
    assert torch.equal(o[:, :12], o2[:, :12]) and not torch.equal(o[:, 39], o2[:, 39])
