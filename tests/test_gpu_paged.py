"""The paged-cache operators on the GPU against plain 64-bit forms, element by
element within derived bounds (tests/_paged.py), at the sizes, masks and lengths
where they can go wrong, alone and together."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from bwd_sparse_mqa_gb300 import (_lib, paged_kv_append, paged_plan, paged_release,
                                  sparse_mqa_fwd_interface, sparse_mqa_paged_fwd)
from bwd_sparse_mqa_gb300.api import device_status
from tests import _paged as ref

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------- plan
PLANS = {
    "one token": ([0], [1], 16, 4, 1, 3),
    "decode": ([15, 16, 17, 0, 31, 32], [1] * 6, 16, 4, 6, 20),
    "prompts": ([0, 5, 64, 0, 100], [130, 0, 64, 1, 29], 64, 8, 240, 9),
    "nothing new": ([3, 0, 40], [0, 0, 0], 32, 2, 4, 5),
    "padded and negative": ([-5, 10, 0], [3, -2, 7], 16, 3, 33, 8),
    "tokens past max_tokens": ([10, 20], [50, 50], 16, 9, 60, 12),
    "stack runs out": ([0, 30, 0], [40, 40, 100], 16, 8, 200, 4),
    "positions past the table": ([30, 0], [40, 90], 16, 3, 140, 9),
    "one wide row": ([0], [5000], 16, 400, 5003, 330),
    "no stack": ([0, 3], [2, 2], 16, 2, 5, 0),
}


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("name", PLANS)
def test_plan(name, inplace):
    ctx, qry, page, W, N, pool = PLANS[name]
    n_pages = 1000
    lens = [min(max(c, 0), W * page) for c in ctx]
    table, free = ref.deal(lens, page, W, n_pages, 1)
    free = free[:pool]
    want = ref.plan(ctx, qry, table.tolist(), free.tolist(), pool, page, N, n_pages)
    t, c = table.cuda(), _i32([pool])
    got = paged_plan(_i32(ctx), _i32(qry), t, free.cuda(), c, page, N, n_pages, inplace=inplace)
    for g, w, f in zip(got, want, got._fields):
        assert g.tolist() == w, f
    if inplace:
        assert got.block_table is t and got.free_count is c
    else:
        assert t.tolist() == table.tolist() and int(c) == pool


@pytest.mark.parametrize("R", [1, 1023, 1025, 5000, 16384])
def test_plan_many_requests(R):
    g = torch.Generator().manual_seed(R)
    ctx = torch.randint(0, 60, (R,), generator=g).tolist()
    qry = torch.randint(0, 4, (R,), generator=g).tolist()
    table, free = ref.deal(ctx, 16, 5, 6 * R + 5, 2)
    want = ref.plan(ctx, qry, table.tolist(), free.tolist(), free.numel(), 16, 3 * R, 6 * R + 5)
    for inplace in (False, True):
        got = paged_plan(_i32(ctx), _i32(qry), table.cuda(), free.cuda(), _i32([free.numel()]),
                         16, 3 * R, 6 * R + 5, inplace=inplace)
        for a, b, f in zip(got, want, got._fields):
            assert a.tolist() == b, f


def test_plan_negative_count_and_bad_pages():
    """A stack count below 0 is empty; page ids outside the pool give no slot."""
    got = paged_plan(_i32([0]), _i32([3]), _i32([[-1]]), _i32([7, 8]), _i32([-4]), 16, 3, 9)
    assert got.block_table.tolist() == [[-1]] and got.free_count.tolist() == [-1]
    assert got.slot_mapping.tolist() == [-1, -1, -1]
    got = paged_plan(_i32([2]), _i32([20]), _i32([[99, -1]]), _i32([3, 12]), _i32([2]), 16, 20, 10)
    assert got.block_table.tolist() == [[99, 12]] and got.slot_mapping.tolist() == [-1] * 20


def test_release_gives_back_what_plan_took():
    page, W, n_pages, R = 16, 40, 300, 70
    ctx = [(r * 37) % 600 for r in range(R)]
    ctx = [c if r % 9 == 0 else c % 40 for r, c in enumerate(ctx)]
    table, free = ref.deal(ctx, page, W, n_pages, 5)
    pool = torch.full((n_pages,), -1, dtype=torch.int32)
    pool[:free.numel()] = free
    t, f, c, seq = table.cuda(), pool.cuda(), _i32([free.numel()]), _i32(ctx)
    gone = torch.tensor([r % 3 == 0 for r in range(R)])
    paged_release(t, gone.cuda(), f, c, n_pages, seq)
    back = [p for r in range(R) if gone[r] for p in table[r].tolist() if p >= 0]
    assert c.tolist() == [free.numel() + len(back)]
    assert f.tolist()[:free.numel() + len(back)] == free.tolist() + back
    for r in range(R):
        assert t[r].tolist() == ([-1] * W if gone[r] else table[r].tolist())
        assert int(seq[r]) == (0 if gone[r] else ctx[r])
    paged_release(t, torch.ones(R, dtype=torch.bool, device="cuda"), f, c, n_pages)
    assert sorted(f.tolist()) == list(range(n_pages)) and int(c) == n_pages
    paged_release(t, torch.ones(R, dtype=torch.bool, device="cuda"), f, c, n_pages)
    assert int(c) == n_pages


# ------------------------------------------------------------------------------------- append
def _check_append(new, slot, cache, scale):
    page = cache.shape[1]
    want, want_s = ref.append(new, slot, ref.codes(cache), scale.double(), page)
    c, s = cache.cuda(), scale.cuda()
    back = paged_kv_append(new.cuda(), _i32(slot), c, s)
    assert back[0] is c and back[1] is s
    assert torch.equal(s.cpu().double(), want_s)
    got = ref.codes(c)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    return c, s


@pytest.mark.parametrize("D", [64, 512])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_prompts_and_tokens(D, page):
    """Whole pages, runs that start and end inside a page, single tokens, skipped rows."""
    cache, scale = ref.fill_cache(9, page, D, 3, spread=2)
    slot = (list(range(5 * page, 7 * page + 3))            # two pages and three rows
            + [-1, 9 * page, 2 ** 31 - 1]                  # skipped
            + list(range(page + 5, 2 * page))              # the rest of page 1
            + [3 * page + page - 1, 8 * page, 2 * page + 7])
    g = torch.Generator().manual_seed(page)
    new = (torch.randn(len(slot), D, generator=g) *
           torch.exp2(torch.randint(-4, 5, (len(slot), 1), generator=g).float())).bfloat16()
    _check_append(new, slot, cache, scale)


@pytest.mark.parametrize("D", [64, 512])
@pytest.mark.parametrize("page", [32, 128])
def test_append_runs_of_all_lengths_under_growing_scales(D, page):
    """Runs of every length up to a page, in an order that mixes short and long ones, each in a
    page of its own behind earlier rows whose codes have to be rescaled (or not)."""
    g = torch.Generator().manual_seed(D + page)
    lens = torch.randperm(page, generator=g)[:40].add(1).tolist() + [1] * 20 + [4, 5, 30, 31, 32, page]
    cache, scale = ref.fill_cache(len(lens), page, D, 11, spread=2)
    slot, mag = [], []
    for i, n in enumerate(lens):
        off = int(torch.randint(0, page - n + 1, (1,), generator=g))
        slot += [i * page + off + j for j in range(n)]
        mag += [2.0 ** (3 * (i % 4))] * n
    new = (torch.randn(len(slot), D, generator=g) * torch.tensor(mag)[:, None]).bfloat16()
    _check_append(new, slot, cache, scale)


def test_append_magnitudes():
    """Scales at the border 448 * 2^k, zero pages, the smallest and largest values, rescaling far
    enough to reach e4m3's subnormals, NaN and infinities, and values behind the run."""
    page, D = 16, 64
    cache, scale = ref.fill_cache(12, page, D, 4)
    rows = []
    for v in (448.0, 449.0, 450.0, 7.0, 7.03125, 2.0 ** -60, 2.0 ** -100, 0.0, 3.3e38, 1e-40):
        x = torch.zeros(D)
        x[::3] = v
        x[1::7] = -v * 0.37
        rows.append(x)
    new = torch.stack(rows).bfloat16()
    _check_append(new, [page * r for r in range(10)], cache, scale)          # row 0 of ten pages
    c, s = _check_append(new * 2.0 ** -3, [page * r + 1 for r in range(10)], cache, scale)
    big = torch.full((1, D), 2.0 ** 9).bfloat16()
    _check_append(big, [page * 4 + 2], c.cpu(), s.cpu())                     # far below the new scale
    odd = torch.randn(3, D).bfloat16()
    odd[0, 0], odd[1, 5], odd[2, 9] = float("nan"), float("inf"), float("-inf")
    c, s = _check_append(odd, [page * 11 + 3, page * 11 + 4, page * 11 + 5], cache, scale)
    _check_append(torch.full((1, D), float("nan")).bfloat16(), [page * 10], cache, scale)
    assert torch.equal(c.cpu().view(torch.uint8)[11, 6:], cache.view(torch.uint8)[11, 6:])


def test_append_token_by_token_equals_at_once():
    """Powers of two keep a page's codes the same whether its rows come one at a time or at
    once, as long as none falls into e4m3's subnormals."""
    page, D = 32, 512
    g = torch.Generator().manual_seed(8)
    new = (torch.randn(page, D, generator=g).abs() + 0.5).bfloat16() * torch.sign(torch.randn(page, D, generator=g)).bfloat16()
    new = (new.float() * torch.linspace(1, 3, page)[:, None]).bfloat16().cuda()
    one = torch.zeros(1, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    two, s1, s2 = one.clone(), torch.ones(1, device="cuda"), torch.ones(1, device="cuda")
    paged_kv_append(new, _i32(list(range(page))), one, s1)
    for i in range(page):
        paged_kv_append(new[i:i + 1], _i32([i]), two, s2)
    assert torch.equal(s1, s2) and torch.equal(one.view(torch.uint8), two.view(torch.uint8))


# ------------------------------------------------------------------------------------- attention
def _attn_case(lens, tokens, H, D, topk, page, seed, spread=0, W=None, mask=0.1, pad=0, extra=3):
    """Requests of the given lengths; tokens: (request, position) pairs."""
    g = torch.Generator().manual_seed(seed)
    W = W or max(1, max(-(-n // page) for n in lens)) + 1
    n_pages = sum(-(-n // page) for n in lens) + extra
    cache, scale = ref.fill_cache(n_pages, page, D, seed, spread)
    table, _ = ref.deal(lens, page, W, n_pages, seed)
    used = torch.zeros(n_pages, page, dtype=torch.bool)   # rows that hold no token hold NaN
    for r, n in enumerate(lens):
        for p in range(n):
            used[int(table[r, p // page]), p % page] = True
    raw = cache.view(torch.uint8)
    raw[~used] = 0x7f
    T = len(tokens) + pad
    x = {"q": torch.randn(T, H, D, generator=g).bfloat16(), "kv_cache": raw.view(torch.float8_e4m3fn),
         "kv_scales": scale, "attn_sink": torch.randn(H, generator=g), "block_table": table,
         "seq_lens": torch.tensor(lens, dtype=torch.int32),
         "token_req": torch.tensor([r for r, _ in tokens] + [-1] * pad, dtype=torch.int32),
         "positions": torch.tensor([p for _, p in tokens] + [-1] * pad, dtype=torch.int32),
         "topk_idxs": None}
    if topk:
        idx = torch.full((T, topk), -1, dtype=torch.int32)
        for t, (r, p) in enumerate(tokens):
            n = min(p + 1, lens[r])
            perm = torch.randperm(n, generator=g)[:topk].to(torch.int32)
            idx[t, :perm.numel()] = perm
        drop = torch.rand(T, topk, generator=g) < mask
        far = torch.randint(0, 3, (T, topk), generator=g)
        bad = torch.tensor([-1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)[far]
        x["topk_idxs"] = torch.where(drop, bad, idx)
    return x


def _run(x, **kw):
    d = {k: (None if v is None else v.cuda()) for k, v in x.items()}
    got = sparse_mqa_paged_fwd(d["q"], d["kv_cache"], d["kv_scales"], d["attn_sink"], d["block_table"],
                               d["seq_lens"], d["token_req"], d["positions"], d["topk_idxs"], **kw)
    torch.cuda.synchronize()
    assert device_status() == 0
    return got


def _want(x, **kw):
    return ref.attn(x["q"], ref.codes(x["kv_cache"]), x["kv_scales"].double(), x["attn_sink"],
                    x["block_table"], x["seq_lens"], x["token_req"], x["positions"], x["topk_idxs"], **kw)


def _check(x, **kw):
    ref.check_attn(_run(x, **kw), _want(x, **kw))


@pytest.mark.parametrize("D", [64, 512])
@pytest.mark.parametrize("H", [1, 16, 33, 64, 65, 128])
def test_attn_heads(H, D):
    """Two requests, several tokens, a list that ends inside a block of slots, masked slots and
    padding rows between and behind the tokens."""
    x = _attn_case([300, 150], [(0, 299), (1, 149), (0, 40), (1, 0)], H, D, 200, 64, H + D, pad=2)
    x["token_req"][1] = -7                                # padding in the middle
    _check(x)
    x["topk_idxs"] = None
    _check(x)


@pytest.mark.parametrize("topk", [1, 31, 127, 128, 129, 256, 1000, 2048])
def test_attn_list_lengths(topk):
    _check(_attn_case([2500], [(0, 2499), (0, 600)], 64, 512, topk, 64, topk))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_attn_dense_lengths(page):
    """Lengths of zero and one, around the blocks of 128 and inside a page; a position behind the
    length, and before the first token."""
    lens = [0, 1, 2, 127, 128, 129, 255, 256, 257, 640, 1100]
    tokens = [(r, n - 1) for r, n in enumerate(lens)] + [(4, 500), (5, -3), (10, 0), (10, 383)]
    for D, H in ((512, 20), (64, 100)):
        _check(_attn_case(lens, tokens, H, D, 0, page, page + D))


@pytest.mark.parametrize("T", [1, 2, 3, 37, 76, 77, 153])
def test_attn_tokens(T):
    """Token counts around the number of CTAs, each token with its own length."""
    lens = [(53 * r) % 701 + 1 for r in range(T)]
    for topk in (0, 300):
        _check(_attn_case(lens, [(r, n - 1) for r, n in enumerate(lens)], 16, 64, topk, 16, T + topk))
    _check(_attn_case([900], [(0, 900 - T + i) for i in range(T)], 65, 512, 400, 128, T))


def test_attn_long_context_is_split():
    _check(_attn_case([20000, 3], [(0, 19999), (1, 2)], 16, 512, 0, 64, 3))
    _check(_attn_case([9000], [(0, 8999)], 128, 64, 8000, 64, 4))


def test_attn_masked_rows_and_duplicates():
    x = _attn_case([200], [(0, 199)] * 6, 48, 512, 150, 32, 11, mask=0)
    x["topk_idxs"][0] = -1                                # nothing left
    x["topk_idxs"][1] = 200                               # behind the length
    x["topk_idxs"][2, :149] = 2 ** 31 - 1                 # one slot left, the last
    x["topk_idxs"][3, 1:] = -1                            # the first
    x["topk_idxs"][4, :100] = 17                          # one position a hundred times
    x["block_table"][0, 2] = -1                           # a page that is not there
    x["block_table"][0, 3] = x["kv_cache"].shape[0]
    _check(x)
    o, lse = _run(x)
    assert torch.all(o[:2] == 0)
    assert torch.allclose(lse[0].cpu(), x["attn_sink"] / 0.6931471805599453, rtol=2 ** -22)


def test_attn_sinks():
    x = _attn_case([300], [(0, 299), (0, 5)], 8, 512, 140, 64, 12)
    x["attn_sink"] = torch.tensor([float("-inf"), -1e4, -30.0, 0.0, 30.0, 1e4, 80.0, -80.0])
    x["topk_idxs"][1] = -1
    _check(x)
    o, lse = _run(x)
    assert float(lse[1, 0]) == float("-inf") and torch.all(o[1] == 0)


@pytest.mark.parametrize("spread", [6, 20])
def test_attn_pages_of_unlike_magnitude(spread):
    """Page scales that differ by many powers of two; the query keeps the logits moderate."""
    x = _attn_case([700], [(0, 699)] * 3, 40, 512, 500, 16, 13 + spread, spread=spread)
    x["q"] = (x["q"].float() * 2.0 ** -spread).bfloat16()
    _check(x)
    x["topk_idxs"] = None
    _check(x)


@pytest.mark.parametrize("power", [-40, -12, 5])
def test_attn_query_magnitudes(power):
    """Peaked and flat weights: rows of q from 2^-40 to 2^5, and unlike rows side by side."""
    x = _attn_case([900], [(0, 899)] * 2, 64, 512, 600, 64, 40 + power)
    x["q"] = (x["q"].float() * 2.0 ** power).bfloat16()
    x["q"][:, ::3] = 0
    x["q"][0, 1, 7] *= 64.0
    _check(x)
    _check(x, sm_scale=0.25)


def test_attn_growing_logits():
    """Each block of slots has larger logits than the one before: the running maximum grows in
    every block, for some heads and not for others."""
    x = _attn_case([1024], [(0, 1023)], 32, 512, 0, 128, 50)
    u = torch.sign(torch.randn(512, generator=torch.Generator().manual_seed(1)))
    rows = (u[None, :] * torch.linspace(0.1, 6.0, 1024)[:, None]).bfloat16()
    val, scale = ref.append(rows, [int(x["block_table"][0, p // 128]) * 128 + p % 128 for p in range(1024)],
                            ref.codes(x["kv_cache"]).nan_to_num(), x["kv_scales"].double(), 128)
    x["kv_cache"], x["kv_scales"] = val.float().to(torch.float8_e4m3fn), scale.float()
    x["q"][0, ::2] = (0.3 * u).bfloat16()
    x["q"][0, 1::4] = (-0.3 * u).bfloat16()
    _check(x)


def test_attn_nan_and_infinite_queries_stay_in_their_head():
    x = _attn_case([300], [(0, 299), (0, 100)], 66, 512, 260, 64, 14)
    q = x["q"].clone()
    q[0, 3, 100], q[0, 40, 0], q[1, 65, 511] = float("nan"), float("inf"), float("-inf")
    want = list(_want(x))
    x["q"] = q
    for t, h in ((0, 3), (0, 40), (1, 65)):
        want[0][t, h] = want[1][t, h] = float("nan")
    ref.check_attn(_run(x), want)


def test_attn_nan_in_a_row_that_is_read():
    """A NaN in a cached row reaches every head's logit, and so all of O of the tokens that read
    the row, and of no other."""
    x = _attn_case([300], [(0, 299), (0, 298)], 64, 512, 260, 64, 15, mask=0)
    x["topk_idxs"][0, :3] = torch.tensor([0, 7, 9])
    x["topk_idxs"][1][x["topk_idxs"][1] == 7] = 8
    raw = x["kv_cache"].view(torch.uint8)
    raw[int(x["block_table"][0, 0]), 7, 5] = 0x7f
    o, lse = _run(x)
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
    assert torch.isfinite(o[1]).all() and torch.isfinite(lse[1]).all()


def test_attn_equals_the_bf16_forward_on_the_same_rows():
    """e4m3 codes times a power of two are exact in bf16, so the contiguous forward on the rows
    the cache stands for computes the same O and LSE, up to both kernels' roundings."""
    x = _attn_case([512], [(0, p) for p in range(480, 512)], 128, 512, 256, 64, 16)
    o, lse = _run(x)
    val = ref.codes(x["kv_cache"]) * x["kv_scales"].double()[:, None, None]
    rows = val[x["block_table"][0, :8].long()].reshape(512, 512).bfloat16()
    o2, lse2 = sparse_mqa_fwd_interface(x["q"][None].cuda(), rows[None].cuda(), x["attn_sink"].cuda(),
                                        x["topk_idxs"][None].cuda())
    assert float((o.float() - o2[0].float()).abs().max()) <= 2e-2 * float(o2.float().abs().max())
    assert float((lse - lse2[0]).abs().max()) <= 1e-4 * float(lse2.abs().max())


@pytest.mark.parametrize("H,D,T,ctx,topk", [(128, 512, 128, 1200, 1024), (128, 512, 9, 6000, 0), (48, 64, 100, 900, 0)])
def test_attn_many_calls_in_a_row(H, D, T, ctx, topk):
    """Back to back, the same call gives the same bits and no wait runs out: every phase of the
    kernel's barriers is told from the one before, however far a group of warps falls behind."""
    x = _attn_case([ctx] * 3, [(t % 3, ctx - 1 - t // 3) for t in range(T)], H, D, topk, 64, 5)
    d = {k: (None if v is None else v.cuda()) for k, v in x.items()}

    def call():
        return sparse_mqa_paged_fwd(d["q"], d["kv_cache"], d["kv_scales"], d["attn_sink"], d["block_table"],
                                    d["seq_lens"], d["token_req"], d["positions"], d["topk_idxs"])
    o, lse = call()
    for _ in range(20):
        for _ in range(200):
            o2, lse2 = call()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert device_status() == 0


def test_attn_out_keeps_padding_and_workspace_is_reused():
    x = _attn_case([300, 200], [(0, 299), (1, 199)], 24, 512, 130, 64, 17, pad=3)
    o = torch.full((5, 24, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 24), 5.0, device="cuda")
    d = {k: v.cuda() for k, v in x.items()}
    shp = _lib.PagedShape(5, 2, 24, 512, 130, 64, d["block_table"].shape[1], d["kv_cache"].shape[0])
    ws = torch.full((max(256, _lib.load().smqa_paged_fwd_workspace_bytes(shp)),), 0xff,
                    dtype=torch.uint8, device="cuda")
    got = _run(x, out=(o, lse), workspace=ws)
    assert got[0] is o and got[1] is lse
    assert torch.all(o[2:] == 7.0) and torch.all(lse[2:] == 5.0)
    fresh = _run(x)
    assert torch.equal(fresh[0][:2], o[:2]) and torch.equal(fresh[1][:2], lse[:2])
    assert torch.all(fresh[0][2:] == 0) and torch.all(fresh[1][2:] == float("-inf"))
    again = _run(x, out=(o, lse), workspace=ws)          # its contents left by the first call
    assert torch.equal(fresh[0][:2], again[0][:2]) and torch.equal(fresh[1][:2], again[1][:2])


def test_offsets_past_32_bits():
    """Pages behind the first 4 GiB of the cache: written and read there, and nowhere else."""
    page, D, n_pages = 128, 512, 70000                   # 4.59e9 bytes
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB of device memory")
    cache = torch.zeros(n_pages, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scale = torch.ones(n_pages, device="cuda")
    table = _i32([[69999, 2, 69000]])
    new = torch.randn(300, D, generator=torch.Generator().manual_seed(3)).bfloat16()
    slot = [int(table[0, p // page]) * page + p % page for p in range(300)]
    paged_kv_append(new.cuda(), _i32(slot), cache, scale)
    pages = torch.tensor([69999, 2, 69000])
    small = cache.view(torch.uint8)[pages.cuda()].cpu().view(torch.float8_e4m3fn)
    q = torch.randn(2, 128, D, generator=torch.Generator().manual_seed(4)).bfloat16()
    sink = torch.zeros(128)
    got = sparse_mqa_paged_fwd(q.cuda(), cache, scale, sink.cuda(), table, _i32([300]), _i32([0, 0]), _i32([299, 250]))
    want = ref.attn(q, ref.codes(small), scale[pages.cuda()].cpu().double(), sink, torch.tensor([[0, 1, 2]]),
                    [300], [0, 0], [299, 250])
    ref.check_attn(got, want)
    wv, ws = ref.append(new, list(range(300)), torch.zeros(3, page, D, dtype=torch.float64),
                        torch.ones(3, dtype=torch.float64), page)
    assert torch.equal(ref.codes(small), wv) and torch.equal(scale[pages.cuda()].cpu().double(), ws)
    assert int(cache.view(torch.uint8)[3:68999].count_nonzero()) == 0


# ------------------------------------------------------------------------------------- together
def _serve(steps, D, H, topk, capture):
    """A small server: prompts of uneven length, then decoded tokens, requests ending and others
    taking their rows; every step's O and LSE against the 64-bit form on the cache as the 64-bit
    append leaves it. With ``capture`` the decode steps replay one CUDA graph."""
    page, W, R, n_pages, N = 16, 20, 4, 40, 200
    cache = torch.zeros(n_pages, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.ones(n_pages, device="cuda")
    val, sc = torch.zeros(n_pages, page, D, dtype=torch.float64), torch.ones(n_pages, dtype=torch.float64)
    free = torch.arange(n_pages, dtype=torch.int32, device="cuda")
    count, table = _i32([n_pages]), torch.full((R, W), -1, dtype=torch.int32, device="cuda")
    ctx, qry = _i32([0] * R), _i32([0] * R)
    release = torch.zeros(R, dtype=torch.bool, device="cuda")
    sink = torch.randn(H, generator=torch.Generator().manual_seed(1)).cuda()
    q = torch.zeros(N, H, D, dtype=torch.bfloat16, device="cuda")
    new = torch.zeros(N, D, dtype=torch.bfloat16, device="cuda")
    idx = torch.full((N, topk), -1, dtype=torch.int32, device="cuda") if topk else None

    def step():
        paged_release(table, release, free, count, n_pages, ctx)
        plan = paged_plan(ctx, qry, table, free, count, page, N, n_pages, inplace=True)
        paged_kv_append(new, plan.slot_mapping, cache, scales)
        out = sparse_mqa_paged_fwd(q, cache, scales, sink, plan.block_table, plan.seq_lens,
                                   plan.token_req, plan.positions, idx)
        ctx.copy_(plan.seq_lens)
        return plan, out

    graph, held = None, None
    g = torch.Generator().manual_seed(2)
    lens = [0] * R
    for n, (gone, adds) in enumerate(steps):
        release.copy_(torch.tensor(gone))
        qry.copy_(torch.tensor(adds, dtype=torch.int32))
        lens = [(0 if d else c) for c, d in zip(lens, gone)]
        before, lens = lens, [c + a for c, a in zip(lens, adds)]
        q.copy_(torch.randn(N, H, D, generator=g).bfloat16())
        new.copy_((torch.randn(N, D, generator=g) * 2.0 ** (n % 3)).bfloat16())
        if topk:
            rows = [torch.randint(0, before[r] + i + 1, (topk,), generator=g) for r in range(R) for i in range(adds[r])]
            idx[:len(rows)] = torch.stack(rows).to(torch.int32).cuda()
        if capture and graph is not None:
            graph.replay()
            plan, out = held
        else:
            plan, out = step()
        torch.cuda.synchronize()
        assert device_status() == 0
        T = sum(adds)
        assert plan.seq_lens.tolist() == lens and int(plan.cu_query[-1]) == T
        val, sc = ref.append(new.cpu(), plan.slot_mapping.tolist(), val, sc, page)
        assert torch.equal(ref.codes(cache), val) and torch.equal(scales.cpu().double(), sc)
        want = ref.attn(q.cpu()[:T], val, sc, sink.cpu(), plan.block_table.cpu(), lens,
                        plan.token_req.tolist(), plan.positions.tolist(), None if idx is None else idx.cpu())
        ref.check_attn((out[0][:T], out[1][:T]), want)
        held_pages = [p for r in range(R) for p in plan.block_table[r].tolist() if p >= 0]
        assert len(held_pages) == len(set(held_pages)) == n_pages - int(count)
        if capture and graph is None:
            saved = [x.clone() for x in (table, count, ctx, free, cache.view(torch.uint8), scales)]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                held = step()
            for x, y in zip((table, count, ctx, free, cache.view(torch.uint8), scales), saved):
                assert torch.equal(x, y)                 # capturing ran nothing


STEPS = [([0, 0, 0, 0], [70, 1, 0, 33]), ([0, 0, 0, 0], [1, 1, 1, 1]), ([0, 0, 0, 0], [1, 1, 20, 1]),
         ([1, 0, 0, 1], [45, 1, 1, 0]), ([0, 1, 0, 0], [1, 0, 1, 160]), ([0, 0, 0, 0], [1, 2, 3, 1])]
STEPS = [([bool(v) for v in gone], adds) for gone, adds in STEPS]


@pytest.mark.parametrize("capture", [False, True])
@pytest.mark.parametrize("D,H,topk", [(512, 64, 40), (64, 16, 0), (512, 128, 0)])
def test_serving_steps(D, H, topk, capture):
    _serve(STEPS, D, H, topk, capture)


def test_no_tokens():
    """Calls without tokens do nothing and return empty rows."""
    cache, scale = ref.fill_cache(3, 16, 64, 1)
    c, sc, z = cache.cuda(), scale.cuda(), _i32([0, 0])
    table, count = _i32([[0, -1], [-1, -1]]), _i32([2])
    plan = paged_plan(_i32([5, 0]), z, table, _i32([1, 2]), count, 16, 0, 3)
    assert plan.block_table.tolist() == table.tolist() and int(plan.free_count) == 2
    assert plan.seq_lens.tolist() == [5, 0] and plan.cu_query.tolist() == [0, 0, 0] and plan.token_req.numel() == 0
    paged_kv_append(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), plan.slot_mapping, c, sc)
    assert torch.equal(c.cpu().view(torch.uint8), cache.view(torch.uint8)) and torch.equal(sc.cpu(), scale)
    for idx in (None, torch.empty(0, 7, dtype=torch.int32, device="cuda")):
        o, lse = sparse_mqa_paged_fwd(torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"), c, sc,
                                      torch.zeros(4, device="cuda"), table, plan.seq_lens, plan.token_req,
                                      plan.positions, idx)
        assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


FIRST_CALLS = """
import torch
from bwd_sparse_mqa_gb300 import paged_kv_append, paged_plan, paged_release, sparse_mqa_paged_fwd
torch.manual_seed(0)
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
ctx, qry, free, count = i32([0, 0]), i32([40, 7]), i32([3, 1, 0, 2, 4]), i32([5])
table = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
cache = torch.zeros(5, 16, 512, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
scales, sink = torch.zeros(5, device="cuda"), torch.randn(128, device="cuda")
q = torch.randn(47, 128, 512, device="cuda").bfloat16()
new = torch.randn(47, 512, device="cuda").bfloat16()
stop = torch.tensor([False, True], device="cuda")

def step():
    p = paged_plan(ctx, qry, table, free, count, 16, 47, 5)
    paged_kv_append(new, p.slot_mapping, cache, scales)
    out = sparse_mqa_paged_fwd(q, cache, scales, sink, p.block_table, p.seq_lens, p.token_req, p.positions)
    paged_release(p.block_table, stop, free, p.free_count, 5)
    return *out, p.block_table, p.free_count

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    held = step()
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in held]
free.copy_(i32([3, 1, 0, 2, 4]))
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert got[0].float().abs().max() > 0 and got[2].tolist() == [[4, 2, 0], [-1, -1, -1]] and int(got[3]) == 2
print("OK")
"""


def test_first_calls_inside_a_capture():
    """A process whose first call of every operator is captured: nothing is set up outside the graph."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("OK"), r.stderr[-3000:]


def test_two_streams_at_once():
    """Two calls in flight on two streams, each with its own workspace, give what they give alone."""
    xs = [_attn_case([3000], [(0, 2999)] * 5, 128, 512, 0, 64, 60 + i) for i in range(2)]
    alone = [_run(x) for x in xs]
    ds = [{k: (None if v is None else v.cuda()) for k, v in x.items()} for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                outs.append(sparse_mqa_paged_fwd(d["q"], d["kv_cache"], d["kv_scales"], d["attn_sink"],
                                                 d["block_table"], d["seq_lens"], d["token_req"], d["positions"]))
        torch.cuda.synchronize()
        for a, b in zip(alone, outs):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attn_writes_stay_in_bounds():
    """Guard bytes around o, lse and the workspace stay as they were."""
    from tests.test_gpu_guards import Guarded
    x = _attn_case([2000, 77], [(0, 1999), (1, 76), (0, 3)], 37, 512, 0, 64, 70, pad=2)
    d = {k: (None if v is None else v.cuda()) for k, v in x.items()}
    T, H, D = d["q"].shape
    shp = _lib.PagedShape(T, 2, H, D, 0, 64, d["block_table"].shape[1], d["kv_cache"].shape[0])
    lib = _lib.load()
    o, lse = Guarded(T * H * D * 2), Guarded(T * H * 4)
    ws = Guarded(max(256, lib.smqa_paged_fwd_workspace_bytes(shp)))
    sp = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.smqa_paged_fwd(*[d[k].data_ptr() for k in ("q", "kv_cache", "kv_scales", "attn_sink", "block_table",
                                                          "seq_lens", "token_req", "positions")],
                              None, shp, 0.0, o.ptr(), lse.ptr(), ws.ptr(), ws.n, 0, sp) == 0
    torch.cuda.synchronize()
    assert device_status() == 0
    assert o.intact() and lse.intact() and ws.intact()
    ref.check_attn((o.view(torch.bfloat16, (T, H, D))[:3], lse.view(torch.float32, (T, H))[:3]),
                   [w[:3] for w in _want(x)])


@pytest.mark.parametrize("D,topk,cta", [(512, 300, 0), (512, 0, 3), (64, 0, 1), (512, 2048, 79)])
def test_attn_bounded_wait_runs_out(D, topk, cta):
    """One CTA is stopped after its first MMA: the call ends with the timeout status, by the wait
    limit, and the next one computes as before."""
    from bwd_sparse_mqa_gb300 import set_wait_limit_ns
    x = _attn_case([3000], [(0, 2999 - i) for i in range(40)], 100, D, topk, 64, 80)
    want = _run(x)
    lib = _lib.load()
    before = set_wait_limit_ns(20_000_000)
    lib.smqa_debug_stall(cta)
    try:
        d = {k: (None if v is None else v.cuda()) for k, v in x.items()}
        args = [d[k] for k in ("q", "kv_cache", "kv_scales", "attn_sink", "block_table", "seq_lens", "token_req", "positions")]
        with pytest.raises(_lib.SMQAError) as err:
            sparse_mqa_paged_fwd(*args, d["topk_idxs"], check_status=True)
        assert err.value.status == _lib.SMQA_ERR_DEVICE_TIMEOUT
    finally:
        lib.smqa_debug_stall(-1)
        set_wait_limit_ns(0)
    assert before > 0 and device_status(clear=True) == _lib.SMQA_ERR_DEVICE_TIMEOUT
    got = _run(x)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
