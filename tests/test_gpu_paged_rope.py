"""The paged write with the position rotation applied on the way, and rows of 128.

The kernel rounds each product and sum of the rotation to fp32, as torch's fp32 operations on
the CPU do, and then writes codes and scales as the plain append: those are compared bit by bit.
Against the rotation in 64 bits a stored value is off by half a step of its e4m3 code at most,
which the fp32 rotation can move by 2^-23 (|x cos| + |y sin|): three roundings of 2^-24 each, the
products' and the sum's."""
import math

import pytest
import torch

from bwd_sparse_mqa_gb300 import _lib, paged_kv_append, paged_plan
from tests import _paged as ref

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(n, dim, base=10000.0):
    ang = torch.arange(n, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    return torch.cat([torch.cos(ang), torch.sin(ang)], 1).float()


def _rotate(x, pos, cs, offset, interleaved):
    """In x's type; NaN for positions outside the table."""
    dim = cs.shape[1]
    half = dim // 2
    ok = (pos >= 0) & (pos < cs.shape[0])
    row = cs.to(x.dtype)[torch.where(ok, pos, 0)] if cs.shape[0] else torch.zeros(len(pos), dim, dtype=x.dtype)
    row = torch.where(ok[:, None], row, math.nan)
    c, s = row[:, :half], row[:, half:]
    part = x[:, offset:offset + dim]
    a, b = (part[:, 0::2], part[:, 1::2]) if interleaved else (part[:, :half], part[:, half:])
    u, v = a * c - b * s, b * c + a * s
    out = x.clone()
    out[:, offset:offset + dim] = torch.stack([u, v], 2).flatten(1) if interleaved else torch.cat([u, v], 1)
    return out


def _check(new, slot, pos, cache, scale, cs, offset, interleaved):
    page = cache.shape[1]
    x = _rotate(new.float(), torch.tensor(pos), cs, offset, interleaved)
    want, want_s = ref.append(x, slot, ref.codes(cache), scale.double(), page)
    c, s = cache.cuda(), scale.cuda()
    back = paged_kv_append(new.cuda(), _i32(slot), c, s, positions=_i32(pos), cos_sin=cs.cuda(),
                           rope_offset=offset, interleaved=interleaved)
    assert back[0] is c and back[1] is s
    assert torch.equal(s.cpu().double(), want_s)
    got = ref.codes(c)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    return c, s


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("D,dim,offset", [(512, 64, 448), (128, 64, 0), (128, 128, 0), (64, 16, 8), (64, 48, 16),
                                          (512, 512, 0), (512, 80, 200)])
@pytest.mark.parametrize("page", [16, 64])
def test_rotated_prompts_and_tokens(D, dim, offset, interleaved, page):
    """Prompts over several pages, single tokens and skipped rows; positions far and near."""
    g = torch.Generator().manual_seed(D + dim + page)
    cache, scale = ref.fill_cache(14, page, D, 3, spread=2)
    slot = list(range(3 * page + 5, 6 * page + 2)) + [-1, 9 * page, 7 * page + page - 1, 14 * page, 0, 1, 2]
    slot += list(range(10 * page + 1, 10 * page + 12))
    T = len(slot)
    new = (torch.randn(T, D, generator=g) * 2.0 ** torch.randint(-3, 4, (T, 1), generator=g)).bfloat16()
    pos = torch.randint(0, 5000, (T,), generator=g).tolist()
    pos[0], pos[1] = 0, 4999
    _check(new, slot, pos, cache, scale, _table(5000, dim), offset, interleaved)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation_in_64_bits(interleaved):
    """Each stored value within half a code's step of the exact rotation."""
    T, D, dim, page = 64, 128, 64, 64
    new = torch.randn(T, D, generator=torch.Generator().manual_seed(1)).bfloat16()
    pos = list(range(100000, 100000 + T))
    cs = _table(100064, dim)
    cache = torch.zeros(1, page, D, dtype=torch.uint8).view(torch.float8_e4m3fn)
    c, s = _check(new, list(range(T)), pos, cache, torch.ones(1), cs, 0, interleaved)
    x = new.double()
    want = _rotate(x, torch.tensor(pos), cs, 0, interleaved) / float(s)
    got = ref.codes(c)[0]
    half = dim // 2
    part = x[:, :dim]
    a, b = (part[:, 0::2], part[:, 1::2]) if interleaved else (part[:, :half], part[:, half:])
    size = a.abs() + b.abs()
    size = torch.stack([size, size], 2).flatten(1) if interleaved else torch.cat([size, size], 1)
    slack = torch.zeros_like(x)
    slack[:, :dim] = 2.0 ** -23 * size / float(s)
    # Half a step: 2^-4 of the value, or 2^-10 among the subnormals.
    bound = torch.maximum(2.0 ** -4 * (want.abs() + slack), torch.tensor(2.0 ** -10, dtype=torch.float64)) + slack
    assert bool(((got - want).abs() <= bound).all())


def test_positions_outside_the_table_and_bad_values():
    """A position outside the table, infinities and NaN give NaN codes in their pairs only, and
    do not enter the scale; skipped rows' positions are never looked up."""
    D, page = 64, 16
    g = torch.Generator().manual_seed(7)
    cache, scale = ref.fill_cache(4, page, D, 3)
    new = torch.randn(12, D, generator=g).bfloat16()
    new[3, 20], new[4, 60], new[5, 5] = math.inf, math.nan, -math.inf
    pos = [0, 99, 100, 5, 6, 7, -1, 2 ** 31 - 1, 8, -2 ** 31, 50, 51]
    slot = list(range(10)) + [-1, -5]
    for interleaved in (True, False):
        c, s = _check(new, slot, pos, cache, scale, _table(100, 32), 32, interleaved)
        nan = torch.isnan(ref.codes(c)[0])
        assert nan[[2, 6, 7, 9], 32:].all() and not nan[[2, 6, 7, 9], :32].any() and not nan[:2].any()
    _check(new[:3], [0, 1, 2], [0, 0, 0], cache, scale, _table(0, 32), 32, True)   # an empty table


@pytest.mark.parametrize("D", [128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_rows_of_128(D, page):
    """Index keys without rotation: growing scales, short and long runs."""
    g = torch.Generator().manual_seed(page)
    cache, scale = ref.fill_cache(12, page, D, 5, spread=2)
    slot, rows = [], []
    for pg, (off, n) in enumerate([(0, page), (1, page - 1), (page - 1, 1), (3, 8), (3, 9), (0, 1), (5, 2)]):
        slot += list(range(pg * page + off, pg * page + off + n))
        rows.append(torch.randn(n, D, generator=g) * 2.0 ** (pg - 2))
    new = torch.cat(rows).bfloat16()
    want, want_s = ref.append(new, slot, ref.codes(cache), scale.double(), page)
    c, s = cache.cuda(), scale.cuda()
    paged_kv_append(new.cuda(), _i32(slot), c, s)
    assert torch.equal(s.cpu().double(), want_s) and torch.equal(ref.codes(c), want)


def test_one_by_one_equals_at_once_and_a_captured_call():
    """Rows written one call each (scales growing on the way) end within one e4m3 rounding of the
    rows written at once; a captured call replays on new rows."""
    D, page, T = 512, 64, 64
    g = torch.Generator().manual_seed(2)
    new = torch.randn(T, D, generator=g).bfloat16().cuda()
    pos, cs = _i32(list(range(T))), _table(T, 64).cuda()
    zero = lambda: torch.zeros(1, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # noqa: E731
    a, sa, b, sb = zero(), torch.ones(1, device="cuda"), zero(), torch.ones(1, device="cuda")
    paged_kv_append(new, pos, a, sa, positions=pos, cos_sin=cs, interleaved=True)
    for t in range(T):
        paged_kv_append(new[t:t + 1], pos[t:t + 1], b, sb, positions=pos[t:t + 1], cos_sin=cs, interleaved=True)
    assert torch.equal(sa, sb)
    # (Codes that became subnormal when the scale grew were rounded twice: 2^-10 of the scale more.)
    assert float((ref.codes(a) - ref.codes(b)).abs().max()) <= 2.0 ** -9
    c, sc = zero(), torch.ones(1, device="cuda")
    rows = new.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        paged_kv_append(rows, pos, c, sc, positions=pos, cos_sin=cs, interleaved=True)
    rows.copy_(new.flip(0))
    graph.replay()
    d, sd = zero(), torch.ones(1, device="cuda")
    paged_kv_append(new.flip(0).contiguous(), pos, d, sd, positions=pos, cos_sin=cs, interleaved=True)
    assert torch.equal(c.view(torch.uint8), d.view(torch.uint8)) and torch.equal(sc, sd)


def test_refusals_of_the_rotation():
    D = 64
    cache = torch.zeros(2, 16, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s, new, slot = torch.ones(2, device="cuda"), torch.zeros(3, D, dtype=torch.bfloat16, device="cuda"), _i32([0, 1, 2])
    cs = _table(8, 32).cuda()
    call = lambda **k: paged_kv_append(new, slot, cache, s, **{**dict(positions=slot, cos_sin=cs), **k})  # noqa: E731
    call()
    for bad in ({"positions": slot[:2]}, {"cos_sin": cs.t()}, {"cos_sin": cs[:, :0]}, {"cos_sin": None},
                {"positions": slot.cpu()}, {"rope_offset": -1}, {"cos_sin": None, "positions": None, "rope_offset": 8}):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in ({"positions": None}, {"cos_sin": cs.double()}, {"positions": slot.long()}):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in ({"cos_sin": cs[:, :24].contiguous()}, {"rope_offset": 4}, {"rope_offset": 40},
                {"cos_sin": _table(8, 80).cuda()}):
        with pytest.raises((ValueError, _lib.SMQAError)):
            call(**bad)
    paged_kv_append(new[:0], slot[:0], cache, s, positions=slot[:0], cos_sin=cs)


def test_plan_then_rotated_append():
    """The slots and positions of a plan, padding rows included, straight into the write."""
    page, n_pages, D = 16, 12, 128
    table, free = ref.deal([20, 0], page, 4, n_pages, 1)
    plan = paged_plan(_i32([20, 0]), _i32([3, 18]), table.cuda(), free.cuda(), _i32([free.numel()]), page, 24, n_pages)
    cache, scale = ref.fill_cache(n_pages, page, D, 3)
    new = torch.randn(24, D, generator=torch.Generator().manual_seed(3)).bfloat16()
    c, s = cache.cuda(), scale.cuda()
    cs = _table(64, 64)
    paged_kv_append(new.cuda(), plan.slot_mapping, c, s, positions=plan.positions, cos_sin=cs.cuda(), rope_offset=0)
    x = _rotate(new.float(), plan.positions.cpu().long(), cs, 0, False)
    want, want_s = ref.append(x, plan.slot_mapping.tolist(), ref.codes(cache), scale.double(), page)
    assert torch.equal(s.cpu().double(), want_s) and torch.equal(ref.codes(c), want)
