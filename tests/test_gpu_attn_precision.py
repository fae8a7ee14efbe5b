"""How exact the attention is (needs a GPU): bounds that follow from the stated roundings, and
caches and queries of far apart magnitudes, where a unit that is held in few bits shows."""
import pytest
import torch

import _attn
import _attn_bounds
import sparse_attention_indexer_packed_gb300 as idx
from test_gpu_attn import draws, drafts, lists_for, run

pytestmark = pytest.mark.gpu
DTYPES = ["bf16", "fp8_e4m3"]
SM = 128 ** -0.5
WIDE = [False, True]          # 4 draft rows of 4 heads, or of 16: the tcgen05 kernel


def heads(wide):
    return 16 if wide else 4


def rows_of(c, r, n):
    return _attn.token_rows(c.page_table[int(c.slot_ids[r])].tolist(), n, 0, c.kv_heads)


def set_keys(c, rows, keys):
    """Key rows of an e4m3 cache, quantized as the store does."""
    c.k[0][rows], c.k[1][rows] = _attn.quantize(keys)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("blocks", [False, True])
def test_no_less_exact_than_stated(dtype, wide, blocks):
    Hq = heads(wide)
    lens = [drafts(L, 4) for L in (700, 65, 33, 1500)]
    c = _attn.make(dtype, lens, 1, 201)
    q = draws(4, 4, Hq, 202)
    ids = lists_for(lens, 1, 5, 203, 4) if blocks else None
    out, l, flags = run(c, q, block_ids=ids, lists=1 if blocks else 0)
    assert flags == 0
    ref = _attn_bounds.reference(c, q, SM, ids, 1, split_query=wide and dtype != "bf16")
    _attn_bounds.check(out, l, ref, rows=torch.isfinite(ref[1]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", WIDE)
def test_few_tokens_of_like_weights(dtype, wide):
    """Where the weights' own rounding does not average out: bf16 weights of one term instead of
    two would be past the bound several times over (test_attn_bounds_cpu.py)."""
    lens = [drafts(L, 4) for L in range(5, 29)]
    c = _attn.make(dtype, lens, 1, 218)
    q = draws(len(lens), 4, heads(wide), 219, scale=0.3)
    out, l, flags = run(c, q)
    assert flags == 0
    _attn_bounds.check(out, l, _attn_bounds.reference(c, q, SM, split_query=wide and dtype != "bf16"))


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("ctas", [1, 0])
def test_zero_values_before_large_ones_stay_in_the_sum(wide, ctas):
    """Tokens of value zero weigh as much as the others, whatever the others' values are."""
    lens = [drafts(L, 4) for L in (1100, 90)]
    q = draws(2, 4, heads(wide), 204)
    c = _attn.make("fp8_e4m3", lens, 1, 205)
    for r, n, zeros in ((0, 1100, 560), (1, 90, 64)):
        at = rows_of(c, r, n)
        c.v[0][at[:zeros]] = 0
        c.v[1][at[:zeros]] = 2.0 ** -96 / 448
        c.v[1][at[zeros:]] = 6e10 / 448
    idx.idx_set_grid_limit(ctas)
    try:
        out, l, flags = run(c, q)
        c2 = _attn.make("fp8_e4m3", lens, 1, 205)
        _, l2, _ = run(c2, q)
    finally:
        idx.idx_set_grid_limit(0)
    assert flags == 0
    assert torch.equal(l, l2)           # the values have no part in the weights' sum
    _attn_bounds.check(out, l, _attn_bounds.reference(c, q, SM, split_query=wide))


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("below", [40, 60])
@pytest.mark.parametrize("factor", [2.0 ** 20, 2.0 ** 26, 2.0 ** 37])
def test_a_large_value_of_little_weight(wide, blocks, below, factor):
    """A visible token whose values are far above the others' but whose weight is 2^-below."""
    lens = [drafts(L, 4) for L in (40, 300, 257, 610)]
    c = _attn.make("fp8_e4m3", lens, 1, 206)
    q = draws(4, 4, heads(wide), 207)
    q[..., 0] = 8.0
    for r, at in ((0, 0), (1, 150), (2, 253), (3, 300)):       # first, middle, last token that all see
        rows = rows_of(c, r, max(lens[r]))
        k = _attn.values64(c.k, rows).float()
        k[:, 0] = 0
        k[at] = 0
        k[at, 0] = -below * 0.6931472 / (8 * SM)
        set_keys(c, rows, k)
        c.v[1][rows[at]] *= factor
    ids = torch.arange(5, dtype=torch.int32).expand(4, 4, 5).contiguous() if blocks else None
    out, l, flags = run(c, q, block_ids=ids, lists=1 if blocks else 0)
    assert flags == 0
    _attn_bounds.check(out, l, _attn_bounds.reference(c, q, SM, ids, 1, split_query=wide))


@pytest.mark.parametrize("wide", WIDE)
def test_a_value_past_the_reach_of_the_others_unit(wide):
    """Values of 2^-60 and one token's of 2^75 with a weight of 2^-160: no unit holds both."""
    lens = [drafts(L, 4) for L in (40, 300)]
    c = _attn.make("fp8_e4m3", lens, 1, 222)
    q = draws(2, 4, heads(wide), 223)
    q[..., 0] = 8.0
    c.v[1].mul_(2.0 ** -60)
    for r, at in ((0, 17), (1, 200)):
        rows = rows_of(c, r, max(lens[r]))
        k = _attn.values64(c.k, rows).float()
        k[:, 0] = 0
        k[at] = 0
        k[at, 0] = -160 * 0.6931472 / (8 * SM)
        set_keys(c, rows, k)
        c.v[1][rows[at]] *= 2.0 ** 68
        c.v[1][rows[at]] *= 2.0 ** 67      # (2^135 is no fp32)
    out, l, flags = run(c, q)
    assert flags == 0
    _attn_bounds.check(out, l, _attn_bounds.reference(c, q, SM, split_query=wide))


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("up", [True, False])
def test_scores_and_value_scales_that_run_against_each_other(wide, up):
    """The maximum rises by 2^7 log2 units (or falls) along the cache while the values shrink (or
    grow) by as much: every token counts the same, none of them in another's unit."""
    n = 900
    lens = [drafts(n, 4)]
    c = _attn.make("fp8_e4m3", lens, 1, 208)
    q = draws(1, 4, heads(wide), 209)
    q[..., 0] = 16.0
    rows = rows_of(c, 0, n)
    ramp = torch.linspace(-64, 64, n) * (1 if up else -1)          # log2 units
    k = _attn.values64(c.k, rows).float() * 0.25
    k[:, 0] = ramp * 0.6931472 / (16 * SM)
    set_keys(c, rows, k)
    c.v[1][rows] = c.v[1][rows] * torch.exp2(-ramp)[:, None]
    out, l, flags = run(c, q)
    assert flags == 0
    _attn_bounds.check(out, l, _attn_bounds.reference(c, q, SM, split_query=wide))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", WIDE)
def test_a_query_with_an_outlier_channel(dtype, wide):
    """One channel 2^12 above the others, which no key goes by: the scores are the others'."""
    lens = [drafts(300, 4), drafts(70, 4)]
    c = _attn.make(dtype, lens, 1, 210)
    g = torch.Generator().manual_seed(211)
    q = (1 + torch.rand((2, 4, heads(wide), 128), generator=g)) * (
        2.0 * torch.randint(0, 2, (2, 4, heads(wide), 128), generator=g) - 1)
    q[..., 5] = 4096.0
    q = q.to(torch.bfloat16)
    if dtype == "bf16":
        c.k[0][:, 5] = 0
    else:
        c.k[0][:, 5] &= 0x80        # a zero
    for r in range(2):              # (what no row sees is NaN again)
        assert torch.isfinite(_attn.values64(c.k, rows_of(c, r, max(lens[r])))).all()
    out, l, flags = run(c, q)
    assert flags == 0
    _attn_bounds.check(out, l, _attn_bounds.reference(c, q, SM, split_query=wide and dtype != "bf16"))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_query_that_is_not_finite(dtype, wide, bad):
    """Its row is NaN (keys of either sign meet it); the others do not notice."""
    lens = [drafts(200, 4)]
    c = _attn.make(dtype, lens, 1, 212)
    q = draws(1, 4, heads(wide), 213)
    ref = _attn_bounds.reference(c, q, SM, split_query=wide and dtype != "bf16")
    q[0, 1, 3, 7] = bad
    out, l, flags = run(c, q)
    assert flags == 0
    rows = torch.ones((1, 4, heads(wide)), dtype=torch.bool)
    rows[0, 1, 3] = False
    _attn_bounds.check(out, l, ref, rows=rows)
    assert torch.isnan(out[0, 1, 3].float()).all() and torch.isnan(l[0, 1, 3])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", WIDE)
def test_queries_near_the_largest_number(dtype, wide):
    """Queries of 2^118 on keys of 2^-118: ordinary scores."""
    lens = [drafts(150, 4)]
    c = _attn.make(dtype, lens, 1, 214)
    q = draws(1, 4, heads(wide), 215)
    clean = _attn_bounds.reference(c, q, SM, split_query=wide and dtype != "bf16")
    if dtype == "bf16":
        c.k[0].mul_(2.0 ** -118)
    else:
        c.k[1].mul_(2.0 ** -118)
    out, l, flags = run(c, q * 2.0 ** 118)
    assert flags == 0
    _attn_bounds.check(out, l, clean)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", WIDE)
def test_scores_that_are_next_to_nothing(dtype, wide):
    """Queries of 2^-110 under a scale of 1e-20: every visible token counts the same."""
    lens = [drafts(150, 4), drafts(20, 4)]
    c = _attn.make(dtype, lens, 1, 220)
    q = draws(2, 4, heads(wide), 221) * 2.0 ** -110
    out, l, flags = run(c, q, sm_scale=1e-20)
    assert flags == 0
    _attn_bounds.check(out, l, _attn_bounds.reference(c, q, 1e-20))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_token_that_the_last_of_many_draft_rows_sees(dtype, bad):
    """70 draft rows in one unit, the newest token not finite: the rows past the 32nd are
    recomputed token by token and come out as if it were not there."""
    P, n = 70, 150
    c = _attn.make(dtype, [drafts(n, P)], 1, 216)
    q = draws(1, P, 1, 217)
    ref = _attn_bounds.reference(c, q, SM, split_query=dtype != "bf16")
    last = rows_of(c, 0, n)[-1]
    (c.v[0] if dtype == "bf16" else c.v[1])[last] = bad
    out, l, flags = run(c, q)
    assert flags == 0
    rows = torch.ones((1, P, 1), dtype=torch.bool)
    rows[0, P - 1] = False
    _attn_bounds.check(out, l, ref, rows=rows)
    assert not torch.isfinite(out[0, P - 1].float()).all()
