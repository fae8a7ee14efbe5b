"""The attention's stated roundings, and that the GPU tests' bounds would see coarser ones (CPU)."""
import pytest
import torch

import _attn
import _attn_bounds

SM = 128 ** -0.5


def test_a_query_is_an_e4m3_and_an_e5m2_term():
    """The tcgen05 kernel's split of a query element, over every bf16 magnitude of a row whose
    largest is in [2^7, 2^8): exact within 2^13 of it, off by 2^-21 of it at most."""
    x = torch.arange(1, 1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double()
    x = x[x < 256]                      # (NaN and infinity are not)
    hi = x.float().to(torch.float8_e4m3fn).double()
    lo = (x - hi).float().to(torch.float8_e5m2).double()
    off = (x - hi - lo).abs()
    assert (off[x >= 2.0 ** -6] == 0).all()
    assert (off <= 2.0 ** -14).all()


def one_row(seed, dtype, n=6):
    """A query row, its few keys and values, and the exact result with its bound."""
    c = _attn.make(dtype, [[n]], 1, seed)
    g = torch.Generator().manual_seed(seed)
    q = (0.3 * torch.randn(128, generator=g)).to(torch.bfloat16).double()
    at = _attn.token_rows(c.page_table[int(c.slot_ids[0])].tolist(), n, 0, 1)
    k, v = _attn.values64(c.k, at), _attn.values64(c.v, at)
    scale = None if dtype == "bf16" else c.v[1][at].double()
    s = k @ q * SM
    z = torch.logsumexp(s, 0)
    w = torch.exp(s - z)
    return w, v, scale, w @ v, _attn_bounds.bounds(q, k, v, scale, w, z, SM)[0]


def to(x, dtype):
    return x.float().to(dtype).double()


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_bounds_of_a_bf16_cache_see_a_dropped_weight_term(seed):
    w, v, _, want, tol = one_row(seed, "bf16")
    p = w / w.max()
    hi = to(p, torch.bfloat16)
    two = hi + to(p - hi, torch.bfloat16)
    assert ((to(two @ v * w.max(), torch.bfloat16) - want).abs() <= tol).all()
    assert ((to(hi @ v * w.max(), torch.bfloat16) - want).abs() > tol).any()


@pytest.mark.parametrize("seed", [4, 5, 6])
def test_bounds_of_an_e4m3_cache_see_a_unit_set_by_a_scale_alone(seed):
    """One token of 2^30 times larger values and a weight of 2^-50 (the unit its scale would set)."""
    w, v, scale, want, _ = one_row(seed, "fp8_e4m3")
    w, v, scale = w.clone(), v.clone(), scale.flatten().clone()
    w[3] = w.max() * 2.0 ** -50
    v[3] *= 2.0 ** 30
    scale[3] *= 2.0 ** 30
    want = w @ v
    r = w * scale
    codes = v / scale[:, None]
    tol = _attn_bounds.bounds(torch.zeros(128, dtype=torch.float64), torch.zeros_like(v), v,
                              scale, w, torch.zeros(()), SM)[0]
    good = r.max() / 8
    coarse = scale.max()
    assert ((to(r / good, torch.float16) @ codes * good - want).abs() <= tol).all()
    assert ((to(r / coarse, torch.float16) @ codes * coarse - want).abs() > tol).any()
