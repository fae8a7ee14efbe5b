"""The two stores into NVFP4 planes (needs a GPU) given values that are not finite."""
import pytest
import torch

import _nvfp4
import sparse_attention_indexer_packed_gb300 as idx

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def both(src):
    """Bytes of idx_store_nvfp4 and of idx_store_kv_nvfp4 with an outer scale of 1."""
    T = len(src)
    slots = torch.arange(T, device="cuda")
    planes = [[torch.full((-(-T // 64) * 64, n), 0xee, dtype=torch.uint8, device="cuda") for n in (64, 8)]
              for _ in range(2)]
    idx.idx_store_nvfp4(src.cuda(), slots, tuple(planes[0]))
    idx.idx_store_kv_nvfp4(src.cuda()[:, None], None, slots, *planes[1], None, None, 1)
    return [[t[:T].cpu() for t in p] for p in planes]


def rows():
    g = torch.Generator().manual_seed(3)
    x = torch.randn((70, 128), generator=g)
    x[3:] *= torch.exp2(torch.randint(-20, 100, (67, 1), generator=g).float())
    return x.to(torch.bfloat16)


def test_infinities_are_held_as_the_largest_value_of_their_sign():
    src = rows()
    src[0, 3], src[1, 20], src[2, :16], src[3, 127] = INF, -INF, -INF, INF
    src[4, 32], src[4, 40], src[5, 1::2] = INF, -INF, -INF
    codes, scale = _nvfp4.quantize(src)      # the oracle's bytes
    for payload, s in both(src):
        assert torch.equal(s, scale)
        assert torch.equal(payload, codes)


def test_a_nan_in_the_index_pool_and_in_the_cache():
    src = rows()[:8]
    clean = src.clone()
    src[0, 5], src[1, 16:32] = NAN, NAN
    src[2, 0], src[2, 1] = NAN, -INF
    clean[0, 5], clean[2, 0], clean[2, 1] = 0, 0, -INF
    (p, s), (pc, sc) = both(src)
    codes, scale = _nvfp4.quantize(clean)
    # the index pool: left out of the maximum, the code of 6; a group of nothing else NaN
    codes[0, 2] = (codes[0, 2] & 0x0f) | 0x70
    codes[2, 0] = (codes[2, 0] & 0xf0) | 0x07
    codes[1, 8:16], scale[1, 1] = 0x77, 0x7f
    assert torch.equal(s, scale) and torch.equal(p, codes)
    # the cache: the group's scale is NaN
    for row, group in ((0, 0), (1, 1), (2, 0)):
        codes[row, group * 8:group * 8 + 8], scale[row, group] = 0, 0x7f
    assert torch.equal(sc, scale) and torch.equal(pc, codes)
