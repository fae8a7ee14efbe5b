"""Stores into NVFP4 planes (needs a GPU) at the sizes where a thread takes one row or four."""
import pytest
import torch

import _nvfp4
import sparse_attention_indexer_packed_gb300 as idx
from test_gpu_nvfp4 import tokens

pytestmark = pytest.mark.gpu


# rows = tokens * heads * planes; four a thread from 49,152 on, 128 tokens a CTA
@pytest.mark.parametrize("T,H,values", [(12287, 2, True), (12288, 2, True), (6200, 4, True), (12345, 3, True),
                                        (49151, 1, False), (49153, 1, False), (5000, 5, True)])
@pytest.mark.parametrize("outers", [(1.0, 1.0), (0.125, 32.0)])
def test_rows_a_thread(T, H, values, outers):
    pages = T // 64 + 4
    src = tokens(T, H, T + H)
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(pages * 64, generator=g)[:T]
    slots[5], slots[9], slots[11], slots[T - 2] = -1, pages * 64, -2 ** 62, 2 ** 62
    pools = [_nvfp4.plane(pages * H * 64, 5 + i) for i in range(2)]
    dev = [tuple(t.cuda() for t in p) for p in pools]
    d = src.cuda()
    k, v = d[:, H:2 * H], d[:, 2 * H:] if values else None
    idx.idx_store_kv_nvfp4(k, v, slots.cuda(), *dev[0], *(dev[1] if values else (None, None)), H, *outers)
    ok = (slots >= 0) & (slots < pages * 64)
    for i in range(2):
        payload, scale = (t.clone() for t in pools[i])
        if i == 0 or values:
            codes, s = _nvfp4.quantize(src[:, (1 + i) * H:(2 + i) * H], outers[i])
            for h in range(H):
                rows = (slots[ok] // 64 * H + h) * 64 + slots[ok] % 64
                payload[rows], scale[rows] = codes[ok, h], s[ok, h]
        assert torch.equal(dev[i][0].cpu(), payload)
        assert torch.equal(dev[i][1].cpu(), scale)
