"""idx_store_kv and idx_add_rmsnorm_fp8 (needs a GPU): stored bytes bit for bit against the
rule in plain fp32, the norm against 64 bits."""
import pytest
import torch

import _attn
import sparse_attention_indexer_packed_gb300 as idx

pytestmark = pytest.mark.gpu


def tokens(T, H, seed, wide=3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, wide * H, 128), generator=g)
    x *= torch.exp2(torch.randint(-20, 20, (T, 1, 1), generator=g).float())
    return x.to(torch.bfloat16)


def expected(src, slots, pool, H, pages):
    payload, scale = (None if t is None else t.clone() for t in pool)
    for i, s in enumerate(slots.tolist()):
        if not 0 <= s < pages * 64:
            continue
        for h in range(H):
            row = (s // 64 * H + h) * 64 + s % 64
            if scale is None:
                payload[row] = src[i, h]
            else:
                codes, sc = _attn.quantize(src[i, h].float()[None])
                payload[row], scale[row] = codes[0], sc[0]
    return payload, scale


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("T,H,values", [(1, 1, False), (1, 2, True), (63, 1, True), (64, 3, True),
                                        (257, 4, True), (1000, 1, False)])
def test_store(dtype, T, H, values):
    pages = T // 64 + 4
    src = tokens(T, H, 3 + T)
    src[0, 0] = 0
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(pages * 64, generator=g)[:T]
    if T > 60:
        slots[5], slots[9], slots[11] = -1, pages * 64, -2 ** 62
    pools = [_attn.plane(pages * H * 64, dtype, 5 + i) for i in range(2)]
    dev = [tuple(None if t is None else t.cuda() for t in p) for p in pools]
    d = src.cuda()
    k, v = d[:, H:2 * H], d[:, 2 * H:] if values else None
    idx.idx_store_kv(k, v, slots.cuda(), *dev[0], *(dev[1] if values else (None, None)), dtype, H)
    torch.cuda.synchronize()
    for i in range(2):
        s = src[:, (1 + i) * H:(2 + i) * H]
        want = expected(s, slots, pools[i], H, pages) if i == 0 or values else pools[i]
        for got, ref in zip(dev[i], want):
            if ref is not None:
                assert torch.equal(got.cpu().view(torch.uint8), ref.view(torch.uint8))


def test_store_of_values_that_are_not_finite():
    src = tokens(4, 1, 9, wide=1)
    src[1, 0, 7] = float("nan")
    src[2, 0, 7] = float("inf")
    src[3] = 1e-38          # below the smallest amax a scale is made from
    pool = _attn.plane(64, "fp8_e4m3", 5)
    dev = tuple(t.cuda() for t in pool)
    idx.idx_store_kv(src.cuda(), None, torch.arange(4).cuda(), *dev, None, None, "fp8_e4m3", 1)
    codes = dev[0].cpu().view(torch.float8_e4m3fn).float()
    scale = dev[1].cpu()
    assert torch.isnan(scale[1]) and torch.isnan(codes[1]).all()
    assert torch.isinf(scale[2]) and torch.isnan(codes[2, 7]) and (codes[2, :7] == 0).all()
    assert scale[3] == 2.0 ** -96 / 448 and (codes[3].abs() <= 1).all()
    want = _attn.quantize(src[0].float())
    assert torch.equal(dev[0][:1].cpu(), want[0]) and torch.equal(scale[:1], want[1])


def test_store_past_32_bit_offsets():
    pages, H = 150_000, 2
    k = torch.empty((pages * H * 64, 128), dtype=torch.bfloat16, device="cuda")
    src = tokens(3, H, 10, wide=1)
    slots = torch.tensor([pages * 64 - 1, 5, pages * 64 - 64], dtype=torch.int64)
    idx.idx_store_kv(src.cuda(), None, slots.cuda(), k, None, None, None, "bf16", H)
    for i, s in enumerate(slots.tolist()):
        for h in range(H):
            assert torch.equal(k[(s // 64 * H + h) * 64 + s % 64].cpu(), src[i, h])


def norm_reference(x, res, w, eps, group):
    h = x.double() + (0 if res is None else res.double())
    n = x.shape[1]
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w.double()
    g = group or n
    groups = [y[:, a:a + g] for a in range(0, n, g)]
    scale = torch.stack([t.abs().amax(1).clamp_min(2.0 ** -96) / 448 for t in groups], 1)
    return h, y, scale


def run_norm(x, res, w, eps, group, out_residual=True):
    T, n = x.shape
    out = torch.empty((T, n), dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty((T, -(-n // group) if group else 1), device="cuda")
    new = torch.empty((T, n), dtype=torch.bfloat16, device="cuda") if out_residual else None
    idx.idx_add_rmsnorm_fp8(x, res, w, eps, group, out, sc, new)
    torch.cuda.synchronize()
    return out, sc, new


def check_norm(x, res, w, eps, group, got):
    """y is off by at most e = (n / 16 + 8) 2^-23 relative (the fp32 sum of squares: at most
    n / 64 terms a thread and a tree; rsqrt, two products), so a scale by e + 2^-23, and a code
    by half a step of e4m3 (2^-4 of it, 2^-10 below 2^-6) and e of the value."""
    out, sc, new = (None if t is None else t.cpu() for t in got)
    h, y, scale = norm_reference(x.cpu(), None if res is None else res.cpu(), w.cpu(), eps, group)
    n = x.shape[1]
    e = (n / 16 + 8) * 2.0 ** -23
    assert ((sc.double() - scale).abs() <= (e + 2.0 ** -23) * scale).all()
    if new is not None:
        assert torch.equal(new, h.float().to(torch.bfloat16))
    per = scale.repeat_interleave(group or n, 1)[:, :n]
    quotient = y / per
    d = (out.float().double() - quotient).abs()
    assert (d <= quotient.abs() * (2.0 ** -4 + 3 * e) + 2.0 ** -10).all()


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("T,n", [(1, 1), (3, 7), (5, 100), (1, 128), (64, 128), (2, 136), (7, 1000),
                                 (3, 1001), (4, 4096), (2, 6144), (300, 520), (2, 16384), (1, 32768),
                                 (1, 32767)])
def test_norm(T, n, group):
    g = torch.Generator().manual_seed(T * 7 + n)
    x = torch.randn((T, n), generator=g).to(torch.bfloat16).cuda()
    res = (4 * torch.randn((T, n), generator=g)).to(torch.bfloat16).cuda()
    w = (1 + 0.2 * torch.randn(n, generator=g)).to(torch.bfloat16).cuda()
    check_norm(x, res, w, 1e-6, group, run_norm(x, res, w, 1e-6, group))
    check_norm(x, None, w, 1e-5, group, run_norm(x, None, w, 1e-5, group, out_residual=False))


@pytest.mark.parametrize("n,pad", [(256, 8), (256, 3), (100, 1)])
def test_norm_of_strided_rows_in_place(n, pad):
    g = torch.Generator().manual_seed(n + pad)
    x = torch.randn((9, n + pad), generator=g).to(torch.bfloat16).cuda()[:, pad:]
    res = torch.randn((9, n), generator=g).to(torch.bfloat16).cuda()
    w = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    before = res.clone()
    out = torch.empty((9, n), dtype=torch.uint8, device="cuda")
    sc = torch.empty(9, device="cuda")
    idx.idx_add_rmsnorm_fp8(x, res, w, 1e-6, 0, out, sc, res)
    check_norm(x, before, w, 1e-6, 0, (out.view(torch.float8_e4m3fn), sc[:, None], res))


def test_norm_of_zero_and_not_finite_rows():
    n = 384
    x = torch.randn((4, n), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[0] = 0
    x[1, 200] = float("nan")
    x[2, 200] = float("inf")
    w = torch.ones(n, dtype=torch.bfloat16)
    for group in (0, 128):
        for cut in (0, 1):     # the 16-byte path and the element-wise one
            xx = x.cuda() if not cut else torch.cat([x[:, :1], x], 1).cuda()[:, 1:]
            out, sc, _ = (t.cpu() for t in run_norm(xx, None, w.cuda(), 1e-6, group))
            out = out.float()
            assert (out[0] == 0).all() and (sc[0] == 2.0 ** -96 / 448).all()
            assert torch.isnan(sc[1]).all() and torch.isnan(out[1]).all()
            assert torch.isnan(out[2, 200]) and torch.isnan(sc[2, 200 // group if group else 0])
            assert torch.isfinite(out[3]).all() and torch.isfinite(sc[3]).all()


def test_norm_makes_the_index_steps_e4m3_queries():
    """dim 128, group 0: codes and scales as idx_score_topk takes them."""
    x = torch.randn((12, 128), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    out, sc, _ = run_norm(x, None, w, 1e-6, 0)
    y = x.double() / torch.sqrt((x.double() ** 2).mean(1, keepdim=True) + 1e-6)
    back = out.float().double() * sc.double()
    assert ((back - y).abs() <= y.abs() * 2.0 ** -4 + sc.double() * 2.0 ** -10 + 1e-6).all()


def test_the_native_calls_and_the_python_ones_agree():
    """The CPython module's functions, the Python functions of the same names, keywords and a
    given stream (which the module hands on), and what both refuse."""
    from sparse_attention_indexer_packed_gb300 import _lib
    assert idx.idx_store_kv is not _lib.idx_store_kv, "the CPython module has not been built"
    src = tokens(70, 2, 21).cuda()
    slots = torch.randperm(128, generator=torch.Generator().manual_seed(1))[:70].cuda()
    for dtype in ("bf16", "fp8_e4m3"):
        got = []
        for call in (lambda *a: idx.idx_store_kv(*a), lambda *a: _lib.idx_store_kv(*a),
                     lambda *a: idx.idx_store_kv(*a, stream=torch.cuda.current_stream())):
            planes = [tuple(None if t is None else t.cuda() for t in _attn.plane(256, dtype, 7)) for _ in range(2)]
            call(src[:, :2], src[:, 2:4], slots, *planes[0], *planes[1], dtype, 2)
            got.append([t.cpu() for p in planes for t in p if t is not None])
        for other in got[1:]:
            assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(got[0], other))
    x = torch.randn((5, 256), device="cuda").to(torch.bfloat16)
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    out, sc = torch.empty((5, 256), dtype=torch.uint8, device="cuda"), torch.empty((5, 2), device="cuda")
    for call in (idx.idx_add_rmsnorm_fp8, _lib.idx_add_rmsnorm_fp8):
        out.zero_()
        call(x, None, w, 1e-6, 128, out, sc)
        check_norm(x, None, w, 1e-6, 128, (out.view(torch.float8_e4m3fn), sc, None))
        for bad in ((x.float(), None, w, 1e-6, 128, out, sc), (x, None, w[:7], 1e-6, 128, out, sc),
                    (x, None, w, 1e-6, 64, out, sc), (x, x.t(), w, 1e-6, 128, out, sc),
                    (x, None, w, 1e-6, 128, out, sc[:, :1]), (x.cpu(), None, w, 1e-6, 128, out, sc)):
            with pytest.raises(idx.IdxError):
                call(*bad)
