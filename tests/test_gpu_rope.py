"""idx_norm_rope_store (needs a GPU) against 64 bits: norm, rotation on one or several axes,
queries in bf16 and e4m3, keys and values in every type of cache."""
import pytest
import torch

import _attn
import _nvfp4
import sparse_attention_indexer_packed_gb300 as idx

pytestmark = pytest.mark.gpu
EPS = 1e-6


def plane(rows, dtype, seed):
    if dtype == "nvfp4":
        return _nvfp4.plane(rows, seed)
    return _attn.plane(rows, dtype, seed)


def projection(T, Hq, H, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, Hq + 2 * H, 128), generator=g)
    x *= torch.exp2(torch.randint(-6, 7, (T, Hq + 2 * H, 1), generator=g).float())
    return x.to(torch.bfloat16)


class Case:
    def __init__(self, T, Hq, H, dtype, seed=1, rotary_dim=128, interleaved=False, axes=1, norm=True,
                 q_codes=False, values=True, pair_axis=None, outers=(1.0, 1.0)):
        g = torch.Generator().manual_seed(seed)
        self.__dict__.update(T=T, Hq=Hq, H=H, dtype=dtype, rotary_dim=rotary_dim, interleaved=interleaved,
                             axes=axes, q_codes=q_codes, outers=outers)
        self.x = projection(T, Hq, H, seed)
        self.pages = T // 64 + 3
        self.slots = torch.randperm(self.pages * 64, generator=g)[:T]
        if T > 4:
            self.slots[1], self.slots[3], self.slots[4] = -1, self.pages * 64, -2 ** 60
        self.qw, self.kw = [(1 + 0.2 * torch.randn(128, generator=g)).to(torch.bfloat16) if norm else None
                            for _ in range(2)]
        n = rotary_dim // 2
        angle = torch.randn((500, n), generator=g, dtype=torch.float64) * 3
        self.table = torch.cat([angle.cos(), angle.sin()], 1).float() if n else None
        self.pos = torch.randint(0, 500, (axes, T), generator=g).to(torch.int32) if n else None
        self.pair_axis = pair_axis if pair_axis is not None or axes == 1 else bytes(
            torch.randint(0, axes, (n,), generator=g).tolist())
        self.k, self.v = plane(self.pages * H * 64, dtype, 5), plane(self.pages * H * 64, dtype, 6)
        self.values = values

    def run(self):
        d = lambda t: None if t is None else t.cuda()  # noqa: E731
        Hq, H, T = self.Hq, self.H, self.T
        x = self.x.cuda()
        q = x[:, :Hq] if Hq else None
        out = outs = None
        if Hq:
            out = torch.full((T, Hq, 128), 7.0, device="cuda").to(
                torch.float8_e4m3fn if self.q_codes else torch.bfloat16)
            outs = torch.full((T, Hq), 7.0, device="cuda") if self.q_codes else None
        k, v = tuple(map(d, self.k)), tuple(map(d, self.v))
        pos = self.pos if self.pos is None or self.axes > 1 else self.pos[0]
        idx.idx_norm_rope_store(q, x[:, Hq:Hq + H], x[:, Hq + H:] if self.values else None, d(self.qw), d(self.kw),
                                EPS, d(self.table), d(pos), self.pair_axis, self.interleaved, d(self.slots),
                                out, outs, *k, *(v if self.values else (None, None)), self.dtype, H,
                                *self.outers)
        c = lambda t: None if t is None else t.cpu()  # noqa: E731
        return c(out), c(outs), tuple(map(c, k)), tuple(map(c, v))

    def turned(self, x, weight):
        """Normed and rotated rows in 64 bits, and the bound on an fp32 evaluation's error: a sum
        of 128 squares in chains of 12 roundings, half of it in the root; rsqrt 2^-22, two
        products; the rotation's two products and sum: below 2^-19 of |a cos| + |b sin|."""
        x = x.double()
        if weight is not None:
            x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
        y, size = x.clone(), x.abs()
        n = self.rotary_dim // 2
        for i in range(n):
            a, b = (2 * i, 2 * i + 1) if self.interleaved else (i, i + n)
            p = self.pos[self.pair_axis[i] if self.pair_axis else 0].long()
            c, z = self.table[p, i].double()[:, None], self.table[p, n + i].double()[:, None]
            y[..., a] = x[..., a] * c - x[..., b] * z
            y[..., b] = x[..., b] * c + x[..., a] * z
            size[..., a] = x[..., a].abs() * c.abs() + x[..., b].abs() * z.abs()
            size[..., b] = x[..., b].abs() * c.abs() + x[..., a].abs() * z.abs()
        return y, size * 2.0 ** -19


def check_bf16(got, y, e):
    d = (got.double() - y).abs()
    assert (d <= e + (y.abs() + e) * 2.0 ** -8).all()


def check_e4m3(codes, scale, y, e):
    """scale = amax / 448 (the error of the largest element, two roundings); codes: half a step."""
    amax, ea = y.abs().amax(-1), e.amax(-1)
    assert ((scale.double() * 448 - amax).abs() <= ea + amax * 2.0 ** -22).all()
    s = scale.double()[..., None]
    d = (codes.view(torch.float8_e4m3fn).double() * s - y).abs()
    assert (d <= e + (y.abs() + e) * (2.0 ** -4 + 2.0 ** -20) + s * 2.0 ** -10).all()


def check_nvfp4(payload, scale, y, e, outer):
    y, e = y / outer, e / outer
    amax, ea = y.abs().unflatten(-1, (8, 16)).amax(-1), e.unflatten(-1, (8, 16)).amax(-1)
    s = scale.contiguous().view(torch.float8_e4m3fn).double()
    want = (amax / 6).clamp(max=448)
    assert ((s - want).abs() <= ea / 6 + want * 2.0 ** -4 + 2.0 ** -10).all()
    s = s.repeat_interleave(16, -1)
    rows = payload.reshape(-1, 64)
    code = _nvfp4.values64((rows, torch.full((len(rows), 8), 0x38, dtype=torch.uint8)),
                           torch.arange(len(rows))).reshape(y.shape)
    ratio = y.abs() / s.clamp_min(2.0 ** -20)
    # half the gap between codes; past 6 the code saturates and is off by ratio - 6 (a scale below
    # 2^-6 is held in steps of 2^-9: amax / 6 = 1.4 * 2^-9 gives the scale 2^-9 and the ratio 8.4)
    half = torch.where(ratio <= 2, 0.25, torch.where(ratio <= 4, 0.5, (ratio - 6).clamp_min(1.0)))
    assert ((code * s - y).abs() <= e + s * half + (ratio + 1) * s * 2.0 ** -20).all()


def check_case(c):
    out, outs, k, v = c.run()
    Hq, H = c.Hq, c.H
    if Hq:
        y, e = c.turned(c.x[:, :Hq], c.qw)
        if c.q_codes:
            check_e4m3(out, outs, y, e)
        else:
            check_bf16(out, y, e)
    ok = (c.slots >= 0) & (c.slots < c.pages * 64)
    y, e = c.turned(c.x[:, Hq:Hq + H], c.kw)
    rows = torch.stack([(c.slots[ok] // 64 * H + h) * 64 + c.slots[ok] % 64 for h in range(H)], 1)
    untouched = torch.ones(len(k[0]), dtype=torch.bool)
    untouched[rows] = False
    for new, old in ((k, c.k), (v, c.v)):
        for a, b in zip(new, old):
            if b is not None:
                assert torch.equal(a[untouched].view(torch.uint8), b[untouched].view(torch.uint8))
    y, e = y[ok], e[ok]
    if c.dtype == "bf16":
        check_bf16(k[0][rows], y, e)
    elif c.dtype == "fp8_e4m3":
        check_e4m3(k[0][rows], k[1][rows][..., 0], y, e)
    else:
        check_nvfp4(k[0][rows], k[1][rows], y, e, c.outers[0])
    # the values: the bytes of the store
    ref = tuple(None if t is None else t.clone().cuda() for t in c.v)
    if c.values:
        src, slots = c.x[:, Hq + H:].cuda(), c.slots.cuda()
        if c.dtype == "nvfp4":
            idx.idx_store_kv_nvfp4(src, None, slots, *ref, None, None, H, c.outers[1])
        else:
            idx.idx_store_kv(src, None, slots, *ref, None, None, c.dtype, H)
    for a, b in zip(v, ref):
        if b is not None:
            assert torch.equal(a.view(torch.uint8), b.cpu().view(torch.uint8))


DTYPES = ["bf16", "fp8_e4m3", "nvfp4"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,Hq,H", [(1, 1, 1), (1, 16, 2), (2, 3, 1), (15, 4, 4), (16, 8, 1), (17, 5, 3),
                                    (64, 16, 2), (300, 32, 4), (2001, 6, 2), (700, 0, 1)])
def test_sizes(dtype, T, Hq, H):
    check_case(Case(T, Hq, H, dtype, seed=T + Hq))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary_dim", [0, 16, 32, 48, 64, 80, 96, 112, 128])
def test_rotated_parts(dtype, interleaved, rotary_dim):
    check_case(Case(70, 6, 2, dtype, seed=rotary_dim, rotary_dim=rotary_dim, interleaved=interleaved))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("rotary_dim", [32, 96, 128])
@pytest.mark.parametrize("how", ["any", "runs", "turns"])
def test_axes(interleaved, axes, rotary_dim, how):
    n = rotary_dim // 2
    by = {"any": None, "runs": bytes(i * axes // n for i in range(n)), "turns": bytes(i % axes for i in range(n))}[how]
    for T in (5, 400):
        check_case(Case(T, 9, 1, "nvfp4" if T == 5 else "bf16", seed=axes + n, rotary_dim=rotary_dim,
                        interleaved=interleaved, axes=axes, pair_axis=by))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("norm,q_codes,values", [(False, False, True), (True, True, False), (False, True, True),
                                                 (True, False, False)])
def test_parts_left_out(dtype, norm, q_codes, values):
    for T in (33, 600):
        check_case(Case(T, 7, 2, dtype, seed=T, norm=norm, q_codes=q_codes, values=values, rotary_dim=64))


def test_outer_scales():
    for T in (3, 500):
        check_case(Case(T, 4, 2, "nvfp4", seed=T, outers=(0.25, 8.0)))


@pytest.mark.parametrize("dtype", DTYPES)
def test_without_norm_and_rotation_keys_are_the_stores(dtype):
    c = Case(90, 4, 2, dtype, seed=3, norm=False, rotary_dim=0)
    out, _, k, v = c.run()
    assert torch.equal(out.view(torch.int16), c.x[:, :4].contiguous().view(torch.int16))
    k2, v2 = [tuple(None if t is None else t.cuda() for t in p) for p in (c.k, c.v)]
    x = c.x.cuda()
    if dtype == "nvfp4":
        idx.idx_store_kv_nvfp4(x[:, 4:6], x[:, 6:], c.slots.cuda(), *k2, *v2, 2)
    else:
        idx.idx_store_kv(x[:, 4:6], x[:, 6:], c.slots.cuda(), *k2, *v2, dtype, 2)
    for a, b in zip(k + v, k2 + v2):
        if b is not None:
            assert torch.equal(a.view(torch.uint8), b.cpu().view(torch.uint8))


@pytest.mark.parametrize("dtype", DTYPES)
def test_positions_outside_the_table_are_nan(dtype):
    c = Case(40, 3, 1, dtype, seed=5, rotary_dim=64, axes=2, pair_axis=bytes(i // 16 for i in range(32)))
    c.slots = torch.arange(40)
    c.pos[0, 7], c.pos[1, 9], c.pos[1, 11] = 500, -1, 2 ** 31 - 1
    out, _, k, _ = c.run()
    bad = {7: range(0, 16), 9: range(16, 32), 11: range(16, 32)}
    nan = torch.zeros((40, 128), dtype=torch.bool)
    for t, pairs in bad.items():
        for i in pairs:
            nan[t, i] = nan[t, i + 32] = True
    assert torch.equal(torch.isnan(out.float()), nan[:, None].expand(-1, 3, -1))
    if dtype == "bf16":
        got = torch.isnan(k[0][:40].float())
    elif dtype == "fp8_e4m3":
        got = torch.isnan(k[0][:40].view(torch.float8_e4m3fn).float()) & torch.isnan(k[1][:40])
        nan = nan.any(1, keepdim=True).expand(-1, 128)
    else:
        got = torch.isnan(_nvfp4.values64(k, torch.arange(40)))
        nan = nan.unflatten(1, (8, 16)).any(2, keepdim=True).expand(-1, -1, 16).flatten(1)
    assert torch.equal(got, nan)


def test_rows_that_are_not_finite_or_zero():
    c = Case(20, 2, 1, "bf16", seed=8)
    c.slots = torch.arange(20)
    c.x[3, 0, 5], c.x[4, 2, 9], c.x[5] = float("nan"), float("inf"), 0
    out, _, k, _ = c.run()
    assert torch.isnan(out[3, 0].float()).all() and not torch.isnan(out[3, 1].float()).any()
    assert torch.isnan(k[0][4].float()).any()
    assert (out[5] == 0).all() and (k[0][5] == 0).all()
    others = [i for i in range(20) if i not in (3, 4)]
    assert torch.isfinite(out[others].float()).all() and torch.isfinite(k[0][others].float()).all()


def test_replayed_on_a_stream_of_its_own():
    c = Case(100, 8, 2, "nvfp4", seed=9)
    first = c.run()
    x, slots = c.x.cuda(), c.slots.cuda()
    out = torch.empty((100, 8, 128), dtype=torch.bfloat16, device="cuda")
    k, v = [tuple(t.cuda() for t in p) for p in (c.k, c.v)]
    args = (x[:, :8], x[:, 8:10], x[:, 10:], c.qw.cuda(), c.kw.cuda(), EPS, c.table.cuda(), c.pos[0].cuda(), None,
            False, slots, out, None, *k, *v, "nvfp4", 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    idx.idx_norm_rope_store(*args, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        idx.idx_norm_rope_store(*args)
    out.zero_()
    for t, old in zip(k + v, c.k + c.v):
        t.copy_(old)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), first[0])
    for a, b in zip(k + v, first[2] + first[3]):
        assert torch.equal(a.cpu(), b)


def test_no_tokens():
    c = Case(0, 2, 1, "bf16")
    c.run()
