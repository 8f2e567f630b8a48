"""The grouped products of block-scaled operands against plain 64-bit forms.

Tolerance.  A product of two E4M3 (or E2M1) values has at most 8 (4)
significant bits and its scales are powers of two, so it is exact in fp32; a
sum of n of them in any order, with at most one unit in the last place (2^-23
relative) lost at each of the n additions, is off by at most n 2^-23 sum |a w|.
The one rounding to the output adds half a step of it: 2^-8 (bf16) or 2^-24
(fp32) of the result.  So |out - ref| <= h |ref| + (1 + h) n 2^-23 sum |a w|.
"""
import ctypes

import pytest
import torch

import moe_gated_activation_b200 as mg
import products_ref as ref
from moe_gated_activation_b200 import _capi

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _codes(g, *shape):
    """Every finite E4M3 code."""
    c = torch.randint(0, 254, shape, generator=g, device="cuda", dtype=torch.int32)
    return (c + (c >= 0x7F)).to(torch.uint8)


def _scales(g, *shape):
    return torch.randint(118, 131, shape, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)


def _bytes(g, *shape):
    return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)


def _offs(splits):
    o = [0]
    for m in splits:
        o.append(o[-1] + m)
    return o


def _dev(offs):
    return torch.tensor(offs, dtype=torch.int64, device="cuda")


def _blocks(splits):
    return _offs([(m + 31) // 32 for m in splits])


def _check(got, want, size, n, what):
    h = HALF[got.dtype]
    err = (got.double() - want).abs()
    lim = h * want.abs() + (1 + h) * n * 2.0 ** -23 * size
    assert got.shape == want.shape
    bad = ~(err <= lim)
    if bad.any():
        i = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first {i}: "
                             f"{got[tuple(i)].item()} for {want[tuple(i)].item()}")


def _rows_case(op, splits, K, H, seed):
    """(call, reference, sum of magnitudes, length of the sum, output width)
    of a row product; K: the weights' columns, H: their rows."""
    g = _gen(seed)
    offs, E, M = _offs(splits), len(splits), sum(splits)
    ro = _dev(offs)
    if op == "gemm4":
        a, sa = _bytes(g, M, K // 2), _scales(g, M, K // 32)
        w, sw = _bytes(g, E * H, K // 2), _scales(g, E * H, K // 32)
        av, wv = ref.values4(a, sa), ref.values4(w, sw).unflatten(0, (E, H)).mT
        call = lambda **kw: mg.grouped_mxfp4_gemm(mg.MXFP4(a, sa), mg.MXFP4(w, sw), ro, **kw)
    elif op == "gemm":
        a, sa = _codes(g, M, K), _scales(g, M, K // 32)
        w, sw = _codes(g, E * H, K), _scales(g, E * H, K // 32)
        av, wv = ref.values8(a, sa, 1), ref.values8(w, sw, 1).unflatten(0, (E, H)).mT
        call = lambda **kw: mg.grouped_mxfp8_gemm(mg.MXFP8(a, None, sa, None),
                                                  mg.MXFP8(w, None, sw, None), ro, **kw)
    else:
        a, sa = _codes(g, M, H), _scales(g, M, H // 32)
        w, sw = _codes(g, E * H, K), _scales(g, E * H // 32, K)
        av, wv = ref.values8(a, sa, 1), ref.values8(w, sw, 0).unflatten(0, (E, H))
        call = lambda **kw: mg.grouped_mxfp8_dgrad(mg.MXFP8(a, None, sa, None),
                                                   mg.MXFP8(None, w, None, sw), ro, **kw)
    want = ref.grouped(lambda e, r: av[r] @ wv[e], offs)
    size = ref.grouped(lambda e, r: av[r].abs() @ wv[e].abs(), offs)
    return call, want, size, (H if op == "dgrad" else K), want.shape[1], (a, sa, w, sw, ro)


RAGGED = [0, 1, 31, 33, 0, 127, 129, 64, 255, 257, 0]
SHAPES = [
    ([1], 32, 32),                       # one row, one block
    ([1], 2048, 1536),                   # one token of a wide expert
    ([128], 128, 128),                   # one full tile
    (RAGGED, 96, 160),
    (RAGGED, 416, 288),
    ([3, 0, 2, 1], 2080, 544),
    ([2, 0, 1] * 100, 64, 32),           # 300 groups
    ([700, 0, 1300, 130], 1056, 2592),   # pairs of SMs
    ([4000], 288, 1312),
    ([513] * 9, 32, 1024),
]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("op", ["gemm", "dgrad", "gemm4"])
def test_row_products(cuda_device, op, i, out_dtype):
    splits, K, H = SHAPES[i]
    call, want, size, n, _, _ = _rows_case(op, splits, K, H, 10 + i)
    out, status = call(out_dtype=out_dtype)
    assert int(status) == 0
    _check(out, want, size, n, (op, splits, K, H))


def _wgrad_case(splits, H, K, seed):
    g = _gen(seed)
    M, offs, cb = sum(splits), _offs(splits), _blocks(splits)
    dy, x = _codes(g, M, H), _codes(g, M, K)
    sy, sx = _scales(g, cb[-1], H), _scales(g, cb[-1], K)
    yv, xv = ref.values8(dy, sy, 0, offs), ref.values8(x, sx, 0, offs)
    r = [slice(lo, hi) for lo, hi in zip(offs[:-1], offs[1:])]
    want = torch.stack([yv[s].T @ xv[s] for s in r])
    size = torch.stack([yv[s].abs().T @ xv[s].abs() for s in r])
    return dy, x, sy, sx, _dev(offs), _dev(cb), want, size


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("splits,H,K", [
    ([1], 32, 32), ([31], 128, 128), ([128], 256, 256), (RAGGED, 160, 96), (RAGGED, 288, 416),
    ([3, 0, 2, 1], 544, 2080), ([2, 0, 1] * 100, 32, 64), ([700, 0, 1301, 130], 2592, 1056),
    ([0, 0], 64, 64), ([5000], 320, 2560),
])
def test_wgrad(cuda_device, splits, H, K, out_dtype):
    dy, x, sy, sx, ro, cb, want, size = _wgrad_case(splits, H, K, 40)
    dw, status = mg.grouped_mxfp8_wgrad(mg.MXFP8(None, dy, None, sy), mg.MXFP8(None, x, None, sx),
                                        ro, cb, out_dtype=out_dtype)
    assert int(status) == 0
    _check(dw, want, size, max(splits), (splits, H, K))


def test_wgrad_accumulates(cuda_device):
    splits, H, K = [33, 0, 95], 96, 288
    dy, x, sy, sx, ro, cb, want, size = _wgrad_case(splits, H, K, 41)
    a, b = mg.MXFP8(None, dy, None, sy), mg.MXFP8(None, x, None, sx)
    once, _ = mg.grouped_mxfp8_wgrad(a, b, ro, cb)
    held = torch.randn(once.shape, generator=_gen(1), device="cuda")
    out = held.clone()
    got, _ = mg.grouped_mxfp8_wgrad(a, b, ro, cb, out=out, accumulate=True)
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(out, held + once)         # one fp32 addition


def test_wgrad_accumulates_subnormals(cuda_device):
    """What dw holds and what is added, from 2^-100 down to below the smallest
    number: the bits of one fp32 addition."""
    g, H, K = _gen(43), 96, 288
    dy, x = _codes(g, 40, H), _codes(g, 40, K)
    e = 60 - torch.arange(K, device="cuda", dtype=torch.int32) % 61
    sx = e.to(torch.uint8).expand(2, K).contiguous()
    sy = torch.full((2, H), 87, dtype=torch.uint8, device="cuda")
    a, b = mg.MXFP8(None, dy, None, sy), mg.MXFP8(None, x, None, sx)
    ro, cb = _dev([0, 40]), _dev([0, 2])
    once, _ = mg.grouped_mxfp8_wgrad(a, b, ro, cb)
    held = torch.ldexp(torch.randn(once.shape, generator=g, device="cuda"),
                       torch.randint(-150, -100, once.shape, generator=g, device="cuda"))
    small = lambda t: bool(((t != 0) & (t.abs() < 2.0 ** -126)).any())
    assert small(once) and small(held) and small(held + once)
    out = held.clone()
    mg.grouped_mxfp8_wgrad(a, b, ro, cb, out=out, accumulate=True)
    assert torch.equal(out, held + once)


def test_wgrad_accumulates_long_sums(cuda_device):
    splits, H, K = [8193, 0, 20011, 31, 8192, 9000], 1312, 288
    dy, x, sy, sx, ro, cb, want, size = _wgrad_case(splits, H, K, 42)
    out = torch.randn(want.shape, generator=_gen(2), device="cuda")
    want, size = want + out.double(), size + out.double().abs()
    a, b = mg.MXFP8(None, dy, None, sy), mg.MXFP8(None, x, None, sx)
    mg.grouped_mxfp8_wgrad(a, b, ro, cb, out=out, accumulate=True)
    _check(out, want, size, max(splits), "accumulate")


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("splits", [[1, 0, 17], [300, 0, 2000, 130]])
@pytest.mark.parametrize("op", ["gemm", "dgrad", "gemm4"])
def test_long_row_sums(cuda_device, op, splits, out_dtype):
    K, H = (2592, 16480) if op == "dgrad" else (16480, 2592)
    call, want, size, n, _, _ = _rows_case(op, splits, K, H, 60)
    out, status = call(out_dtype=out_dtype)
    assert int(status) == 0
    _check(out, want, size, n, (op, splits))


@pytest.mark.parametrize("rows,cols", [(65536, 128), (65519, 128), (65536, 2048)])
@pytest.mark.parametrize("op", ["wgrad", "gemm", "dgrad", "gemm4"])
def test_long_sums_keep_small_terms(cuda_device, op, rows, cols):
    """A sum over `rows` products of 2^23 (the first block) and 2^-5 for every
    other block.  In fp32 beside 2^23 a term of 2^-5 is 1/32 of a step and may
    vanish.  Sums in segments of 256 steps (of 32 products, MXFP4: 64) lose
    those of the first segment, at most 256 / 32 = 8 (MXFP4: 512 / 32 = 16);
    later ones are sums of at most 16, exact by themselves, and each is added
    with at most half a step of 2^23, 0.5, for 7 (MXFP4: 3) of them: 11.5
    (17.5).  One sum would lose up to 64, all of them."""
    if op != "wgrad" and rows % 32:
        pytest.skip("the summed index is whole blocks there")
    nb, m = (rows + 31) // 32, cols if op == "wgrad" else min(cols, 1600)
    ones8 = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device="cuda")
    ones4 = lambda *s: torch.full(s, 0x22, dtype=torch.uint8, device="cuda")
    scale = lambda *s: torch.full(s, 127, dtype=torch.uint8, device="cuda")
    exps = torch.full((nb,), 127 - 10, dtype=torch.uint8, device="cuda")
    exps[0] = 127 + 18
    byrow = exps.expand(m, nb).contiguous()
    ro = _dev([0, m])
    if op == "wgrad":
        dy = mg.MXFP8(None, ones8(rows, m), None, exps[:, None].expand(nb, m).contiguous())
        x = mg.MXFP8(None, ones8(rows, cols), None, scale(nb, cols))
        out, status = mg.grouped_mxfp8_wgrad(dy, x, _dev([0, rows]), _dev([0, nb]))
    elif op == "gemm":
        out, status = mg.grouped_mxfp8_gemm(
            mg.MXFP8(ones8(m, rows), None, byrow, None),
            mg.MXFP8(ones8(cols, rows), None, scale(cols, nb), None), ro, out_dtype=torch.float32)
    elif op == "dgrad":
        out, status = mg.grouped_mxfp8_dgrad(
            mg.MXFP8(ones8(m, rows), None, byrow, None),
            mg.MXFP8(None, ones8(rows, cols), None, scale(nb, cols)), ro, out_dtype=torch.float32)
    else:
        out, status = mg.grouped_mxfp4_gemm(
            mg.MXFP4(ones4(m, rows // 2), byrow),
            mg.MXFP4(ones4(cols, rows // 2), scale(cols, nb)), ro, out_dtype=torch.float32)
    assert int(status) == 0
    last = rows - 32 * (nb - 1)
    want = 2.0 ** 23 + (nb - 2) / 32 + last / 1024
    err = (out.double() - want).abs().max().item()
    assert err <= (17.5 if op == "gemm4" else 11.5), err


@pytest.mark.parametrize("op", ["wgrad", "gemm", "dgrad", "gemm4"])
def test_long_bf16_sums_keep_small_terms(cuda_device, op):
    """A bf16 output's sum of 131,072 steps, the first of 2^23 and the others of
    1/2, which one accumulator drops: 2^16 in all, a whole step of bf16 there.
    In parts of 256 steps only the first part's are dropped, less than 128; the
    other parts are exact, and so are their additions, of integers below 2^24.
    The rounding takes half a step, 2^15, at most."""
    per, steps = (64, 131072) if op == "gemm4" else (32, 131072)
    n, m, cols = per * steps, 32, 64
    ones8 = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device="cuda")
    ones4 = lambda *s: torch.full(s, 0x22, dtype=torch.uint8, device="cuda")
    scale = lambda *s: torch.full(s, 127, dtype=torch.uint8, device="cuda")
    exps = torch.full((n // 32,), 127 - (7 if op == "gemm4" else 6), dtype=torch.uint8, device="cuda")
    exps[0] = 127 + 18
    if op == "gemm4":
        exps[1] = 0      # the first step's other half
    byrow, ro = exps.expand(m, -1).contiguous(), _dev([0, m])
    if op == "wgrad":
        dy = mg.MXFP8(None, ones8(n, m), None, exps[:, None].expand(-1, m).contiguous())
        x = mg.MXFP8(None, ones8(n, cols), None, scale(n // 32, cols))
        out, st = mg.grouped_mxfp8_wgrad(dy, x, _dev([0, n]), _dev([0, n // 32]),
                                         out_dtype=torch.bfloat16)
    elif op == "gemm":
        out, st = mg.grouped_mxfp8_gemm(mg.MXFP8(ones8(m, n), None, byrow, None),
                                        mg.MXFP8(ones8(cols, n), None, scale(cols, n // 32), None), ro)
    elif op == "dgrad":
        out, st = mg.grouped_mxfp8_dgrad(mg.MXFP8(ones8(m, n), None, byrow, None),
                                         mg.MXFP8(None, ones8(n, cols), None, scale(n // 32, cols)), ro)
    else:
        out, st = mg.grouped_mxfp4_gemm(mg.MXFP4(ones4(m, n // 2), byrow),
                                        mg.MXFP4(ones4(cols, n // 2), scale(cols, n // 32)), ro)
    assert int(st) == 0 and out.dtype == torch.bfloat16
    want = 2.0 ** 23 + (steps - 1) / 2
    err = (out.double() - want).abs().max().item()
    assert err <= 2.0 ** 15 + 128, err


@pytest.mark.parametrize("op", ["wgrad", "gemm", "dgrad", "gemm4"])
def test_long_bf16_sums_are_the_fp32_ones_rounded(cuda_device, op):
    """Both are made of the same parts, added in the same order; several such
    tiles and short ones follow one another on an SM."""
    g = _gen(51)
    n = (1 << 20) + 32 if op == "gemm4" else (1 << 19) + 32      # 16385 steps
    if op == "gemm4":
        n += 32
    if op == "wgrad":
        splits, H, K = [n, 0, 8000, 600001, 77, 31] + [5] * 20, 288, 1312
        M, offs, cb = sum(splits), _offs(splits), _blocks(splits)
        dy = mg.MXFP8(None, _codes(g, M, H), None, _scales(g, cb[-1], H))
        x = mg.MXFP8(None, _codes(g, M, K), None, _scales(g, cb[-1], K))
        call = lambda dt: mg.grouped_mxfp8_wgrad(dy, x, _dev(offs), _dev(cb), out_dtype=dt)
    else:
        M, N, ro = 1030, 2592, _dev([0, 1030])
        if op == "gemm4":
            a = mg.MXFP4(_bytes(g, M, n // 2), _scales(g, M, n // 32))
            w = mg.MXFP4(_bytes(g, N, n // 2), _scales(g, N, n // 32))
            call = lambda dt: mg.grouped_mxfp4_gemm(a, w, ro, out_dtype=dt)
        else:
            a = mg.MXFP8(_codes(g, M, n), None, _scales(g, M, n // 32), None)
            if op == "gemm":
                w = mg.MXFP8(_codes(g, N, n), None, _scales(g, N, n // 32), None)
                call = lambda dt: mg.grouped_mxfp8_gemm(a, w, ro, out_dtype=dt)
            else:
                w = mg.MXFP8(None, _codes(g, n, N), None, _scales(g, n // 32, N))
                call = lambda dt: mg.grouped_mxfp8_dgrad(a, w, ro, out_dtype=dt)
    short, st = call(torch.bfloat16)
    full, _ = call(torch.float32)
    assert int(st) == 0 and torch.equal(short, full.bfloat16())


def test_long_bf16_wgrad_in_a_graph(cuda_device):
    """Its two launches follow the offsets of each replay, a long group beside an
    empty or a short one (of at most 256 steps: one sum for fp32 outputs too);
    bad offsets and a set no-op flag write nothing."""
    g, M, H, K = _gen(52), (1 << 19) + 8192 + 96, 160, 192
    nb = M // 32 + 2
    dy = mg.MXFP8(None, _codes(g, M, H), None, _scales(g, nb, H))
    x = mg.MXFP8(None, _codes(g, M, K), None, _scales(g, nb, K))
    ro, cb, st = _dev([0, M, M]), _dev([0, M // 32, M // 32]), torch.zeros(1, dtype=torch.int32, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty(2, H, K, dtype=torch.bfloat16, device="cuda")
    call = lambda: mg.grouped_mxfp8_wgrad(dy, x, ro, cb, out=out, status=st, noop_flag=flag)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for splits in ([M, 0], [8000, M - 8000], [M - 8187, 8187], [41, M - 41]):
        ro.copy_(_dev(_offs(splits)))
        cb.copy_(_dev(_blocks(splits)))
        full, _ = mg.grouped_mxfp8_wgrad(dy, x, ro, cb)
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert int(st) == 0 and torch.equal(out, full.bfloat16()), splits
    out.fill_(7)
    flag.fill_(1)
    graph.replay()
    flag.fill_(0)
    ro.copy_(_dev([0, M + 1, M]))
    graph.replay()
    torch.cuda.synchronize()
    assert int(st) == _capi.DEV_BAD_OFFSETS and bool((out == 7).all())


@pytest.mark.parametrize("op", ["gemm", "dgrad", "gemm4"])
def test_parts_of_sums_add_alike_in_every_row(cuda_device, op):
    """fp32 sums made in parts, down to parts and results below 2^-126: a row's
    bits do not depend on how many rows its group has after it.  All rows are
    alike and so are all groups' weights, whose scales run from 2^-8 to 2^-111
    over the columns.  The usual tolerance holds where the sum of magnitudes is
    2^-90 or more: it is 2^-99 there, far above any loss at the 2^-126 where
    fp32 has fewer bits."""
    splits, N, n = [64 + 5, 3, 32], 416, 32768 if op == "gemm4" else 16384
    g, E, M = _gen(50), 3, 104
    ro = _dev(_offs(splits))
    wexp = (119 - torch.arange(N, device="cuda") // 4).to(torch.uint8)   # of each output column
    sa = torch.full((M, n // 32), 40, dtype=torch.uint8, device="cuda")
    f32 = dict(out_dtype=torch.float32)
    if op == "gemm4":
        a, w = _bytes(g, 1, n // 2).expand(M, -1).contiguous(), _bytes(g, N, n // 2).repeat(E, 1)
        sw = wexp.repeat(E)[:, None].expand(-1, n // 32).contiguous()
        out, _ = mg.grouped_mxfp4_gemm(mg.MXFP4(a, sa), mg.MXFP4(w, sw), ro, **f32)
        av, wv = ref.values4(a[:1], sa[:1]), ref.values4(w[:N], sw[:N]).T
    elif op == "gemm":
        a, w = _codes(g, 1, n).expand(M, -1).contiguous(), _codes(g, N, n).repeat(E, 1)
        sw = wexp.repeat(E)[:, None].expand(-1, n // 32).contiguous()
        out, _ = mg.grouped_mxfp8_gemm(mg.MXFP8(a, None, sa, None), mg.MXFP8(w, None, sw, None),
                                       ro, **f32)
        av, wv = ref.values8(a[:1], sa[:1], 1), ref.values8(w[:N], sw[:N], 1).T
    else:
        a, w = _codes(g, 1, n).expand(M, -1).contiguous(), _codes(g, n, N).repeat(E, 1)
        sw = wexp[None].expand(E * n // 32, -1).contiguous()
        out, _ = mg.grouped_mxfp8_dgrad(mg.MXFP8(a, None, sa, None), mg.MXFP8(None, w, None, sw),
                                        ro, **f32)
        av, wv = ref.values8(a[:1], sa[:1], 1), ref.values8(w[:n], sw[:n // 32], 0)
    bits = out.view(torch.int32)
    assert torch.equal(bits, bits[:1].expand_as(bits))
    want, size = av @ wv, av.abs() @ wv.abs()
    big = size[0] >= 2.0 ** -90
    assert 0 < int(big.sum()) < N and bool((out[:, -1] == 0).all())
    _check(out[:1, big], want[:, big], size[:, big], n, op)


@pytest.mark.parametrize("splits", [[128, 0, 256], [1280, 128, 640]])
def test_tiled_scales(cuda_device, splits):
    """Scales in the GEMM-ready layout give the row-major ones' bits."""
    K, H = 384, 2560
    E = len(splits)
    for op in ("gemm", "dgrad", "gemm4"):
        call, want, size, n, _, (a, sa, w, sw, ro) = _rows_case(op, splits, K, H, 3)
        plain, _ = call()
        ta = ref.tile_scales(sa)
        tw = ref.tile_col_scales(sw, [E * H // 32]) if op == "dgrad" else ref.tile_scales(sw)
        for a_t, w_t in ((True, True), (True, False), (False, True)):
            s1, s2 = (ta if a_t else sa), (tw if w_t else sw)
            kw = dict(gemm_scales=a_t, w_gemm_scales=w_t)
            if op == "gemm4":
                got, _ = mg.grouped_mxfp4_gemm(mg.MXFP4(a, s1), mg.MXFP4(w, s2), ro, **kw)
            elif op == "gemm":
                got, _ = mg.grouped_mxfp8_gemm(mg.MXFP8(a, None, s1, None),
                                               mg.MXFP8(w, None, s2, None), ro, **kw)
            else:
                got, _ = mg.grouped_mxfp8_dgrad(mg.MXFP8(a, None, s1, None),
                                                mg.MXFP8(None, w, None, s2), ro, **kw)
            assert torch.equal(got, plain), (op, a_t, w_t)
    dy, x, sy, sx, ro, cb, want, size = _wgrad_case(splits, H, K, 4)
    plain, _ = mg.grouped_mxfp8_wgrad(mg.MXFP8(None, dy, None, sy), mg.MXFP8(None, x, None, sx), ro, cb)
    nb = [m // 32 for m in splits]
    got, st = mg.grouped_mxfp8_wgrad(mg.MXFP8(None, dy, None, ref.tile_col_scales(sy, nb)),
                                     mg.MXFP8(None, x, None, ref.tile_col_scales(sx, nb)), ro, cb,
                                     gemm_scales=True)
    assert int(st) == 0 and torch.equal(got, plain)


@pytest.mark.parametrize("K", [384, 1280])
@pytest.mark.parametrize("splits", [[5, 123, 0, 130, 126], [128, 3, 125, 256, 1, 127] * 3,
                                    [128, 700, 129, 1, 322, 1280], [640, 641, 1, 639, 639]])
@pytest.mark.parametrize("op", ["gemm", "dgrad", "gemm4"])
def test_tiled_scales_of_ragged_groups(cuda_device, op, splits, K):
    """The row products take tiled scales of groups that start anywhere in a
    tile: groups at a tile's start and inside one, in one launch, on single SMs
    and on pairs, give the row-major scales' bits."""
    H = 2560
    call, want, size, n, _, (a, sa, w, sw, ro) = _rows_case(
        op, splits, *((H, K) if op == "dgrad" else (K, H)), 30)
    plain, _ = call()
    _check(plain, want, size, n, (op, splits))
    ta = ref.tile_scales(sa)
    for _ in range(4):
        if op == "gemm4":
            got, st = mg.grouped_mxfp4_gemm(mg.MXFP4(a, ta), mg.MXFP4(w, sw), ro, gemm_scales=True)
        elif op == "gemm":
            got, st = mg.grouped_mxfp8_gemm(mg.MXFP8(a, None, ta, None),
                                            mg.MXFP8(w, None, sw, None), ro, gemm_scales=True)
        else:
            got, st = mg.grouped_mxfp8_dgrad(mg.MXFP8(a, None, ta, None),
                                             mg.MXFP8(None, w, None, sw), ro, gemm_scales=True)
        assert int(st) == 0 and torch.equal(got, plain)


def test_tiled_scales_need_whole_groups(cuda_device):
    dy, x, sy, sx, ro, cb, _, _ = _wgrad_case([64, 64], 128, 128, 4)
    out = torch.full((2, 128, 128), 7.0, device="cuda")
    _, st = mg.grouped_mxfp8_wgrad(mg.MXFP8(None, dy, None, sy), mg.MXFP8(None, x, None, sx), ro,
                                   cb, gemm_scales=True, out=out)
    assert int(st) == _capi.DEV_UNALIGNED_GROUPS and bool((out == 7).all())


@pytest.mark.parametrize("splits,K,H", [([5, 0, 40, 1], 160, 96), ([300, 0, 2000, 130], 288, 2592)])
def test_nan_stays_in_its_group(cuda_device, splits, K, H):
    """A group full of NaN (codes and scales) makes no other group's output
    NaN, whichever tiles its rows share."""
    bad = 2
    lo, hi = _offs(splits)[bad:bad + 2]
    for op in ("gemm", "dgrad", "gemm4"):
        call, want, size, n, _, (a, sa, w, sw, ro) = _rows_case(op, splits, K, H, 5)
        a[lo:hi] = 0x7F
        sa[lo:hi] = 255
        e = w.shape[0] // len(splits)
        w[bad * e:(bad + 1) * e] = 0x7F
        sw.view(len(splits), -1, sw.shape[1])[bad] = 255
        out, _ = call()
        assert bool(out[lo:hi].isnan().all())
        keep = [r for r in range(sum(splits)) if not lo <= r < hi]
        _check(out[keep], want[keep], size[keep], n, op)
    dy, x, sy, sx, ro, cb, want, size = _wgrad_case(splits, H, K, 6)
    b0, b1 = _blocks(splits)[bad:bad + 2]
    for t, s in ((dy, sy), (x, sx)):
        t[lo:hi] = 0x7F
        s[b0:b1] = 255
    dw, _ = mg.grouped_mxfp8_wgrad(mg.MXFP8(None, dy, None, sy), mg.MXFP8(None, x, None, sx), ro, cb)
    assert bool(dw[bad].isnan().all())
    keep = [e for e in range(len(splits)) if e != bad]
    _check(dw[keep], want[keep], size[keep], max(splits), "wgrad")


@pytest.mark.parametrize("seed", range(4))
def test_nan_after_every_group_end(cuda_device, seed):
    """wgrad on pairs: every other group is NaN and every group ends inside a
    block of 32, whose remaining rows, the next group's, take no part in either
    SM of a pair."""
    g = torch.Generator().manual_seed(seed)
    splits = [int(m) for m in torch.randint(1, 180, (64,), generator=g)]
    splits = [m + (m % 32 == 0) for m in splits]
    H, K = 544, 512
    dy, x, sy, sx, ro, cb, want, size = _wgrad_case(splits, H, K, 20 + seed)
    offs, blocks = _offs(splits), _blocks(splits)
    for e in range(1, 64, 2):
        for t, s in ((dy, sy), (x, sx)):
            t[offs[e]:offs[e + 1]] = 0x7F
            s[blocks[e]:blocks[e + 1]] = 255
    for _ in range(8):
        dw, st = mg.grouped_mxfp8_wgrad(mg.MXFP8(None, dy, None, sy), mg.MXFP8(None, x, None, sx),
                                        ro, cb)
        assert int(st) == 0 and bool(dw[1::2].isnan().all())
        _check(dw[::2], want[::2], size[::2], max(splits), splits)


@pytest.mark.parametrize("splits", [[5120], [3, 5110, 7], [1, 0, 31, 5087, 1], [5089, 31]])
def test_wgrad_of_whole_allocations(cuda_device, splits):
    """Code arrays that fill allocations of whole pages from their first byte to
    their last: the blocks at either end touch nothing beside them."""
    H, K = 4096, 6144
    dy, x, sy, sx, ro, cb, want, size = _wgrad_case(splits, H, K, 21)
    assert dy.numel() % (2 << 20) == 0 and x.numel() % (2 << 20) == 0
    for dt in HALF:
        dw, st = mg.grouped_mxfp8_wgrad(mg.MXFP8(None, dy, None, sy), mg.MXFP8(None, x, None, sx),
                                        ro, cb, out_dtype=dt)
        assert int(st) == 0
        _check(dw, want, size, max(splits), splits)


@pytest.mark.parametrize("M,H,K", [(1, 32, 32), (6, 3648, 3008), (9, 96, 4096), (40, 2592, 320)])
def test_wgrad_of_few_rows(cuda_device, M, H, K):
    """A few rows on a few groups, in arrays at ever other places."""
    g = torch.Generator().manual_seed(M)
    keep = []
    for i in range(12):
        cuts = sorted(int(v) for v in torch.randint(0, M + 1, (3,), generator=g))
        splits = [b - a for a, b in zip([0] + cuts, cuts + [M])]
        case = _wgrad_case(splits, H, K, 22 + i)
        dy, x, sy, sx, ro, cb, want, size = case
        dw, st = mg.grouped_mxfp8_wgrad(mg.MXFP8(None, dy, None, sy), mg.MXFP8(None, x, None, sx),
                                        ro, cb)
        assert int(st) == 0
        _check(dw, want, size, M, splits)
        keep.append((dy, x))


def test_extreme_scales(cuda_device):
    """Scales whose product leaves fp32's range overflow to infinity and
    vanish to zero; 2^-127 times 2^127 is one."""
    for b, want in ((254, float("inf")), (0, 0.0)):
        a = torch.full((4, 32), 0x38, dtype=torch.uint8, device="cuda")      # 1.0
        s = torch.full((4, 1), b, dtype=torch.uint8, device="cuda")
        w, sw = a.repeat(8, 1), s.repeat(8, 1)
        ro = _dev([0, 4])
        out, _ = mg.grouped_mxfp8_gemm(mg.MXFP8(a, None, s, None), mg.MXFP8(w, None, sw, None), ro,
                                       out_dtype=torch.float32)
        assert bool((out == want).all()), b
        out, _ = mg.grouped_mxfp8_gemm(mg.MXFP8(a, None, s, None),
                                       mg.MXFP8(w, None, 254 - sw, None), ro,
                                       out_dtype=torch.float32)
        assert bool((out == 32).all()), b


@pytest.mark.parametrize("op", ["gemm", "dgrad", "gemm4"])
def test_wide_output_and_status(cuda_device, op):
    """A view of a wider output keeps its other columns; bad offsets and a set
    no-op flag write nothing."""
    splits, K, H = [40, 0, 90], 160, 96
    call, want, size, n, N, case = _rows_case(op, splits, K, H, 7)
    M = sum(splits)
    for dt in HALF:
        wide = torch.full((M, N + 16), 5.0, dtype=dt, device="cuda")
        out, _ = call(out=wide[:, 8:8 + N])
        _check(out, want, size, n, op)
        assert bool((wide[:, :8] == 5).all()) and bool((wide[:, 8 + N:] == 5).all())
    ro = case[4]
    good = ro.clone()
    for bad in ([-1, 40, 40, 130], [0, 50, 40, 130], [0, 40, 40, 129], [0, 40, 200, 130]):
        ro.copy_(_dev(bad))
        out = torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda")
        _, st = call(out=out)
        assert int(st) == _capi.DEV_BAD_OFFSETS and bool((out == 5).all())
    ro.copy_(good)
    st = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    call(out=out, status=st, noop_flag=torch.ones(1, dtype=torch.int32, device="cuda"))
    assert int(st) == 99 and bool((out == 5).all())
    call(out=out, status=st, noop_flag=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert int(st) == 0
    _check(out, want, size, n, op)


def test_wgrad_status(cuda_device):
    dy, x, sy, sx, ro, cb, want, size = _wgrad_case([40, 0, 90], 96, 160, 8)
    a, b = mg.MXFP8(None, dy, None, sy), mg.MXFP8(None, x, None, sx)
    out = torch.full(want.shape, 5.0, device="cuda")
    for r, c in (([0, 50, 40, 130], cb), (ro, [0, 2, 2, 4]), (ro, [1, 3, 3, 6]), (ro, [0, 2, 3, 6])):
        r = r if isinstance(r, torch.Tensor) else _dev(r)
        c = c if isinstance(c, torch.Tensor) else _dev(c)
        _, st = mg.grouped_mxfp8_wgrad(a, b, r, c, out=out)
        assert int(st) == _capi.DEV_BAD_OFFSETS and bool((out == 5).all())
    # offsets that need more scale rows than there are: 130 single rows
    one = _dev(list(range(131)))
    _, st = mg.grouped_mxfp8_wgrad(a, b, one, one)
    assert int(st) == _capi.DEV_BAD_OFFSETS
    mg.grouped_mxfp8_wgrad(a, b, ro, cb, out=out,
                           noop_flag=torch.ones(1, dtype=torch.int32, device="cuda"))
    assert bool((out == 5).all())


def test_no_rows(cuda_device):
    g = _gen(1)
    ro = _dev([0, 0, 0])
    e = torch.empty((0, 64), dtype=torch.uint8, device="cuda")
    es = torch.empty((0, 2), dtype=torch.uint8, device="cuda")
    w, sw = _codes(g, 128, 64), _scales(g, 128, 2)
    out, st = mg.grouped_mxfp8_gemm(mg.MXFP8(e, None, es, None), mg.MXFP8(w, None, sw, None), ro)
    assert out.shape == (0, 64) and int(st) == 0
    es = torch.empty((0, 64), dtype=torch.uint8, device="cuda")
    dw, st = mg.grouped_mxfp8_wgrad(mg.MXFP8(None, e, None, es), mg.MXFP8(None, e, None, es), ro, ro)
    assert int(st) == 0 and dw.shape == (2, 64, 64) and bool((dw == 0).all())


def test_graph_replay_with_new_rows(cuda_device):
    """A captured product follows the offsets and contents of each replay; two
    graphs and an eager call on another stream do not disturb one another."""
    K, H = 288, 2592
    first, second = [700, 0, 1300, 130], [30, 2000, 99, 1]
    call, want, size, n, _, (a, sa, w, sw, ro) = _rows_case("gemm", first, K, H, 9)
    out = torch.empty((2130, H), dtype=torch.bfloat16, device="cuda")
    dy, x, sy, sx, ro2, cb2, dwant, dsize = _wgrad_case([50, 0, 201], 288, 544, 10)
    dw = torch.empty(dwant.shape, device="cuda")
    ya, xa = mg.MXFP8(None, dy, None, sy), mg.MXFP8(None, x, None, sx)
    call(out=out)
    mg.grouped_mxfp8_wgrad(ya, xa, ro2, cb2, out=dw)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        call(out=out)
    with torch.cuda.graph(g2):
        mg.grouped_mxfp8_wgrad(ya, xa, ro2, cb2, out=dw)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for splits in (first, second):
        offs = _offs(splits)
        ro.copy_(_dev(offs))
        av, wv = ref.values8(a, sa, 1), ref.values8(w, sw, 1).unflatten(0, (4, H)).mT
        want = ref.grouped(lambda e, r: av[r] @ wv[e], offs)
        size = ref.grouped(lambda e, r: av[r].abs() @ wv[e].abs(), offs)
        out.zero_()
        dw.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
            eager, _ = call()
        torch.cuda.synchronize()
        _check(out, want, size, n, splits)
        _check(eager, want, size, n, splits)
        _check(dw, dwant, dsize, 201, "wgrad")


def test_offsets_past_32_bits(cuda_device):
    """Outputs and gradients of more than 2^31 values: the last rows land where
    they belong."""
    g = _gen(14)
    M, K, N = 66049, 32, 33024
    a, sa, w, sw = _codes(g, M, K), _scales(g, M, 1), _codes(g, N, K), _scales(g, N, 1)
    out, _ = mg.grouped_mxfp8_gemm(mg.MXFP8(a, None, sa, None), mg.MXFP8(w, None, sw, None),
                                   _dev([0, M]))
    assert out.numel() > 2 ** 31
    av, wv = ref.values8(a[-300:], sa[-300:], 1), ref.values8(w, sw, 1)
    _check(out[-300:], av @ wv.T, av.abs() @ wv.abs().T, K, "gemm")
    del out, wv
    E, H, K = 3, 32768, 32768
    dy, x = _codes(g, 40, H), _codes(g, 40, K)
    sy, sx = _scales(g, 3, H), _scales(g, 3, K)
    ro, cb = _dev([0, 0, 7, 40]), _dev([0, 0, 1, 3])
    dw, _ = mg.grouped_mxfp8_wgrad(mg.MXFP8(None, dy, None, sy), mg.MXFP8(None, x, None, sx), ro, cb,
                                   out_dtype=torch.bfloat16)
    yv, xv = ref.values8(dy, sy, 0, [0, 0, 7, 40])[7:], ref.values8(x, sx, 0, [0, 0, 7, 40])[7:]
    h = yv[:, -130:]
    _check(dw[2, -130:], h.T @ xv, h.abs().T @ xv.abs(), 33, "wgrad")
    assert bool((dw[0] == 0).all())


def test_most_groups(cuda_device):
    """MAX_GROUPS groups, most of them empty, on one SM and on pairs."""
    E, K, H = _capi.MAX_GROUPS, 64, 32
    splits = [3 if e % 50 == 7 else 0 for e in range(E)]
    for op in ("gemm", "dgrad", "gemm4"):
        call, want, size, n, _, _ = _rows_case(op, splits, K, H, 15)
        out, st = call()
        assert int(st) == 0
        _check(out, want, size, n, op)
    splits[11] = 300000
    call, want, size, n, _, _ = _rows_case("gemm", splits, K, H, 16)
    out, st = call()
    assert int(st) == 0
    _check(out, want, size, n, "many rows")
    dy, x, sy, sx, ro, cb, want, size = _wgrad_case([e % 3 for e in range(E)], 160, 64, 17)
    dw, st = mg.grouped_mxfp8_wgrad(mg.MXFP8(None, dy, None, sy), mg.MXFP8(None, x, None, sx), ro, cb)
    assert int(st) == 0
    _check(dw, want, size, 2, "wgrad")


@pytest.mark.parametrize("pitch_k", [32 * k for k in (1, 2, 3, 4, 7, 8, 12, 15, 16, 20, 24, 31, 32,
                                                      33, 36, 40, 48, 64, 65, 66, 68, 80)])
def test_scale_row_lengths(cuda_device, pitch_k):
    """Every way the rows' scales are copied (rows of 1 to 80 bytes, groups at odd
    rows), single SMs and pairs."""
    for splits, H in (([5, 0, 1, 130, 40], 96), ([1031, 0, 900], 1376)):
        for op in ("gemm", "gemm4"):
            call, want, size, n, _, _ = _rows_case(op, splits, pitch_k, H, pitch_k)
            out, _ = call(out_dtype=torch.float32)
            _check(out, want, size, n, (op, splits, pitch_k))


def test_scales_and_codes_at_the_end_of_their_memory(cuda_device):
    """Rows in the middle of larger buffers, their neighbours NaN: nothing beyond
    the rows' own bytes takes part."""
    M, K, H = 37, 96, 64
    call, want, size, n, _, (a, sa, w, sw, ro) = _rows_case("gemm4", [20, 17], K, H, 18)
    def inside(t):
        flat = torch.full((t.numel() + 512,), 255, dtype=torch.uint8, device="cuda")
        v = flat[256:256 + t.numel()].view(t.shape)
        v.copy_(t)
        return v
    out, _ = mg.grouped_mxfp4_gemm(mg.MXFP4(inside(a), inside(sa)), mg.MXFP4(inside(w), inside(sw)), ro)
    _check(out, want, size, n, "inside")


@pytest.mark.parametrize("rows", [[1], [20, 17], [128, 0, 131], [1030, 0, 901]])
@pytest.mark.parametrize("op", ["gemm", "dgrad", "gemm4"])
def test_odd_scale_rows_at_the_end_of_their_memory(cuda_device, op, rows):
    """Rows of 33 scales, whose last word is the array's in part, with NaN after
    it and before it."""
    K, H = (1408, 1056) if op == "dgrad" else (1056, 1408)
    call, want, size, n, _, (a, sa, w, sw, ro) = _rows_case(op, rows, K, H, 19)
    flat = torch.full((sa.numel() + 512,), 255, dtype=torch.uint8, device="cuda")
    inside = flat[256:256 + sa.numel()].view(sa.shape)
    inside.copy_(sa)
    if op == "gemm4":
        out, _ = mg.grouped_mxfp4_gemm(mg.MXFP4(a, inside), mg.MXFP4(w, sw), ro)
    elif op == "gemm":
        out, _ = mg.grouped_mxfp8_gemm(mg.MXFP8(a, None, inside, None),
                                       mg.MXFP8(w, None, sw, None), ro)
    else:
        out, _ = mg.grouped_mxfp8_dgrad(mg.MXFP8(a, None, inside, None),
                                        mg.MXFP8(None, w, None, sw), ro)
    _check(out, want, size, n, (op, rows))


def test_results_repeat(cuda_device):
    """The same call gives the same bits."""
    call, *_ = _rows_case("dgrad", [700, 0, 1300, 130], 1056, 2592, 11)
    a, b = call()[0], call()[0]
    assert torch.equal(a, b)


def _exact_values(g, *shape):
    """Quarters of at most 15/4: any 32 of them are exact in MXFP8, whichever
    way the blocks run."""
    return (torch.randint(-15, 16, shape, generator=g, device="cuda") / 4).bfloat16()


@pytest.mark.parametrize("splits,K,H", [([5, 0, 33, 1], 96, 160), ([400, 0, 1900, 130], 288, 2592)])
def test_gradients_are_the_products_gradients(cuda_device, splits, K, H):
    """On values that MXFP8 holds exactly: <dOut, A W^T> has the gradients
    dgrad and wgrad give, by the formula and by differences of the product."""
    g = _gen(12)
    E, M, offs = len(splits), sum(splits), _offs(splits)
    x, w, dy = _exact_values(g, M, K), _exact_values(g, E * H, K), _exact_values(g, M, H)
    ro, cb, _ = mg.splits_to_offsets(torch.tensor(splits, device="cuda"), M)
    qx, _ = mg.grouped_mxfp8_quantize(x, ro, cb)
    qy, _ = mg.grouped_mxfp8_quantize(dy, ro, cb)
    qw = mg.mxfp8_quantize(w)
    f32 = dict(out_dtype=torch.float32)
    out, _ = mg.grouped_mxfp8_gemm(qx, qw, ro, **f32)
    dx, _ = mg.grouped_mxfp8_dgrad(qy, qw, ro, **f32)
    dw, _ = mg.grouped_mxfp8_wgrad(qy, qx, ro, cb, **f32)
    xd, wd, yd = x.double(), w.double().unflatten(0, (E, H)), dy.double()
    # sums of sixteenths below 2^15: exact in fp32
    assert torch.equal(out.double(), ref.grouped(lambda e, r: xd[r] @ wd[e].T, offs))
    assert torch.equal(dx.double(), ref.grouped(lambda e, r: yd[r] @ wd[e], offs))
    want = torch.stack([yd[lo:hi].T @ xd[lo:hi] for lo, hi in zip(offs[:-1], offs[1:])])
    assert torch.equal(dw.double(), want)
    # differences: the product is linear, so a step in one entry moves
    # <dOut, out> by exactly the step times the gradient
    row, col = offs[2] + 3, 37
    x2 = x.clone()
    x2[row, col] = 1.25 if x[row, col] != 1.25 else -0.5
    q2, _ = mg.grouped_mxfp8_quantize(x2, ro, cb)
    out2, _ = mg.grouped_mxfp8_gemm(q2, qw, ro, **f32)
    step = (x2[row, col] - x[row, col]).double()
    moved = ((out2.double() - out.double()) * yd).sum()
    assert moved == step * dx[row, col].double()
    w2 = w.clone()
    w2[2 * H + 7, col] = 1.25 if w[2 * H + 7, col] != 1.25 else -0.5
    out3, _ = mg.grouped_mxfp8_gemm(qx, mg.mxfp8_quantize(w2), ro, **f32)
    step = (w2[2 * H + 7, col] - w[2 * H + 7, col]).double()
    assert ((out3.double() - out.double()) * yd).sum() == step * dw[2, 7, col].double()


def test_expert_layer_step(cuda_device):
    """The run of an expert layer's training step: quantize, first product,
    activation, second product, and back, each product against 64-bit forms of
    the operands that the step before it wrote."""
    tokens, hidden, inner = [65, 0, 200, 7], 256, 160
    E, M, offs = len(tokens), sum(tokens), _offs(tokens)
    g = _gen(13)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    x, dout, s = rnd(M, hidden), rnd(M, hidden), torch.rand(M, generator=g, device="cuda")
    w1 = mg.mxfp8_quantize(rnd(E * 2 * inner, hidden) / 16)
    w2 = mg.mxfp8_quantize(rnd(E * hidden, inner) / 16)
    ro, cb, _ = mg.splits_to_offsets(torch.tensor(tokens, device="cuda"), M)
    qx, _ = mg.grouped_mxfp8_quantize(x, ro, cb)
    h, _ = mg.grouped_mxfp8_gemm(qx, w1, ro)
    qa, _ = mg.grouped_scaled_swiglu_mxfp8_fwd(h, s, ro, cb)
    out, _ = mg.grouped_mxfp8_gemm(qa, w2, ro)
    qd, _ = mg.grouped_mxfp8_quantize(dout, ro, cb)
    da, _ = mg.grouped_mxfp8_dgrad(qd, w2, ro)
    dw2, _ = mg.grouped_mxfp8_wgrad(qd, qa, ro, cb)
    bw, _ = mg.grouped_scaled_swiglu_mxfp8_bwd(da, h, s, ro, cb)
    dx, _ = mg.grouped_mxfp8_dgrad(bw.mx, w1, ro)
    dw1, _ = mg.grouped_mxfp8_wgrad(bw.mx, qx, ro, cb)

    def rows(q, w, wdim):
        a = ref.values8(q.row_codes, q.row_scales, 1)
        b = (ref.values8(w.row_codes, w.row_scales, 1) if wdim == 1 else
             ref.values8(w.col_codes, w.col_scales, 0)).unflatten(0, (E, -1))
        b = b.mT if wdim == 1 else b
        return [ref.grouped(lambda e, r: f(a[r]) @ f(b[e]), offs) for f in (lambda t: t, torch.abs)]

    def weights(p, q):
        a, b = (ref.values8(t.col_codes, t.col_scales, 0, offs) for t in (p, q))
        r = [slice(lo, hi) for lo, hi in zip(offs[:-1], offs[1:])]
        return [torch.stack([f(a[i]).T @ f(b[i]) for i in r]) for f in (lambda t: t, torch.abs)]

    _check(h, *rows(qx, w1, 1), hidden, "h")
    _check(out, *rows(qa, w2, 1), inner, "out")
    _check(da, *rows(qd, w2, 0), hidden, "da")
    _check(dx, *rows(bw.mx, w1, 0), 2 * inner, "dx")
    _check(dw2, *weights(qd, qa), 200, "dw2")
    _check(dw1, *weights(bw.mx, qx), 200, "dw1")
    err = ctypes.c_uint32(0)
    _capi.call("moeact_device_error", ctypes.byref(err))
    assert err.value == 0
