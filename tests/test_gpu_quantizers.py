"""The plain MXFP8 and MXFP4 quantizers: codes and scales bitwise equal to
64-bit forms written from the definitions."""
import pytest
import torch

import moe_gated_activation_b200 as mg
import products_ref as ref

pytestmark = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _values(M, N, seed):
    """bf16 rows whose blocks span every exponent, with zeros, ties of both
    formats, infinities, NaNs and the lowest value of the type."""
    g = _gen(seed)
    x = torch.randn(M, N, generator=g, device="cuda")
    e = torch.randint(-130, 127, (M, N // 32), generator=g, device="cuda").float()
    x = x * torch.exp2(e).repeat_interleave(32, 1)
    flat = x.view(-1)
    n = flat.numel()
    pick = lambda k: torch.randint(0, n, (max(1, n // k),), generator=g, device="cuda")
    flat[pick(50)] = 0.0
    flat[pick(50)] = -0.0
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -5.0], device="cuda")
    b = x.view(M, N // 32, 32)
    b[:, 0, :9] = ties
    b[:, 0, 9:] = 0.5
    if n > 2000:
        flat[pick(900)] = float("inf")
        flat[pick(900)] = -float("inf")
        flat[pick(1500)] = float("nan")
        flat[pick(900)] = torch.finfo(torch.bfloat16).min
        if M > 3:
            x[3] = 0.0
    return x.bfloat16()


def _quantize8(x, dim):
    """(codes, scales) of MXFP8 from the definition, for rows a multiple of 32
    long (dim 1) or columns padded with zeros to one (dim 0)."""
    t = x if dim == 1 else x.T
    n = t.shape[1]
    t = torch.nn.functional.pad(t.double(), (0, -n % 32)).unflatten(1, (-1, 32))
    s = ref.exponent(t.abs().amax(2), 448.0)
    v = t / ref.scale_values(s).unsqueeze(2)
    grid = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    c = ref.nearest_even(v.abs().nan_to_num(nan=0.0), grid) + 128 * torch.signbit(v).long()
    c = torch.where((s == 255).unsqueeze(2), 0x7F, c).flatten(1)[:, :n].to(torch.uint8)
    return (c, s) if dim == 1 else (c.T, s.T)


SIZES = [(1, 32), (1, 2048), (7, 96), (33, 160), (128, 128), (300, 1056), (130, 288)]


@pytest.mark.parametrize("M,N", SIZES)
def test_mxfp4(cuda_device, M, N):
    x = _values(M, N, 1)
    q = mg.mxfp4_quantize(x)
    codes, scales = ref.quantize4(x)
    assert torch.equal(q.scales, scales)
    assert torch.equal(q.codes, codes)
    back = mg.mxfp4_dequantize(q)
    assert back.dtype == torch.bfloat16
    # exact, but for overflow: bf16 holds every product that fits its range
    want = ref.values4(codes, scales)
    assert torch.equal(back.double().nan_to_num(nan=1e300),
                       want.bfloat16().double().nan_to_num(nan=1e300))
    fine = want.isfinite() & (want.abs() < 2.0 ** 128)
    assert torch.equal(back.double()[fine], want[fine])


def test_mxfp4_every_code_and_scale(cuda_device):
    """The dequantizer on all 16 codes with all 256 scales."""
    codes = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8)
    q = mg.MXFP4(codes.repeat(16).view(256, 16).contiguous(),
                 torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8).view(256, 1))
    want = ref.values4(q.codes, q.scales).bfloat16()
    got = mg.mxfp4_dequantize(q)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))


def test_mxfp4_every_bf16_rounding(cuda_device):
    """Every finite bf16 in [0, 6] next to a 6 (scale one): nearest-even codes."""
    bits = torch.arange(0x40C1, device="cuda", dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16)
    v = torch.cat([v, -v])
    n = -(-v.numel() // 31)
    x = torch.zeros(n * 31, dtype=torch.bfloat16, device="cuda")
    x[:v.numel()] = v
    x = torch.cat([x.view(n, 31), torch.full((n, 1), 6.0, dtype=torch.bfloat16, device="cuda")], 1)
    q = mg.mxfp4_quantize(x)
    codes, scales = ref.quantize4(x)
    assert bool((scales == 127).all())
    assert torch.equal(q.scales, scales) and torch.equal(q.codes, codes)


def test_mxfp4_strided_tiled_and_flagged(cuda_device):
    x = _values(256, 512, 2)
    wide = torch.zeros(256, 1024, dtype=torch.bfloat16, device="cuda")
    wide[:, 16:528] = x
    q = mg.mxfp4_quantize(wide[:, 16:528])
    p = mg.mxfp4_quantize(x)
    assert torch.equal(q.codes, p.codes) and torch.equal(q.scales, p.scales)
    t = mg.mxfp4_quantize(x, gemm_scales=True)
    assert torch.equal(t.codes, p.codes) and torch.equal(t.scales, ref.tile_scales(p.scales))
    out = torch.full((256, 1024), 3.0, dtype=torch.bfloat16, device="cuda")
    mg.mxfp4_dequantize(t, gemm_scales=True, out=out[:, 8:520])
    want = mg.mxfp4_dequantize(p)
    assert torch.equal(out[:, 8:520].nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
    assert bool((out[:, :8] == 3).all()) and bool((out[:, 520:] == 3).all())
    on = torch.ones(1, dtype=torch.int32, device="cuda")
    held = mg.MXFP4(torch.full_like(p.codes, 9), torch.full_like(p.scales, 9))
    got = mg.mxfp4_quantize(x, out=held, noop_flag=on)
    assert got.codes.data_ptr() == held.codes.data_ptr()
    assert bool((held.codes == 9).all()) and bool((held.scales == 9).all())
    on.zero_()
    mg.mxfp4_quantize(x, out=held, noop_flag=on)
    assert torch.equal(held.codes, p.codes) and torch.equal(held.scales, p.scales)


@pytest.mark.parametrize("M,N", SIZES)
def test_mxfp8_dense(cuda_device, M, N):
    x = _values(M, N, 3)
    q = mg.mxfp8_quantize(x)
    for dim, codes, scales in ((1, q.row_codes, q.row_scales), (0, q.col_codes, q.col_scales)):
        c, s = _quantize8(x, dim)
        assert torch.equal(scales, s), dim
        assert torch.equal(codes.view(torch.uint8), c), dim
    one = mg.mxfp8_quantize(x, colwise=False)
    assert torch.equal(one.row_codes.view(torch.uint8), q.row_codes.view(torch.uint8))
    assert one.col_codes.numel() == 0


def test_mxfp8_grouped(cuda_device):
    splits, N = [0, 1, 31, 33, 0, 127, 129, 64], 288
    M = sum(splits)
    x = _values(M, N, 4)
    ro, cb, _ = mg.splits_to_offsets(torch.tensor(splits, device="cuda"), M)
    q, st = mg.grouped_mxfp8_quantize(x, ro, cb, col_scale_rows=int(cb[-1]))
    assert int(st) == 0
    c, s = _quantize8(x, 1)
    assert torch.equal(q.row_codes.view(torch.uint8), c) and torch.equal(q.row_scales, s)
    lo, parts = 0, []
    for m in splits:
        if m:
            parts.append(_quantize8(x[lo:lo + m], 0))
        lo += m
    assert torch.equal(q.col_codes.view(torch.uint8), torch.cat([p[0] for p in parts]))
    assert torch.equal(q.col_scales, torch.cat([p[1] for p in parts]))
    bad = ro.clone()
    bad[1] = 500
    out = mg.MXFP8(*(torch.full_like(t.view(torch.uint8), 9) for t in mg.grouped_mxfp8_quantize(
        x, ro, cb)[0]))
    _, st = mg.grouped_mxfp8_quantize(x, bad, cb, out=out)
    assert int(st) == 3 and all(bool((t == 9).all()) for t in out)


def test_mxfp8_tiled_and_strided(cuda_device):
    splits, N = [128, 0, 256], 256
    M = sum(splits)
    x = _values(M, N, 5)
    wide = torch.zeros(M, 512, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:264] = x
    ro, cb, _ = mg.splits_to_offsets(torch.tensor(splits, device="cuda"), M)
    p, _ = mg.grouped_mxfp8_quantize(x, ro, cb, col_scale_rows=M // 32)
    q, _ = mg.grouped_mxfp8_quantize(wide[:, 8:264], ro, cb, gemm_scales=True,
                                     col_scale_rows=M // 32)
    for a, b in ((p.row_codes, q.row_codes), (p.col_codes, q.col_codes)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(q.row_scales, ref.tile_scales(p.row_scales))
    assert torch.equal(q.col_scales, ref.tile_col_scales(p.col_scales, [m // 32 for m in splits]))


@pytest.mark.parametrize("M,N", SIZES)
def test_mxfp8_rowwise_only(cuda_device, M, N):
    """Rowwise alone: the bits of both directions' rowwise half, dense, grouped,
    strided, under a no-op flag, and nothing at all for bad offsets."""
    x = _values(M, N, 6)
    c, s = _quantize8(x, 1)
    wide = torch.zeros(M, N + 24, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + N] = x
    E = min(M, 5)
    ro, cb, _ = mg.splits_to_offsets(torch.tensor([M - E + 1] + [1] * (E - 1), device="cuda"), M)
    for v in (x, wide[:, 8:8 + N]):
        for q in (mg.mxfp8_quantize(v, colwise=False),
                  mg.grouped_mxfp8_quantize(v, ro, cb, colwise=False)[0]):
            assert torch.equal(q.row_codes.view(torch.uint8), c) and torch.equal(q.row_scales, s)
            assert q.col_codes.numel() == 0 and q.col_scales.numel() == 0
    held = mg.MXFP8(torch.full_like(c, 9), None, torch.full_like(s, 9), None)
    on = torch.ones(1, dtype=torch.int32, device="cuda")
    st = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    mg.grouped_mxfp8_quantize(x, ro, cb, colwise=False, out=held, noop_flag=on, status=st)
    assert int(st) == 99 and bool((held.row_codes == 9).all()) and bool((held.row_scales == 9).all())
    bad = ro.clone()
    bad[-1] += 1
    mg.grouped_mxfp8_quantize(x, bad, cb, colwise=False, out=held, status=st)
    assert int(st) == 3 and bool((held.row_codes == 9).all()) and bool((held.row_scales == 9).all())


def test_mxfp8_rowwise_only_tiled(cuda_device):
    splits, N = [128, 0, 256], 384
    x = _values(sum(splits), N, 7)
    c, s = _quantize8(x, 1)
    ro, cb, _ = mg.splits_to_offsets(torch.tensor(splits, device="cuda"), sum(splits))
    q, st = mg.grouped_mxfp8_quantize(x, ro, cb, colwise=False, gemm_scales=True)
    assert int(st) == 0 and torch.equal(q.row_scales, ref.tile_scales(s))
    assert torch.equal(q.row_codes.view(torch.uint8), c)
    ro2, cb2, _ = mg.splits_to_offsets(torch.tensor([64, 320], device="cuda"), 384)
    _, st = mg.grouped_mxfp8_quantize(x, ro2, cb2, colwise=False, gemm_scales=True)
    assert int(st) == 4


def test_no_rows(cuda_device):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert mg.mxfp8_quantize(x).row_codes.shape == (0, 64)
    q = mg.mxfp4_quantize(x)
    assert q.codes.shape == (0, 32) and mg.mxfp4_dequantize(q).shape == (0, 64)
    z = torch.zeros(3, dtype=torch.int64, device="cuda")
    _, st = mg.grouped_mxfp8_quantize(x, z, z)
    assert int(st) == 0
