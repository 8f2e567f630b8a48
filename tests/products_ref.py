"""Plain 64-bit forms of the block-scaled quantizers and grouped products, for
the tests: from the definitions, on whatever device the tensors are on."""
import torch

E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                    dtype=torch.float64)


def scale_values(b):
    """2^(b - 127), NaN for 255."""
    v = torch.exp2(b.double() - 127)
    return torch.where(b == 255, torch.nan, v)


def values8(codes, scales, dim, offs=None):
    """Values of E4M3 codes [R, C] with scales to every 32 columns (dim 1) or
    32 rows (dim 0; offs: the blocks restart at these row offsets)."""
    v, s = codes.view(torch.float8_e4m3fn).double(), scale_values(scales)
    if dim == 1:
        return v * s.repeat_interleave(32, 1)
    if offs is None:
        return v * s.repeat_interleave(32, 0)[:v.shape[0]]
    at, b = [], 0
    for lo, hi in zip(offs[:-1], offs[1:]):
        at += [b + i // 32 for i in range(hi - lo)]
        b += (hi - lo + 31) // 32
    return v * s[torch.tensor(at, dtype=torch.int64, device=v.device)]


def values4(codes, scales):
    t = E2M1.to(codes.device)
    v = torch.stack([t[(codes & 15).long()], t[(codes >> 4).long()]], 2).flatten(1)
    return v * scale_values(scales).repeat_interleave(32, 1)


def exponent(amax, largest):
    """The E8M0 byte of blocks with these largest magnitudes, by search over
    every e: the smallest with amax <= largest 2^e."""
    e = torch.arange(-127, 128, dtype=torch.float64, device=amax.device)
    fits = amax.double().unsqueeze(-1) <= largest * torch.exp2(e)
    b = torch.where(fits.any(-1), fits.int().argmax(-1), 254)
    return torch.where(amax.isnan(), 255, b).to(torch.uint8)


def nearest_even(v, grid):
    """Index of the nearest entry of an ascending grid; ties to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo = torch.bucketize(v.contiguous(), mid)                       # v <= mid[lo]: ties down
    tie = (lo < len(mid)) & (v == mid[lo.clamp_max(len(mid) - 1)])
    return torch.where(tie & (lo % 2 == 1), lo + 1, lo)


def quantize4(x):
    """(codes, scales) of MXFP4 rows."""
    b = x.double().unflatten(1, (-1, 32))
    s = exponent(b.abs().amax(2), 6.0)
    v = b / scale_values(s).unsqueeze(2)
    m = nearest_even(v.abs().nan_to_num(nan=6.0), E2M1[:8].to(x.device))
    nan = (s == 255).unsqueeze(2)
    c = torch.where(nan, 7, m + 8 * torch.signbit(v).long()).flatten(1).to(torch.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4), s


def tile_scales(s):
    """[R, C] scale matrix (R, C multiples of 128 and 4) in tiles of 128 x 4,
    element (r, c) of a tile at byte (r % 32) 16 + (r // 32) 4 + c."""
    R, C = s.shape
    return s.reshape(R // 128, 4, 32, C // 4, 4).permute(0, 3, 2, 1, 4).reshape(R, C).contiguous()


def tile_col_scales(s, nblocks):
    """Colwise scales [S, W] of groups with these block counts, each group's
    transposed [W, blocks] matrix tiled, groups one after another."""
    out, b = [], 0
    for n in nblocks:
        if n:
            out.append(tile_scales(s[b:b + n].T.contiguous()).reshape(-1))
        b += n
    return torch.cat(out).reshape(s[:b].shape)


def grouped(fn, offs):
    return torch.cat([fn(e, slice(lo, hi)) for e, (lo, hi) in enumerate(zip(offs[:-1], offs[1:]))])
