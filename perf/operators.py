"""The block-scaled quantisers and the products grouped by expert: what is timed and
compared, and their plain forms in elementary torch operations.

Operators (``own`` true: the package's entry points):
  quantize8   MXFP8 of bf16 rows, blocks of 32 along the row and / or down an
              expert's rows (``grouped_mxfp8_quantize``)
  quantize4   MXFP4 of bf16 rows and the values it stands for
              (``mxfp4_quantize``, ``mxfp4_dequantize``)
  gemm        out[i] = A[i] W_e^T for the rows of each expert, MXFP8
              (``grouped_mxfp8_gemm``)
  dgrad       its gradient by A: dA[i] = dOut[i] W_e (``grouped_mxfp8_dgrad``)
  wgrad       its gradient by W: dW_e = dOut_e^T A_e (``grouped_mxfp8_wgrad``)
  gemm4       gemm with MXFP4 operands (``grouped_mxfp4_gemm``)
"""
import math
import random

import numpy as np
import torch

own = False

CHUNK = 1 << 26   # values that a preparation works on at a time


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # decoding: 8 tokens sent to their top 8 of 128 experts, hidden size
        # 2048, quantised once for the experts' first product
        {"name": "quantize8 decode", "op": "quantize8", "rows": 64, "cols": 2048, "experts": 128,
         "active": 50, "skew": 0.0, "dirs": "row"},
        # a training step's dispatched tokens, 8192 x top 8, both directions
        # (the first product and its weight gradient)
        {"name": "quantize8 train", "op": "quantize8", "rows": 65536, "cols": 2048,
         "experts": 128, "active": 103, "skew": 0.5, "dirs": "both"},
        # one token's activations
        {"name": "quantize4 one token", "op": "quantize4", "rows": 1, "cols": 2048},
        # the largest activation of one expert group, outliers included
        {"name": "quantize4 prompt", "op": "quantize4", "rows": 16384, "cols": 7168},
        # decoding through the experts' gate and up projection
        {"name": "gemm decode", "op": "gemm", "rows": 64, "k": 2048, "h": 1536, "experts": 128,
         "active": 50, "skew": 0.0, "out": "bf16"},
        # a training step's gate and up projection, 8192 tokens x top 8, ragged
        {"name": "gemm train", "op": "gemm", "rows": 65536, "k": 2048, "h": 1536,
         "experts": 128, "active": 103, "skew": 0.5, "out": "bf16"},
        # the down projection of 32 wide experts under a Zipf-like router: the largest
        {"name": "gemm wide", "op": "gemm", "rows": 131072, "k": 8192, "h": 2048, "experts": 32,
         "active": 32, "skew": 1.1, "out": "bf16"},
        # the gradient by the rows of the training step's gate and up projection
        {"name": "dgrad train", "op": "dgrad", "rows": 65536, "k": 2048, "h": 1536,
         "experts": 128, "active": 103, "skew": 0.5, "out": "bf16"},
        # its gradient by the weights, kept in 32 bits for accumulation
        {"name": "wgrad train", "op": "wgrad", "rows": 65536, "k": 2048, "h": 1536,
         "experts": 128, "active": 103, "skew": 0.5, "out": "fp32"},
        # a short ragged micro-batch of a down projection, gradients in 16 bits
        {"name": "wgrad short", "op": "wgrad", "rows": 1999, "k": 768, "h": 2048, "experts": 32,
         "active": 29, "skew": 0.5, "out": "bf16"},
        # decoding through the down projection with 4-bit weights and activations
        {"name": "gemm4 decode", "op": "gemm4", "rows": 64, "k": 768, "h": 2048, "experts": 128,
         "active": 50, "skew": 0.0, "out": "bf16"},
        # a prompt batch through the same experts' gate and up projection
        {"name": "gemm4 prompt", "op": "gemm4", "rows": 65536, "k": 2048, "h": 1536,
         "experts": 128, "active": 103, "skew": 0.5, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["quantize8", "quantize4", "gemm", "dgrad", "wgrad", "gemm4"])
    if op == "quantize4":
        return {"op": op, "rows": _log(rng, 1, 16384), "cols": 32 * _log(rng, 2, 224)}
    experts = _log(rng, 1, 128)
    active = rng.randint(max(1, experts // 3), experts)
    rows = max(active, _log(rng, 1, 65536))
    skew = rng.choice([0.0, 0.5, 1.1])
    if op == "quantize8":
        return {"op": op, "rows": rows, "cols": 32 * _log(rng, 2, 128), "experts": experts,
                "active": active, "skew": skew, "dirs": rng.choice(["row", "col", "both"])}
    k, h = 32 * _log(rng, 4, 128), 32 * _log(rng, 4, 128)
    # the weights and the products no larger than the largest listed case's
    while experts * k * h > 512 << 20 or rows * k * h > 131072 * 8192 * 2048:
        k, h = max(32, k // 64 * 32), max(32, h // 64 * 32)
    return {"op": op, "rows": rows, "k": k, "h": h, "experts": experts, "active": active,
            "skew": skew, "out": rng.choice(["bf16", "bf16", "fp32"])}


def work(case):
    M, op = case["rows"], case["op"]
    if op == "quantize8":
        W = case["cols"]
        blocks = M / 32 + case["active"] / 2       # an expert's last block is half full
        per_row = M * W * 33 / 32
        per_col = M * W + blocks * W
        n = {"row": per_row, "col": per_col, "both": per_row + per_col}[case["dirs"]]
        return {"bytes": 2 * M * W + n, "flops": 4 * M * W}
    if op == "quantize4":
        W = case["cols"]
        # the rows in, the codes and scales out; and these in, the values out
        return {"bytes": 2 * M * W + 2 * (M * W * 17 / 32) + 2 * M * W, "flops": 5 * M * W}
    K, H, E, act = case["k"], case["h"], case["experts"], case["active"]
    width = 2 if case["out"] == "bf16" else 4
    per = 17 / 32 if op == "gemm4" else 33 / 32
    if op == "wgrad":
        nbytes = M * (K + H) * per + E * H * K * width
    else:
        nin, nout = (H, K) if op == "dgrad" else (K, H)
        nbytes = M * nin * per + act * H * K * per + M * nout * width
    return {"bytes": nbytes, "flops": 2 * M * K * H}


# ---------------------------------------------------------------- the inputs
def _splits(case, seed):
    """Rows of each expert: `active` of the experts get one row at least, the
    rest by weights (i + 1)^-skew; the others get none.  The counts go with the
    case, so that outputs of every seed have the same shapes; which expert has
    which count goes with the seed."""
    E, act, M = case["experts"], case["active"], case["rows"]
    p = (1.0 + np.arange(act)) ** -case["skew"]
    got = np.zeros(E, dtype=np.int64)
    got[:act] = 1 + np.random.default_rng([E, act, M]).multinomial(M - act, p / p.sum())
    return np.random.default_rng(seed).permutation(got)


def _normal(gen, rows, cols, std=1.0, outliers=False):
    """bf16 rows of N(0, std^2), with outliers one value in a thousand a hundredfold."""
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    step = max(1, CHUNK // cols)
    for lo in range(0, rows, step):
        x = torch.randn(min(step, rows - lo), cols, generator=gen, device="cuda") * std
        if outliers:
            x = torch.where(torch.rand(x.shape, generator=gen, device="cuda") < 1e-3, 100 * x, x)
        out[lo:lo + step] = x
    return out


def _blocks(case, offs):
    """Where each row stands when every expert's rows start a new block of 32."""
    splits = np.diff(offs)
    starts = np.concatenate([[0], np.cumsum((splits + 31) // 32)])
    at = np.repeat(32 * starts[:-1] - offs[:-1], splits) + np.arange(offs[-1])
    return torch.from_numpy(starts).cuda(), torch.from_numpy(at).cuda()


def _rows_in_chunks(fn, x):
    """fn (rows -> codes, scales) over pieces of x, a multiple of 32 rows each."""
    step = max(32, CHUNK // x.shape[1] // 32 * 32)
    parts = [fn(x[lo:lo + step]) for lo in range(0, x.shape[0], step)]
    return tuple(torch.cat(p) for p in zip(*parts))


def prepare(case, seed):
    op, M = case["op"], case["rows"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if op == "quantize4":
        return {"case": case, "x": _normal(gen, M, case["cols"], math.sqrt(2.0), True)}
    offs = np.concatenate([[0], np.cumsum(_splits(case, seed))])
    starts, at = _blocks(case, offs)
    st = {"case": case, "offs": [int(v) for v in offs], "row_offs": torch.from_numpy(offs).cuda(),
          "colblk_offs": starts, "at": at, "blocks": int(starts[-1])}
    if op == "quantize8":
        st["x"] = _normal(gen, M, case["cols"])
        return st
    K, H, E = case["k"], case["h"], case["experts"]
    if op == "wgrad":
        for name, width in (("dy", H), ("x", K)):
            rows = torch.zeros(32 * st["blocks"], width, dtype=torch.bfloat16, device="cuda")
            rows[at] = _normal(gen, M, width)
            codes, scales = _rows_in_chunks(_colwise8, rows)
            st[name] = (codes[at], scales)
        return st
    four = op == "gemm4"
    a = _normal(gen, M, H if op == "dgrad" else K)
    w = _normal(gen, E * H, K, K ** -0.5)
    st["a"] = _rows_in_chunks(_rowwise4 if four else _rowwise8, a)
    st["w"] = _rows_in_chunks(_rowwise4 if four else _colwise8 if op == "dgrad" else _rowwise8, w)
    return st


# ---------------------------------------------------------------- plain forms
def _exponent(amax, top, over):
    """The E8M0 byte of a block: 127 + the smallest e in [-127, 127] with
    amax <= top 2^over 2^e, top in [0.5, 1); 254 for infinity, 255 for NaN."""
    m, x = torch.frexp(amax)
    e = torch.clamp(x - over + (m > top), -127, 127)
    e = torch.where(amax == 0, -127, torch.where(amax == math.inf, 127, e)) + 127
    return torch.where(amax.isnan(), 255, e).to(torch.uint8)


def _scaled(blocks, dim, top, over):
    """(the blocks over their scales, the scales' bytes), in 32 bits."""
    b = _exponent(blocks.abs().amax(dim), top, over)
    s = torch.where(b == 255, math.nan, torch.ldexp(torch.ones_like(b, dtype=torch.float32),
                                                    127 - b.int()))
    return blocks * s.unsqueeze(dim), b


def _codes8(v):
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _rowwise8(x):
    v, b = _scaled(x.float().unflatten(1, (-1, 32)), 2, 0.875, 9)
    return _codes8(v).flatten(1), b


def _colwise8(x):
    """Blocks of 32 rows; the rows are a multiple of 32."""
    v, b = _scaled(x.float().unflatten(0, (-1, 32)), 1, 0.875, 9)
    return _codes8(v).flatten(0, 1), b


def _rowwise4(x):
    """Two 4-bit codes to a byte, the even column's in the low half."""
    v, b = _scaled(x.float().unflatten(1, (-1, 32)), 2, 0.75, 3)
    m = v.abs().nan_to_num(nan=6.0)
    c = ((m > 0.25).byte() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5)
         + (m > 5.0) + 8 * (torch.signbit(v) & ~v.isnan()).byte())
    c = c.flatten(1)
    return c[:, 0::2] | (c[:, 1::2] << 4), b


def _scale_values(b):
    return b.view(torch.float8_e8m0fnu).float()


def _values8(codes, scales, at=None):
    """fp32 values of codes with a scale to every 32 of a row (`at` None) or
    to every 32 of the rows at the places `at`."""
    if at is None:
        v = codes.float().unflatten(1, (-1, 32)) * _scale_values(scales).unsqueeze(2)
        return v.flatten(1)
    return codes.float() * _scale_values(scales)[at // 32]


def _values4(codes, scales):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                         device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], 2).flatten(1).int()
    v = table[c].unflatten(1, (-1, 32)) * _scale_values(scales).unsqueeze(2)
    return v.flatten(1)


def _e8m0(scales):
    return scales.view(torch.float8_e8m0fnu)


def _spans(offs):
    return list(zip(offs[:-1], offs[1:]))


_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "quantize8":
        out = {}
        if case["dirs"] != "col":
            codes, scales = _rowwise8(st["x"])
            out["row_codes"], out["row_scales"] = codes, _e8m0(scales)
        if case["dirs"] != "row":
            x, at = st["x"], st["at"]
            rows = torch.zeros(32 * st["blocks"], x.shape[1], dtype=x.dtype, device=x.device)
            rows[at] = x
            codes, scales = _colwise8(rows)
            out["col_codes"], out["col_scales"] = codes[at], _e8m0(scales)
        return out
    if op == "quantize4":
        codes, scales = _rowwise4(st["x"])
        return {"values": _values4(codes, scales).bfloat16(), "scales": _e8m0(scales)}
    dt = _DTYPES[case["out"]]
    spans = _spans(st["offs"])
    if op == "wgrad":
        dy, x = _values8(*st["dy"], st["at"]), _values8(*st["x"], st["at"])
        return torch.stack([(dy[lo:hi].T @ x[lo:hi]).to(dt) for lo, hi in spans])
    E, H = case["experts"], case["h"]
    who = [e for e, (lo, hi) in enumerate(spans) if hi > lo]   # only their weights are read
    codes, scales = (t.unflatten(0, (E, -1))[who].flatten(0, 1) for t in st["w"])
    if op == "gemm4":
        a, w = _values4(*st["a"]), _values4(codes, scales)
    elif op == "dgrad":
        a, w = _values8(*st["a"]), _values8(codes, scales, torch.arange(len(codes), device="cuda"))
    else:
        a, w = _values8(*st["a"]), _values8(codes, scales)
    w = w.unflatten(0, (-1, H)) if op == "dgrad" else w.unflatten(0, (-1, H)).mT
    return torch.cat([(a[slice(*spans[e])] @ w[i]).to(dt) for i, e in enumerate(who)])


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return _framework(state)
    return _plain(state)


def _framework(st):
    import moe_gated_activation_b200 as mg
    case = st["case"]
    op = case["op"]
    if op == "quantize8":
        d = case["dirs"]
        q, _ = mg.grouped_mxfp8_quantize(st["x"], st["row_offs"], st["colblk_offs"],
                                         rowwise=d != "col", colwise=d != "row",
                                         col_scale_rows=st["blocks"])
        out = {}
        if d != "col":
            out["row_codes"], out["row_scales"] = q.row_codes, _e8m0(q.row_scales)
        if d != "row":
            out["col_codes"], out["col_scales"] = q.col_codes, _e8m0(q.col_scales)
        return out
    if op == "quantize4":
        q = mg.mxfp4_quantize(st["x"])
        return {"values": mg.mxfp4_dequantize(q), "scales": _e8m0(q.scales)}
    dt = _DTYPES[case["out"]]
    if op == "wgrad":
        (dyc, dys), (xc, xs) = st["dy"], st["x"]
        dw, _ = mg.grouped_mxfp8_wgrad(mg.MXFP8(None, dyc, None, dys), mg.MXFP8(None, xc, None, xs),
                                       st["row_offs"], st["colblk_offs"], out_dtype=dt)
        return dw
    (ac, asc), (wc, ws) = st["a"], st["w"]
    if op == "gemm4":
        out, _ = mg.grouped_mxfp4_gemm(mg.MXFP4(ac, asc), mg.MXFP4(wc, ws), st["row_offs"],
                                       out_dtype=dt)
    elif op == "dgrad":
        out, _ = mg.grouped_mxfp8_dgrad(mg.MXFP8(ac, None, asc, None),
                                        mg.MXFP8(None, wc, None, ws), st["row_offs"],
                                        out_dtype=dt)
    else:
        out, _ = mg.grouped_mxfp8_gemm(mg.MXFP8(ac, None, asc, None),
                                       mg.MXFP8(wc, None, ws, None), st["row_offs"],
                                       out_dtype=dt)
    return out


# ---------------------------------------------------------------- 64 bits
def _exact_block(x, largest):
    """From the definition, in 64 bits: scales 2^e, e the smallest integer in
    [-127, 127] with max |x| <= largest 2^e, over the last axis."""
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(amax.clamp_min(2.0 ** -140) / largest))
    # the logarithm's own rounding, next to a power of two
    e = torch.where(amax <= largest * torch.exp2(e - 1), e - 1, e)
    e = torch.where(amax > largest * torch.exp2(e), e + 1, e)
    return torch.exp2(e.clamp(-127, 127))


def _exact_round(v, bits, lowest, largest):
    """The nearest number with `bits` bits after the point and an exponent of
    at least `lowest`, ties to even."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -60)))
    e = torch.where(v.abs() >= torch.exp2(e + 1), e + 1, e)
    e = torch.where(v.abs() < torch.exp2(e), e - 1, e).clamp_min(lowest)
    step = torch.exp2(e - bits)
    return (torch.round(v / step) * step).clamp(-largest, largest)


def _exact_codes(x, four):
    largest = 6.0 if four else 448.0
    s = _exact_block(x, largest)
    return _exact_round(x / s, *((1, 0) if four else (3, -6)), largest), s.squeeze(-1)


def _in_pieces(fn, x):
    step = max(32, (CHUNK >> 1) // x.shape[1] // 32 * 32)
    parts = [fn(x[lo:lo + step]) for lo in range(0, x.shape[0], step)]
    return tuple(torch.cat(p) for p in zip(*parts))


def _exact_rows(x, four):
    def piece(p):
        c, s = _exact_codes(p.double().reshape(p.shape[0], -1, 32), four)
        return c.reshape(p.shape[0], -1), s
    return _in_pieces(piece, x)


def _exact_cols(x):
    """Blocks of 32 rows, the rows a multiple of 32."""
    def piece(p):
        c, s = _exact_codes(p.double().reshape(-1, 32, p.shape[1]).transpose(1, 2), False)
        return c.transpose(1, 2).reshape(p.shape), s
    return _in_pieces(piece, x)


def _power(b):
    return torch.exp2(b.double() - 127)


def _exact4(codes, scales):
    def value(c):
        m, x = (c & 1).double(), ((c >> 1) & 3).double()
        v = torch.where(x == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(x - 1))
        return torch.where(c >= 8, -v, v)
    v = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    v[:, 0::2], v[:, 1::2] = value(codes % 16), value(codes // 16)
    return v * _power(scales).repeat_interleave(32, 1)


def exact(case, seed):
    st = prepare(case, seed)
    op, offs = case["op"], st["offs"] if "offs" in st else None
    if op == "quantize4":
        c, s = _exact_rows(st["x"], True)
        return {"values": c * s.repeat_interleave(32, 1), "scales": s}
    if op == "quantize8":
        out, x = {}, st["x"]
        if case["dirs"] != "col":
            out["row_codes"], out["row_scales"] = _exact_rows(x, False)
        if case["dirs"] != "row":
            codes, scales = [], []
            for lo, hi in zip(offs[:-1], offs[1:]):
                if hi > lo:
                    p = torch.nn.functional.pad(x[lo:hi], (0, 0, 0, -(hi - lo) % 32))
                    c, s = _exact_cols(p)
                    codes.append(c[:hi - lo])
                    scales.append(s)
            out["col_codes"], out["col_scales"] = torch.cat(codes), torch.cat(scales)
        return out
    E, H, K = case["experts"], case["h"], case["k"]
    parts = []
    for e in range(E):
        lo, hi = offs[e], offs[e + 1]
        if op == "wgrad":
            b0, b1 = int(st["colblk_offs"][e]), int(st["colblk_offs"][e + 1])
            ops = [c[lo:hi].double() * _power(s[b0:b1]).repeat_interleave(32, 0)[:hi - lo]
                   for c, s in (st["dy"], st["x"])]
            parts.append((ops[0].T @ ops[1]).to(torch.float32 if E * H * K > 1 << 28
                                                else torch.float64))
            continue
        (ac, asc), (wc, ws) = st["a"], st["w"]
        if hi == lo:
            continue
        if op == "gemm4":
            a = _exact4(ac[lo:hi], asc[lo:hi])
            parts.append(a @ _exact4(wc[e * H:(e + 1) * H], ws[e * H:(e + 1) * H]).T)
            continue
        a = ac[lo:hi].double() * _power(asc[lo:hi]).repeat_interleave(32, 1)
        w = wc[e * H:(e + 1) * H].double()
        if op == "dgrad":
            parts.append(a @ (w * _power(ws[e * H // 32:(e + 1) * H // 32]).repeat_interleave(32, 0)))
        else:
            parts.append(a @ (w * _power(ws[e * H:(e + 1) * H]).repeat_interleave(32, 1)).T)
    return torch.stack(parts) if op == "wgrad" else torch.cat(parts)
