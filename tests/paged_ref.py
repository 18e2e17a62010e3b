"""Plain fp64 forms of the paged-cache operators and of the e4m3 LM head, with the error
bounds their tests use.  Everything here is CPU torch."""
import math

import torch

BLOCK = 128
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # relative, finfo.eps / 2
EPS32 = 2.0 ** -24
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ rotary append

def rotate(x, cos, sin, rd, interleaved):
    """(rotated fp64, bound) of x [R, heads, D]; cos, sin [R, rd / 2].

    Bound: two products and a sum in fp32 (3 roundings, at most 2^-24 each of |a c| + |b s|),
    then one rounding to the result's type, added by the caller."""
    x = x.double()
    c, s = cos.double()[:, None], sin.double()[:, None]
    out, bound = x.clone(), torch.zeros_like(x)
    a = slice(0, rd, 2) if interleaved else slice(0, rd // 2)
    b = slice(1, rd, 2) if interleaved else slice(rd // 2, rd)
    xa, xb = x[..., a], x[..., b]
    out[..., a] = xa * c - xb * s
    out[..., b] = xb * c + xa * s
    bound[..., a] = 3 * EPS32 * ((xa * c).abs() + (xb * s).abs())
    bound[..., b] = 3 * EPS32 * ((xb * c).abs() + (xa * s).abs())
    return out, bound


# ------------------------------------------------------------------ paged attention

def visible(parents):
    """[N, N] truth: node j is node i or one of its ancestors (a link that does not point to
    an earlier node ends the chain)."""
    n = len(parents)
    see = torch.zeros((n, n), dtype=torch.bool)
    for i in range(n):
        a = i
        while a >= 0:
            see[i, a] = True
            up = int(parents[a])
            a = up if 0 <= up < a else -1
    return see


def gather(pool, table_row, length, g):
    """The first `length` rows of kv head g of one sequence, fp64; rows of a page outside the
    pool are zero."""
    page = pool.shape[2]
    out = torch.zeros((length, pool.shape[3]), dtype=torch.float64)
    for p0 in range(0, length, page):
        n = min(page, length - p0)
        idx = int(table_row[p0 // page])
        if 0 <= idx < pool.shape[0]:
            out[p0:p0 + n] = pool[idx, g, :n].double()
    return out


def attention(q, k_pages, v_pages, table, lens, k_tree, v_tree, parents, scale, dtype):
    """(fp64 output, bound) of paged tree attention.

    Bound, per output element, with A = sum of w |v| over the row's keys:
      scores: a D-long fp32 sum is off by at most (D + 4) 2^-24 of sum |q k|, which moves a
        weight by that relative amount (es), in the numerator and in the denominator;
      bf16 only: a weight is rounded to bf16 for its product with V (2^-8), and 2^x of some
        weights comes from a polynomial within 1.1e-4, in numerator and denominator;
      exponents: x c - m in fp32 is off by 4 2^-24 |x c| (in es), ex2 itself by 2^-22;
      sums over n keys: n 2^-24 in each;
      one rounding of the result."""
    b_, n_, hq, d = q.shape
    hkv = k_pages.shape[1]
    group = hq // hkv
    out = torch.zeros(q.shape, dtype=torch.float64)
    bound = torch.zeros(q.shape, dtype=torch.float64)
    for b in range(b_):
        L = int(lens[b])
        see = torch.cat([torch.ones((n_, L), dtype=torch.bool), visible(parents[b].tolist())], dim=1)
        for g in range(hkv):
            k = torch.cat([gather(k_pages, table[b], L, g), k_tree[b, :, g].double()])
            v = torch.cat([gather(v_pages, table[b], L, g), v_tree[b, :, g].double()])
            qh = q[b, :, g * group:(g + 1) * group].double()
            score = torch.einsum("ngd,kd->ngk", qh, k) * scale
            mag = torch.einsum("ngd,kd->ngk", qh.abs(), k.abs()) * scale
            score = score.masked_fill(~see[:, None], -math.inf)
            w = torch.softmax(score, dim=-1)
            o = torch.einsum("ngk,kd->ngd", w, v)
            a = torch.einsum("ngk,kd->ngd", w, v.abs())
            es = ((d + 8) * EPS32 * mag * see[:, None]).amax(dim=-1, keepdim=True)
            rel = 2 * es + 2 * (2.0 ** -22 + (see.shape[1] + 64) * EPS32)
            if dtype == "bf16":
                rel = rel + 2.0 ** -8 + 2 * 1.1e-4
            out[b, :, g * group:(g + 1) * group] = o
            bound[b, :, g * group:(g + 1) * group] = rel * a + HALF_STEP[dtype] * (o.abs() + rel * a)
    return out, bound


# ------------------------------------------------------------------ e4m3 LM head

def block_scale(amax):
    """2^e with the smallest e >= -126 for which amax <= 448 * 2^e."""
    e = torch.full_like(amax, -126.0)
    nz = amax > 0
    e[nz] = torch.ceil(torch.log2(amax[nz] / 448.0)).clamp(min=-126)
    # log2 and ceil are exact enough to be one off at a border: settle it by the definition
    e = torch.where((e > -126) & (amax <= 448.0 * torch.exp2(e - 1)), e - 1, e)
    e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
    return torch.exp2(e)


def quantize(x, block_rows):
    """(e4m3 values, scales [row blocks, column blocks]) in blocks of block_rows x 128."""
    x = x.double()
    r, h = x.shape
    rb, kb = -(-r // block_rows), -(-h // BLOCK)
    pad = torch.nn.functional.pad(x, (0, kb * BLOCK - h, 0, rb * block_rows - r))
    pad = pad.view(rb, block_rows, kb, BLOCK)
    scale = block_scale(pad.abs().amax(dim=(1, 3)))
    q = (pad / scale[:, None, :, None]).view(rb * block_rows, kb * BLOCK)[:r, :h]
    return q.float().to(torch.float8_e4m3fn), scale  # the quotient is exact


def logits_scaled(x8, xs, w8, ws):
    """(fp64 logits, bound) of x8 [R, H], xs [KB, >= R], w8 [V, H], ws [VB, KB].

    Bound: each of the H products is exact in fp32; H + 4 KB additions, products and scalings
    lose at most 2^-23 each of the sum of magnitudes."""
    r, h = x8.shape
    v = w8.shape[0]
    kb = -(-h // BLOCK)
    x = x8.float().double() * xs[:, :r].double().t().repeat_interleave(BLOCK, 1)[:, :h]
    w = w8.float().double() * ws.double().repeat_interleave(BLOCK, 0)[:v].repeat_interleave(BLOCK, 1)[:, :h]
    return x @ w.t(), (h + 4 * kb) * 2.0 ** -23 * (x.abs() @ w.abs().t())
