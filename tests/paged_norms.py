"""Error limits of paged attention in sums of squares, tight enough that one lost tile of keys
or one operand without its low part shows, however long the cache is.  Any device."""
import math

import torch

from paged_helpers import half_step, least_step


def attention64(q, k, v, p, lost=None, q_low=True):
    """Attention of q [n, H, D] at positions p.. over k, v [Hkv, L, D] in 64 bits: (o, spread,
    size) with spread [n, H] = sqrt(sum_j w_j^2 |v_j|^2) and size [n, H] = the root mean square,
    under the same squares, of a key's sum_d |q_d k_d| / sqrt D.  lost: a slice of keys left out; q_low False: q and k rounded to TF32's 11 bits."""
    n, H, D = q.shape
    Hkv, L, _ = k.shape
    if not q_low:
        q, k = (tf32(x) for x in (q, k))
    q = q.double().view(n, Hkv, H // Hkv, D)
    k, v = k.double(), v.double()
    s = torch.einsum("tged,gld->gtel", q, k) / math.sqrt(D)
    size = torch.einsum("tged,gld->gtel", q.abs(), k.abs()) / math.sqrt(D)
    far = torch.arange(L, device=q.device)[None] > (p + torch.arange(n, device=q.device))[:, None]
    s = s.masked_fill(far[None, :, None], -math.inf)
    if lost is not None:
        s[..., lost] = -math.inf
    w = torch.softmax(s, -1)
    o = torch.einsum("gtel,gld->tged", w, v).reshape(n, H, D)
    squares = w.square_() * (v * v).sum(-1)[:, None, None]
    spread = squares.sum(-1).sqrt()
    size = (squares * size.square_()).sum(-1).sqrt() / spread
    return o, *(x.permute(1, 0, 2).reshape(n, H) for x in (spread, size))


def tf32(x):
    bits = x.float().contiguous().view(torch.int32)
    return ((bits + 0x1000) & -0x2000).view(torch.float32)


def norm_limit(o, spread, size, L, dtype, weights):
    """What the 2-norm over D of a (row, head)'s error may be.  weights: the largest relative
    error of a weight's own rounding before the product with v."""
    f32 = dtype == torch.float32
    D = o.shape[-1]
    u = half_step(dtype)
    # Scores: a sum of D products in D / 8 steps (the tensor cores truncate each: 2^-23 of a
    # partial sum, `size` at most), the sum of the small products and its addition; float32's
    # three TF32 products leave 2^-21 of a product; the exponent's rounding, and ex2's 2^-22.
    ds = size * ((D / 8 + 3) * 2.0 ** -23 + (2.0 ** -21 if f32 else 0)) + 2.0 ** -22
    # Weights times v: in 16 bits L / 16 truncated additions to one accumulator, twice as many
    # for weights in two parts; in float32 twelve a tile, then one rounded addition a tile (roundings of either sign: the root of
    # their number), and the product's 2^-21.  The sum of the weights: rounded additions.
    dv = (12 * 2.0 ** -23 + 2.0 ** -21 + math.sqrt(L / 16) * 2.0 ** -24 if f32 else L / 8 * 2.0 ** -23)
    dv += math.sqrt(L) * 2.0 ** -24 + 8 * 2.0 ** -24
    # An error e_j of weight j moves o by w_j e_j (v_j - o).  Errors of different weights are
    # independent of each other and of v: the squares add up, mean square a third of the
    # largest at most, twice the root of the sum is far behind it; equal weights have equal
    # errors, which move o by e |o| at most.
    norm = o.norm(dim=-1)
    return u * norm + least_step(dtype) * math.sqrt(D) + \
        2 * (ds + dv) * (spread + norm) + weights * (2 * spread + norm)


def worst(got, o, limit):
    """Largest error norm over its limit (NaN counts as infinite)."""
    e = (got.double() - o).norm(dim=-1) / limit
    return float(torch.nan_to_num(e, nan=math.inf).max())


def weight_rounding(dtype, chunk):
    """16-bit chunks round each weight to the type; decode steps hold it in two parts, so that a
    rounding of what the first leaves is left; float32 splits it (counted with the product)."""
    if dtype == torch.float32:
        return 0.0
    u = half_step(dtype)
    return u if chunk else u * u


def check_norms(b, out, where=""):
    """A Paged batch's rows within the limits, row by row and head by head."""
    assert int(b.status.item()) == 0, where
    chunk = max(b.n) * (b.H // b.Hkv) > 16
    far = 0.0
    for i, (n, p) in enumerate(zip(b.n, b.p)):
        if n == 0:
            continue
        a = int(b.offsets_host[i])
        o, spread, size = attention64(b.q[a:a + n], b.k[i], b.v[i], p)
        far = max(far, worst(out[a:a + n], o, norm_limit(o, spread, size, n + p, b.dtype, weight_rounding(b.dtype, chunk))))
    assert far <= 1, f"{where}: {far:.3g} times the limit"
    return far
