"""The 4-bit cache restated for the tests: the layout of its pages byte by
byte, the quantiser's definition, and attention in 64 bits."""
import math

import numpy as np
import torch

ORDER = (0, 2, 4, 6, 1, 3, 5, 7)  # element of a word held by nibble 0, 1, ..., 7
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # of a rounding, relative


def quantise(x):
    """Codes (uint8), scale and zero (fp32 values of x's type) of rows x [.., D]."""
    T = x.dtype
    f = x.float()
    zero, top = f.amin(-1), f.amax(-1)
    scale = ((top - zero) / 15).to(T).float()
    fine = torch.isfinite(f).all(-1) & torch.isfinite(scale)
    q = (f - zero[..., None]) / scale[..., None]
    codes = torch.where((scale[..., None] > 0) & fine[..., None], q, torch.zeros_like(q))
    codes = torch.nan_to_num(codes, 0.0).round().clamp(0, 15).to(torch.uint8)
    return codes, torch.where(fine, scale, torch.nan), torch.where(fine, zero, 0.0)


def pack_words(codes):
    """[.., rows, 8 m] codes to [.., rows, 4 m] bytes."""
    w = codes.reshape(*codes.shape[:-1], -1, 8)[..., list(ORDER)]
    b = w[..., 0::2] | (w[..., 1::2] << 4)
    return b.reshape(*codes.shape[:-1], -1)


def unpack_words(raw):
    n = torch.stack((raw & 15, raw >> 4), -1).reshape(*raw.shape[:-1], -1, 8)
    c = torch.empty_like(n)
    c[..., list(ORDER)] = n
    return c.reshape(*raw.shape[:-1], -1)


class Pages:
    """A cache's contents as codes and parameters, page by page and token by token (on the CPU)."""

    def __init__(self, num, heads, page, D, T):
        self.num, self.heads, self.page, self.D, self.T = num, heads, page, D, T
        self.codes = [torch.zeros((num, heads, page, D), dtype=torch.uint8) for _ in range(2)]
        self.params = [torch.zeros((num, heads, page, 2), dtype=T) for _ in range(2)]  # (scale, zero)

    def random(self, g):
        for i in range(2):
            self.codes[i] = torch.randint(0, 16, self.codes[i].shape, generator=g, dtype=torch.uint8)
            s = 0.25 * torch.exp(0.4 * torch.randn(self.params[i].shape[:-1], generator=g))
            z = -7.5 * s + 0.5 * torch.randn(s.shape, generator=g)
            self.params[i] = torch.stack((s, z), -1).to(self.T)
        return self

    def bytes(self):
        """The uint8 tensor [num, heads, page * (D + 8)] the library takes."""
        t = min(self.page, 64)
        parts = []
        for i in range(2):
            c = self.codes[i].reshape(self.num, self.heads, -1, t, self.D)
            c = pack_words(c if i == 0 else c.transpose(-1, -2).contiguous()).flatten(-2)
            p = self.params[i].reshape(self.num, self.heads, -1, t * 2).contiguous().view(torch.uint8)
            parts += [c, p]
        return torch.cat(parts, -1).reshape(self.num, self.heads, -1).contiguous()

    @classmethod
    def of(cls, raw, page, D, T):
        """Read back from the library's bytes."""
        raw = raw.cpu()
        self = cls(raw.shape[0], raw.shape[1], page, D, T)
        t = min(page, 64)
        x = raw.reshape(raw.shape[0], raw.shape[1], page // t, t * (D + 8))
        half = t * (D + 8) // 2
        for i in range(2):
            y = x[..., i * half:(i + 1) * half]
            c = unpack_words(y[..., :t * D // 2].reshape(*y.shape[:3], *((t, D // 2) if i == 0 else (D, t // 2))))
            self.codes[i] = (c if i == 0 else c.transpose(-1, -2)).reshape(raw.shape[0], raw.shape[1], page, D)
            p = y[..., t * D // 2:].contiguous().view(T)
            self.params[i] = p.reshape(raw.shape[0], raw.shape[1], page, 2)
        return self

    def put(self, part, page, token, rows):
        """Rows [heads, D] of one token, quantised."""
        c, s, z = quantise(rows)
        self.codes[part][page, :, token] = c
        self.params[part][page, :, token] = torch.stack((s, z), -1).to(self.T)

    def rows(self, part, table, n):
        """(values, scales) in 64 bits [n, heads, D], [n, heads] of a sequence's first n tokens."""
        ids = [int(i) for i in table[:-(-n // self.page)]]
        c = self.codes[part][ids].transpose(1, 2).reshape(-1, self.heads, self.D)[:n].double()
        p = self.params[part][ids].transpose(1, 2).reshape(-1, self.heads, 2)[:n].double()
        return p[..., 1:] + p[..., :1] * c, p[..., 0]


def paths(n, parents=None):
    """[n, n]: whether node i sees node j."""
    see = np.zeros((n, n), dtype=bool)
    for i in range(n):
        j = i
        while True:
            see[i, j] = True
            if j == 0:
                break
            j = int(parents[j - 1]) if parents is not None else j - 1
    return torch.from_numpy(see)


def attention(q, k, v, vs, see, scale, T):
    """One sequence in 64 bits: q [n, Hq, D], k and v [t, Hkv, D] (cached, then
    scored rows), vs [t, Hkv] the cached values' scales (0 for scored rows),
    see [n, t].  Returns (out, lse, tolerance of out).

    The tolerance counts the kernels' roundings: a softmax weight (or its
    product with the scale) to 16 bits, off by at most half a step of bf16
    relative to its share of the sum, which weighs codes centred to at most 8
    scales in magnitude, or the value; where values are expanded to bf16 first,
    half a step of each; the output, half a step; and scores in fp32, whose sums
    of D products with an offset of up to 136 scales are off by less than
    2^-20 of the sum of magnitudes, shifting a weight by twice that."""
    n, Hq, D = q.shape
    g = Hq // k.shape[1]
    out, lse, tol = [], [], []
    for h in range(Hq):
        kh, vh, sh = k[:, h // g], v[:, h // g], vs[:, h // g]
        z = (q[:, h].double() @ kh.T) * scale
        z = torch.where(see, z, -math.inf)
        m = z.amax(-1, keepdim=True) if z.shape[1] else torch.full((n, 1), -math.inf, dtype=torch.float64)
        p = torch.where(see, torch.exp(z - torch.where(m == -math.inf, 0.0, m)), 0.0)
        total = p.sum(-1, keepdim=True)
        w = p / torch.where(total == 0, 1.0, total)
        o = w @ torch.where(see.any(0)[:, None], vh, 0.0)
        mag = q[:, h].double().abs().sum(-1) * abs(scale) * (kh.abs().amax() if kh.numel() else 0.0)
        drift = 2.0 ** -20 * 40 * mag[:, None]
        far = w @ (vh.abs() + 8 * sh[:, None])
        t = 2.0 ** -8 * (w @ (2 * vh.abs() + 8 * sh[:, None])) + HALF_STEP[T] * o.abs() + 2 * drift * far + 1e-6
        out.append(o)
        tol.append(t)
        lse.append((torch.log(total) + m)[:, 0])
    return torch.stack(out, 1), torch.stack(lse, 1), torch.stack(tol, 1)
