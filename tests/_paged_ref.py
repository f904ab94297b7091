"""Plain 64-bit forms of the paged KV-cache calls (include/paged_kv.h), on the
CPU, position by position from their definitions, and the tests' inputs.
Shares no code with the library."""
import math

import torch

BF16, E5M2 = 1, 2
TORCH = {BF16: torch.bfloat16, E5M2: torch.float8_e5m2}
RAW = {BF16: torch.int16, E5M2: torch.uint8}


class Setup:
    """A cache with random pages and a batch: new[s] of kv[s] tokens each.
    Everything no sequence has (free pages, slots behind a length) holds NaN."""

    def __init__(self, new, kv, kv_heads, dim, dtype=BF16, page=16, head_major=False, pad=0, seed=0, spare=3,
                 values=None):
        g = torch.Generator().manual_seed(seed)
        self.g, self.new, self.kv, self.heads, self.dim, self.dtype, self.page = g, new, kv, kv_heads, dim, dtype, page
        need = [-(-max(n, 0) // page) for n in kv]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        width = max(need + [1])
        self.table = torch.full((len(kv), width), -1, dtype=torch.int32)
        for s, n in enumerate(need):
            for i in range(n):
                self.table[s, i] = order.pop()
        self.cu = torch.tensor([sum(new[:s]) for s in range(len(new) + 1)], dtype=torch.int32)
        self.kv_lens = torch.tensor(kv, dtype=torch.int32)
        self.total = sum(new) + pad
        draw = values or (lambda *shape: torch.randn(*shape, generator=g))
        self.k, self.v = (self._pool(draw, head_major) for _ in range(2))

    def _pool(self, draw, head_major):
        x = torch.full((self.pages, self.page, self.heads, self.dim), math.nan)
        for s, n in enumerate(self.kv):
            for i in range(-(-n // self.page)):
                rows = min(self.page, n - i * self.page)
                x[self.table[s, i], :rows] = draw(rows, self.heads, self.dim)
        x = x.to(torch.bfloat16).to(TORCH[self.dtype])
        if head_major:
            x = x.view(RAW[self.dtype]).transpose(1, 2).contiguous().transpose(1, 2).view(TORCH[self.dtype])
        return x

    def rows(self, heads, seed=None, dtype=torch.bfloat16):
        g = self.g if seed is None else torch.Generator().manual_seed(seed)
        return torch.randn(self.total, heads, self.dim, generator=g).to(torch.bfloat16).to(dtype)

    def place(self, s, p):
        return int(self.table[s, p // self.page]), p % self.page

    def sequence(self, pool, s):
        """[kv, heads, dim] in 64 bits."""
        out = torch.zeros(self.kv[s], self.heads, self.dim, dtype=torch.float64)
        for p in range(0, self.kv[s], self.page):
            page, n = int(self.table[s, p // self.page]), min(self.page, self.kv[s] - p)
            out[p:p + n] = pool[page, :n].to(torch.float64)
        return out

    def tokens(self):
        """(row, sequence, position) of each new token."""
        for s, n in enumerate(self.new):
            for i in range(n):
                yield int(self.cu[s]) + i, s, self.kv[s] - n + i


def attention(st, q, scale=None, causal=True, window=0):
    """(out, lse, bound on |weights' error| x values, bound on scores' error):
    out [total, q_heads, dim], lse [total, q_heads]; rows of padding are 0.
    spread = sum_j softmax_j |v_j|, wide = the largest scale |q| . |k_j|."""
    heads = q.shape[1]
    group = heads // st.heads
    scale = st.dim ** -0.5 if scale is None else scale
    out = torch.zeros(st.total, heads, st.dim, dtype=torch.float64)
    spread = torch.zeros_like(out)
    lse = torch.zeros(st.total, heads, dtype=torch.float64)
    wide = torch.zeros(st.total, heads, dtype=torch.float64)
    for s, n in enumerate(st.new):
        k, v = st.sequence(st.k, s), st.sequence(st.v, s)
        for i in range(n):
            row, p = int(st.cu[s]) + i, st.kv[s] - n + i
            hi = 0 if p < 0 else p + 1 if causal else st.kv[s]
            lo = max(0, p + 1 - window) if window else 0
            if hi <= lo:
                lse[row] = -math.inf
                continue
            for h in range(heads):
                x, kk, vv = q[row, h].to(torch.float64), k[lo:hi, h // group], v[lo:hi, h // group]
                score = scale * (kk @ x)
                top = score.max()
                w = torch.exp(score - top)
                lse[row, h] = top + torch.log(w.sum())
                w = w / w.sum()
                out[row, h] = (w[:, None] * vv).sum(0)
                spread[row, h] = (w[:, None] * vv.abs()).sum(0)
                wide[row, h] = (scale * (kk.abs() @ x.abs())).max()
    return out, lse, spread, wide


def attention_tolerance(st, q, out, spread, wide):
    """Per-element bounds, from the roundings: the output's (2^-8 of it);
    each weight's to 16 bits (2^-8 for BF16; FP16: 2^-11, and 2^-25 of the
    largest weight where it is subnormal); the scores' in 32 bits, where a dot
    product of dim terms is off by dim 2^-24 of its absolute sum, twice over
    for c s - m and its exponential; sums over n keys by n 2^-24 of theirs."""
    n = max(st.kv + [1])
    score = wide * (st.dim + 8) * 2.0 ** -23 + 2.0 ** -22
    f32 = 2 * score + 2 * n * 2.0 ** -24
    if st.dtype == BF16:
        weight = spread * (2.0 ** -8 + f32[..., None])
    else:
        most = max(float(st.sequence(st.v, s).abs().max()) if st.kv[s] else 0.0 for s in range(len(st.kv)))
        weight = spread * (2.0 ** -11 + f32[..., None]) + n * 2.0 ** -25 * most
    return 2.0 ** -8 * (out.abs() + weight) + weight, score + n * 2.0 ** -24


def norm(x, w, eps):
    x = x.to(torch.float64)
    if w is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.to(torch.float64)


def rotate(x, cos_sin, p, interleaved):
    """x [heads, dim] at position p by row p of the table; (rotated, sum of the terms' magnitudes)."""
    r = cos_sin.shape[1]
    c, s = cos_sin[p, :r // 2].to(torch.float64), cos_sin[p, r // 2:].to(torch.float64)
    y, size = x.clone(), x.abs()
    for i in range(r // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        y[:, a] = x[:, a] * c[i] - x[:, b] * s[i]
        y[:, b] = x[:, b] * c[i] + x[:, a] * s[i]
        size[:, a] = (x[:, a] * c[i]).abs() + (x[:, b] * s[i]).abs()
        size[:, b] = (x[:, b] * c[i]).abs() + (x[:, a] * s[i]).abs()
    return y, size


def round_to(x, torch_dtype):
    """64-bit values to BF16 or E5M2, nearest even, without a rounding between:
    scaled so that a step of the type is 1, rounded there and scaled back."""
    bits, low, top = (8, -133, 3.3961775292304957e38) if torch_dtype == torch.bfloat16 else (3, -16, 61440.0)
    _, e = torch.frexp(x)
    step = torch.clamp(e - bits, min=low)
    y = torch.ldexp(torch.round(torch.ldexp(x, -step)), step)
    return torch.where(x.abs() >= top, torch.copysign(torch.full_like(x, math.inf), x), y)
