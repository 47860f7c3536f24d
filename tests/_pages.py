"""A cache in pages and 8 bits for the tests: pools in which everything that a call must not read is poison, and the
operators in 64 bits with the errors that their arithmetic allows."""
import math

import torch

import deepseek_v4_compressed_csa_gb300 as csa

F8 = torch.float8_e4m3fn
F64 = torch.float64
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # the most that one rounding is off, relative
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}  # and half of the smallest step, below the normal numbers
U32 = 2.0 ** -24
EPS = 1e-6


def layer(small=False, **kw):
    base = dict(dtype=torch.float32, H=8, D=64, R=16, W=32, ratio=4, Hi=4, Di=32, topk=16, X=128) if small else dict(
        dtype=torch.bfloat16, H=64, D=512, R=64, W=128, ratio=4, Hi=64, Di=128, topk=512, X=4096)
    return csa.Layer(**{**base, **kw})


def inv_freq(L, base=160000.0):
    i = torch.arange(L.R // 2, dtype=F64)
    return (base ** (-2.0 * i / L.R)).float().cuda()


def turn(x, p, freq, sign):
    """x [.., dim] in 64 bits, its last values turned by sign * p * freq (the angle is one fp32 product); p [..]."""
    th = (p.float()[..., None] * freq).to(F64)
    c, s, R = th.cos(), sign * th.sin(), 2 * freq.numel()
    u, v = x[..., -R::2], x[..., 1 - R::2]
    return torch.cat((x[..., :-R], torch.stack((u * c - v * s, u * s + v * c), -1).flatten(-2)), -1)


def pair_sum(x, R):
    """x with the last R values replaced by the sum of their pair: how far an error of either reaches after a rotation."""
    y = x.clone()
    y[..., -R:] = (x[..., -R::2] + x[..., 1 - R::2]).repeat_interleave(2, -1)
    return y


def check(got, want, allow, what=""):
    """|got - want| <= allow everywhere, NaN where NaN is wanted and nowhere else."""
    got, want = got.to(F64), want.to(F64)
    assert got.shape == want.shape, what
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    over = torch.where(nan, torch.zeros_like(want), (got - want).abs() - allow)
    worst = over.max().item() if over.numel() else -1.0
    assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} too far, by up to {worst:.3g}"


def check_codes(codes, scales, y, err, what=""):
    """Codes and scales (one a row of codes' last dimension) of the values y, known up to err: the scale is the largest
    magnitude / 448 (one fp32 division), a value within E4M3's half step (2^-4 of it, or half of the smallest step, 2^-10
    of the scale)."""
    want = y.abs().amax(-1) / 448
    check(scales, want, err.amax(-1) / 448 + want * 2 * U32, what + " scales")
    s = scales.to(F64)[..., None]
    back = codes.view(F8).to(F64) * s
    # (a quotient at a rounding border moves by its own fp32 rounding, far below the step: 2^-4 and a little)
    check(back, y, y.abs() * (2.0 ** -4 * (1 + 2.0 ** -10)) + s * 2.0 ** -10 + 2 * err, what + " values")


class Cache:
    """A pool with poison (NaN codes and scales) wherever no row was put, and tables that name no page there."""

    def __init__(self, L, page, n_pages, seed=0, junk=-1):
        self.L, self.page, self.n = L, page, n_pages
        self.codes = torch.full((n_pages, page, L.D), 0x7F, dtype=torch.uint8, device="cuda")
        self.scales = torch.full((n_pages, page), math.nan, device="cuda")
        g = torch.Generator().manual_seed(seed)
        self.free = torch.randperm(n_pages, generator=g).tolist()
        self.junk = junk

    @property
    def pages(self):
        return csa.Pages(self.codes, self.scales)

    def table(self, B, width):
        return torch.full((B, width), self.junk, dtype=torch.int32)

    def place(self, table, b, rows):
        """Physical rows of logical rows of sequence b; pages are taken from the pool as they are met."""
        out = []
        for j in rows:
            k = j // self.page
            if not 0 <= int(table[b, k]) < self.n:
                table[b, k] = self.free.pop()
            out.append(int(table[b, k]) * self.page + j % self.page)
        return out

    def put(self, table, b, rows, x):
        """x [len(rows), D] fp32 as codes and scales at logical rows."""
        s = x.abs().amax(-1) / 448
        q = torch.where(s[:, None] > 0, x / torch.where(s > 0, s, 1.0)[:, None], 0.0).to(F8)
        at = torch.tensor(self.place(table, b, rows), dtype=torch.long, device="cuda")
        self.codes.view(-1, self.L.D)[at] = q.view(torch.uint8)
        self.scales.view(-1)[at] = s

    def values(self, table, b, rows):
        at = torch.tensor([int(table[b, j // self.page]) * self.page + j % self.page for j in rows], dtype=torch.long,
                          device="cuda")
        return (self.codes.view(F8).view(-1, self.L.D)[at].to(F64), self.scales.view(-1)[at].to(F64))


def attend_ref(L, q, codes, s, sink, tensor_cores):
    """(output before its rotation, allowed error) of q [H, D] over the keys s * codes [n, D], in 64 bits."""
    H, D = q.shape
    q = q.to(F64)
    if codes.shape[0] == 0:
        return torch.zeros(H, D, dtype=F64, device="cuda"), torch.zeros(H, D, dtype=F64, device="cuda")
    keys = codes * s[:, None]
    scale = L.scale or D ** -0.5
    lg = q @ keys.T * scale
    both = lg if sink is None else torch.cat((lg, sink.to(F64)[:, None]), 1)
    p = torch.softmax(both, 1)[:, : lg.shape[1]]
    # logits: the products' sums in fp32.  A sum of D terms with a rounding each is off by at most D U32 of the terms'
    # magnitudes (the tensor cores add 32 at a time; what they drop below a step's largest, 2^-22 of it, stays within that)
    mag = (q.abs() @ keys.abs().T).amax(1, keepdim=True) * scale
    d_lg = D * U32 * mag + 8 * U32 * lg.abs().amax(1, keepdim=True)
    A = p @ keys.abs()  # [H, D]
    n = lg.shape[1]
    err = A * (2 * d_lg + (n + 32) * U32)
    # A weight below fp32's smallest normal number, 2^-126, is rounded to a multiple of 2^-149, or counts as nothing (the
    # hardware's exp2 flushes it): its key's values are off by less than 2^-126 of themselves; with the sink far above every
    # key that is all there is.
    err = err + 2.0 ** -126 * keys.abs().sum(0)
    if tensor_cores:
        # The queries' two E4M3 parts: scaled so that the head's largest value is at least 2^7, the first holds four digits,
        # exactly down to 2^-6 and within half of its smallest step, 2^-10, below; the second, 16 times finer, the four digits
        # behind.  So values up to 2^-13 of the largest are off by at most 2^-17 of it, the others exact; exp2 and its
        # argument's fp32 rounding.
        top = q.abs().amax(1, keepdim=True)
        low = (q.abs() <= top * 2.0 ** -13).to(F64) @ keys.abs().T
        err = err + A * (2 * scale * top * 2.0 ** -17 * low.amax(1, keepdim=True) + 2.0 ** -20)
        # The probabilities' parts of w = p s, E5M2 (at most 2^-3 off) and what that leaves in E4M3 (2^-4 of it, or half of
        # its smallest step, 2^-10 where the largest w is at least 2^5); what E5M2's smallest step, 2^-16, leaves is within that.
        w = p * s.abs()
        err = err + (2.0 ** -7 * w + torch.minimum(2.0 ** -3 * w + w.amax(1, keepdim=True) * 2.0 ** -22, w.amax(1, keepdim=True) * 2.0 ** -15)) @ codes.abs()
    return p @ keys, err


def attend_all(L, q, cache, pos, counts, out0, token_table=None, first=0, row_table=None, n_rows=None, sel=None,
               n_sel=None, sink=None, freq=None):
    """(outputs, allowed errors) of a call of attend_pages, query by query; tables on the host."""
    B, T, H, D = q.shape
    want, allow = out0.to(F64).clone(), torch.zeros_like(out0, dtype=F64)
    tensor_cores = L.dtype == torch.bfloat16 and (L.H, L.D, L.R) == (64, 512, 64) and cache.page % 8 == 0
    for b in range(B):
        for i in range(counts[b]):
            p = pos[b] + i
            parts = []
            if row_table is not None:
                if sel is not None:
                    rows = [int(j) for j in sel[b, i, : int(n_sel[b, i])]]
                    rows = [j for j in rows if 0 <= j < n_rows[b]]
                else:
                    rows = list(range(min(n_rows[b], (p + 1) // L.ratio)))
                parts.append(cache.values(row_table, b, rows))
            if token_table is not None:
                parts.append(cache.values(token_table, b, sorted(set(range(max(0, p - L.W + 1), p + 1)) |
                                                                set(range(min(first, p + 1))))))
            codes = torch.cat([c for c, _ in parts])
            s = torch.cat([v for _, v in parts])
            o, e = attend_ref(L, q[b, i], codes, s, sink, tensor_cores)
            if freq is not None:
                at = torch.full((H,), p, device="cuda")
                e = pair_sum(e + 8 * U32 * o.abs(), L.R)
                o = turn(o, at, freq, -1.0)
            want[b, i] = o
            allow[b, i] = e + (o.abs() + e) * HALF[L.dtype] + LEAST[L.dtype]
    return want, allow
