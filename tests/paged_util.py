"""Plain 64-bit forms of the paged-cache operators and their tolerance (not a test module).

Tolerance of an attention output element, from the arithmetic.  With u the type's half step
(torch.finfo(t).eps / 2) and A = sum_j w_j |v_j| the same attention over |v|:
  - a softmax weight is rounded once to the type for the second product, and the sum that
    divides may take the rounded weights: 2u A;
  - the result is rounded once to the type: u |out| <= u A;
  - scores and exponentials in 32 bits: a score is a sum of D <= 128 exact products, within
    D 2^-24 sum |q k| sm_scale of itself, under 130 * 2^-24 * 16 < 2^-13 for the unit-normal rows
    here (sum |q k| / sqrt(D) stays below 16), and the exponential is within 2^-13 relative, so a
    weight is within 2^-12 and the quotient within 2 * 2^-12 = 2^-11 of A.
  - a fp16 weight in the type's subnormal range is off by up to 2^-31 of the row's largest, not by u of
    itself: with L keys up to L 2^-31 max |v|, which the inputs here leave far below the 1e-6 (few
    keys lie so far below the largest) and test_gpu_paged_tails.py counts.
So |out - exact| <= (3u + 2^-11) A + 1e-6 (the last for results in the type's subnormal range).
"""
import math

import torch


def attend(q, k, v, sm_scale=0.0):
    """(out, A) of n rows over L keys in 64 bits: q [n][Hq][D], k and v [L][Hkv][D]; row i sees
    keys 0 .. L - n + i."""
    n, hq, d = q.shape
    L, hkv, _ = k.shape
    scale = sm_scale if sm_scale > 0 else 1.0 / math.sqrt(d)
    rep = torch.arange(hq, device=q.device) // (hq // hkv)
    q, k, v = (x.double() for x in (q, k, v))
    out, mean = torch.zeros_like(q), torch.zeros_like(q)
    i = torch.arange(n, device=q.device)[:, None]
    seen = torch.arange(L, device=q.device)[None, :] <= L - n + i
    some = seen.any(1)
    if not some.any():
        return out, mean
    s = torch.einsum("nhd,lhd->hnl", q, k[:, rep]) * scale
    w = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
    w = torch.where(some[None, :, None], w, torch.zeros_like(w))
    out = torch.einsum("hnl,lhd->nhd", w, v[:, rep])
    mean = torch.einsum("hnl,lhd->nhd", w, v[:, rep].abs())
    return out, mean


def assert_close(got, out, mean, what=""):
    u = torch.finfo(got.dtype).eps / 2
    assert torch.isfinite(got).all(), f"{what}: NaN or infinity"
    err = (got.double() - out).abs()
    bad = err > (3 * u + 2.0 ** -11) * mean + 1e-6
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, max err "
                           f"{err.max().item():.3e}, first at {bad.nonzero()[0].tolist()}")


def gather(pages, table_row, length):
    """The first `length` tokens of a table row's pages [num_pages][Hkv][P][D] -> [length][Hkv][D]."""
    page = pages.shape[2]
    ids = table_row[:-(-length // page)].long()
    return pages[ids].transpose(1, 2).reshape(-1, pages.shape[1], pages.shape[3])[:length]


class Books:
    """The step's bookkeeping in plain Python, the definition of kivi_paged_assign."""

    def __init__(self, lengths, table, free, num_free, page):
        self.lengths, self.table, self.page = list(lengths), [list(r) for r in table], page
        self.free, self.num_free = list(free), num_free

    def step(self, new, rows):
        """(offsets, slots, positions, status) of a step; changes the books if it succeeds."""
        P, B = self.page, len(self.lengths)
        up = lambda n: -(-n // P)  # noqa: E731
        width = len(self.table[0])
        back = sum(up(ln) for ln, n in zip(self.lengths, new) if n < 0 and 0 <= ln <= width * P)
        need = sum(up(ln + n) - up(ln) for ln, n in zip(self.lengths, new) if n >= 0)
        bad = any(ln < 0 or ln > width * P or (n >= 0 and ln + n > width * P)
                  for ln, n in zip(self.lengths, new))
        bad = bad or sum(n for n in new if n > 0) > rows or self.num_free < 0 \
            or self.num_free + back > len(self.free)
        if bad or need > self.num_free + back:
            return [0] * (B + 1), [-1] * rows, [0] * rows, 4 if bad else 8
        for b, n in enumerate(new):
            if n < 0:
                for p in self.table[b][:up(self.lengths[b])]:
                    self.free[self.num_free] = p
                    self.num_free += 1
                self.lengths[b] = 0
        offsets, slots, positions = [0], [], []
        for b, n in enumerate(new):
            n = max(n, 0)
            for j in range(up(self.lengths[b]), up(self.lengths[b] + n)):
                self.num_free -= 1
                self.table[b][j] = self.free[self.num_free]
            for pos in range(self.lengths[b], self.lengths[b] + n):
                slots.append(self.table[b][pos // P] * P + pos % P)
                positions.append(pos)
            self.lengths[b] += n
            offsets.append(offsets[-1] + n)
        pad = rows - len(slots)
        return offsets, slots + [-1] * pad, positions + [0] * pad, 0
