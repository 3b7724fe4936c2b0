"""Shared by the cache tests: a cache filled through the oracle's quantizer, page tables in a mixed
order, and the comparison of an attention result with the oracle's, row by row."""
import numpy as np
import torch

import oracle
from post_weight_quantization_12_b200 import api

DEV = "cuda"


def words_of(codes, bits):
    return torch.from_numpy(oracle.pack_rows(codes, bits).view(np.int32))


class HostCache:
    """numpy codes, scales and zeros of a cache whose every slot holds quantized random rows."""

    def __init__(self, pages, heads, page, dim, bits, group, seed, spread=0.0):
        rng = np.random.default_rng(seed)
        self.bits, self.dim, self.page, self.heads = bits, dim, page, heads
        self.part = {}
        for h in "kv":
            x = rng.standard_normal((pages, heads, page, dim)).astype(np.float32)
            if spread:
                x *= np.exp2(rng.uniform(-spread, spread, (pages, heads, page, 1))).astype(np.float32)
            if h == "k":
                x[..., : max(1, dim // 32)] *= 4
            self.part[h] = oracle.grid_quantize(x, bits, group)

    def device(self):
        t = []
        for h in "kv":
            c, s, z = self.part[h]
            t += [words_of(c, self.bits).to(DEV), torch.from_numpy(s).to(torch.bfloat16).to(DEV),
                  torch.from_numpy(z).to(DEV)]
        return api.QuantizedCache.of_tensors(*t, dim=self.dim)

    def rows(self, half, table_row, first, last, head):
        """(codes, scales, zeros) of positions first .. last - 1 of one head."""
        pos = np.arange(first, last)
        pg, off = np.asarray(table_row)[pos // self.page], pos % self.page
        return tuple(a[pg, head, off] for a in self.part[half])


def make_table(lengths, page, pages, seed, first=0, width=None):
    """int32 [batch, width], each sequence on pages of its own in a mixed order, -1 past its end."""
    need = [-(-n // page) for n in lengths]
    order = np.random.default_rng(seed).permutation(pages - first) + first
    assert sum(need) <= len(order)
    t = np.full((len(lengths), width or max(1, max(need, default=1))), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = order[at:at + k]
        at += k
    return t


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def check_attend(out, host, table, lengths, starts, q, scale, prefix=None, image16=False,
                 rows=None, flip=1.0):
    """Compares rows of `out` [n, q_heads, dim] with the oracle's within its derived bound. prefix:
    (table row, length) that every row meets first; flip: a negative or zero scale's sign."""
    out = out.double().cpu().numpy()
    qf = q.double().cpu().numpy() * np.sign(flip)
    ratio = q.shape[1] // host.heads
    for b in range(len(lengths)):
        for i in range(starts[b], starts[b + 1]):
            if rows is not None and i not in rows:
                continue
            limit = lengths[b] - starts[b + 1] + i + 1
            for h in range(host.heads):
                got = []
                for half in "kv":
                    own = host.rows(half, table[b], 0, max(0, limit), h)
                    if prefix is not None:
                        pre = host.rows(half, prefix[0], 0, prefix[1], h)
                        own = tuple(np.concatenate(t) for t in zip(pre, own))
                    got += own
                for r in range(ratio):
                    qh = h * ratio + r
                    ref, tol = oracle.attend_bound(qf[i, qh], *got, scale, image16)
                    err = np.abs(out[i, qh] - ref)
                    assert np.all(err <= tol), (b, i, qh, float((err / tol).max()),
                                                int((err > tol).sum()))
