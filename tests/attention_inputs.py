"""Sequences, page tables and caches for the tests of the cache and its attention."""
import numpy as np
import torch

BF16, F32 = torch.bfloat16, torch.float32


def int32(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def strided(t, pad):
    """t (rows x n) in rows of n + pad values, the padding NaN."""
    full = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    full[:, :t.shape[1]] = t
    return full[:, :t.shape[1]]


class Paged:
    """A cache whose pages hold garbage (NaN scales), and the table of sequences of given lengths in it."""

    def __init__(self, wr, lengths, heads, dim, page, group, seed=0, spare=2):
        self.wr, self.lengths, self.heads, self.dim, self.page, self.group = wr, list(lengths), heads, dim, page, group
        used = [-(-n // page) for n in lengths]
        self.pages = sum(used) + spare
        self.cache = wr.KvCache(self.pages, heads, dim, page_tokens=page, group=group)
        self.cache.buf.fill_(255)
        order = np.random.default_rng(seed).permutation(self.pages)
        self.table = np.full((len(used), max(max(used), 1)), -1, np.int32)
        at = 0
        for i, n in enumerate(used):
            self.table[i, :n] = order[at:at + n]
            at += n

    def sequences(self, new, lengths=None, most_new=None, most=None):
        lengths = self.lengths if lengths is None else lengths
        starts = np.concatenate([[0], np.cumsum(new)])
        return self.wr.Sequences(int32(starts), int32(lengths), int32(self.table), max(new) if most_new is None else most_new,
                                 max(lengths) if most is None else most)

    def fill(self, ctx, k, v):
        """All positions of all sequences from k and v (rows x heads * dim)."""
        self.wr.wr_kv_write(ctx, self.cache, self.sequences(self.lengths), k, v)
