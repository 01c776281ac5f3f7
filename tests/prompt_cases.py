"""Ragged prompt-side cases over a paged cache and their oracle answers.

Every slot no sequence owns holds NaN (unused blocks, and the slots of a
sequence's last block past its end), so a value read from there shows.

Tolerance.  The kernel rounds each softmax weight to bf16 once (at most 2^-8
of it) before the product with V and the output once (at most 2^-8 of it);
products and sums are fp32.  An fp32 dot product of D terms is off by at most
D 2^-24 sum|q k| scale, below 2^-11 of a score's magnitude-sum for D = 128
and less in the exponential for the inputs here, and ex2's 2^-22 is far
below; both are covered by 2^-10.  So
    |out - ref| <= (2^-8 + 2^-10) sum_t w_t |V_t| + 2^-8 |out|.
"""
import numpy as np
import torch

from oracle import prompt as OP
from oracle import quantize as OQ


class Prompt:
    def __init__(self, news, lens, hq, hkv, d, bs, seed=0, fp8=False, pad_rows=0, std=1.0,
                 spare=3, unowned=float("nan")):
        rng = np.random.default_rng(seed)
        self.news, self.lens, self.hq, self.hkv, self.d, self.bs = news, lens, hq, hkv, d, bs
        B = len(news)
        need = [-(-n // bs) for n in lens]
        self.nb = sum(need) + spare
        order = rng.permutation(self.nb)
        self.tab = -np.ones((B, max(need + [0]) + 1), dtype=np.int32)
        at = 0
        for b, w in enumerate(need):
            self.tab[b, :w] = order[at:at + w]
            at += w
        self.start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: (torch.randn(s, generator=g) * std).to(torch.bfloat16)  # noqa: E731
        T = int(self.start[-1]) + pad_rows
        self.q = rnd(T, hq, d)
        self.k, self.v = rnd(self.nb, hkv, bs, d), rnd(self.nb, hkv, bs, d)
        owned = np.zeros((self.nb, bs), dtype=bool)
        for b, n in enumerate(lens):
            t = np.arange(n)
            owned[self.tab[b][t // bs], t % bs] = True
        self.fp8 = fp8
        self.ks = self.vs = None
        if fp8:
            kn, vn = self.k.float().numpy(), self.v.float().numpy()
            ids, full = list(range(self.nb)), [bs] * self.nb
            kq, ks = OQ.quantize_blocks(kn, ids, full)
            vq, vs = OQ.quantize_blocks(vn, ids, full)
            kq[~owned.any(1)] = 0x7F  # NaN codes
            vq[~owned.any(1)] = 0x7F
            kq.transpose(0, 2, 1, 3)[~owned] = 0x7F
            vq.transpose(0, 2, 1, 3)[~owned] = 0x7F
            self.k, self.v = torch.from_numpy(kq), torch.from_numpy(vq)
            self.ks, self.vs = torch.from_numpy(ks), torch.from_numpy(vs)
        else:
            m = torch.from_numpy(~owned)
            self.k.permute(0, 2, 1, 3)[m] = unowned
            self.v.permute(0, 2, 1, 3)[m] = unowned
        self.scale = d ** -0.5

    def oracle(self, causal, scale=None):
        f = lambda t: None if t is None else t.numpy() if t.dtype == torch.uint8 else t.float().numpy()  # noqa: E731,E501
        return OP.attend_rows(f(self.q), f(self.k), f(self.v), self.tab, self.start, self.lens,
                              self.scale if scale is None else scale, causal, f(self.ks),
                              f(self.vs))

    def device(self):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        return dict(q=c(self.q), k=c(self.k), v=c(self.v), ks=c(self.ks), vs=c(self.vs),
                    tab=torch.from_numpy(self.tab).cuda(),
                    start=torch.from_numpy(self.start).cuda(),
                    lens=torch.tensor(self.lens, dtype=torch.int32).cuda())


def assert_rows(out, ref, spread, what=""):
    """out [T, Hq, d] against the oracle; rows of no sequence must still hold
    the NaN they were filled with."""
    got = out.detach().cpu().double().numpy()
    none = np.isnan(ref)
    assert np.isnan(got[none]).all(), f"{what}: rows behind the last sequence were written"
    assert not np.isnan(got[~none]).any(), f"{what}: NaN in the output"
    lim = (2.0 ** -8 + 2.0 ** -10) * spread[~none] + 2.0 ** -8 * np.abs(got[~none]) + 1e-30
    off = np.abs(got[~none] - ref[~none])
    bad = off > lim
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} values off; worst "
                           f"{(off / lim).max():.2f} of the bound")
