"""The draft-tree and eviction operators from their definitions, in 64 bits, one
sequence and one head at a time; test support only."""
import numpy as np
import torch

import helpers


class Model:
    """Every key and value a batch ever saw, in order: the cache's definition."""

    def __init__(self, plens, W, H, d, dtype, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.plens, self.W, self.H, self.d, self.dtype = list(plens), W, H, d, dtype
        self.g = g
        self.pk = [self.draw(p, H, d) for p in plens]
        self.pv = [self.draw(p, H, d) for p in plens]
        self.gk = [[] for _ in plens]  # generated tokens, each [H, d]
        self.gv = [[] for _ in plens]

    def draw(self, *shape):
        return torch.randn(*shape, generator=self.g, dtype=torch.float32).to(self.dtype)

    def generate(self, counts):
        for b, n in enumerate(counts):
            for _ in range(n):
                self.gk[b].append(self.draw(self.H, self.d))
                self.gv[b].append(self.draw(self.H, self.d))
        return self

    @property
    def t(self):
        return [len(x) for x in self.gk]

    def fill(self, st, layer=0, unheld=float("nan")):
        """The state's cache as ordinary decoding would leave it; `unheld` in empty slots."""
        for b, P in enumerate(self.plens):
            for h in range(self.H):
                for which, p, gen in (("k", self.pk, self.gk), ("v", self.pv, self.gv)):
                    view = st.cache_view(layer, which, b, h)
                    rows = torch.full((P + self.W, self.d), unheld, dtype=self.dtype)
                    rows[:P] = p[b][:, h]
                    for i, x in enumerate(gen[b]):
                        rows[P + i % self.W] = x[h]
                    view.copy_(rows)

    def entries(self, b, h, more_k, more_v, swa=False):
        """Keys and values that the last of the tokens `more` (a path, each [H, d]) sees."""
        k = [x[h] for x in self.gk[b]] + [x[h] for x in more_k]
        v = [x[h] for x in self.gv[b]] + [x[h] for x in more_v]
        pk, pv = self.pk[b][:, h], self.pv[b][:, h]
        if swa:
            cut = max(0, self.plens[b] + len(k) - self.W)
            pk, pv = pk[min(cut, len(pk)):], pv[min(cut, len(pv)):]
        return (torch.cat([pk, torch.stack(k[-self.W:])]).double(),
                torch.cat([pv, torch.stack(v[-self.W:])]).double())


def attend(q, k, v, scale):
    """(output, sum of weight x |value|) of one query in 64 bits."""
    s = (k @ q.double()) * scale
    w = torch.softmax(s, 0)
    return w @ v, w @ v.abs()


def path_of(parent, i):
    p = [i]
    while parent[p[-1]] >= 0:
        p.append(parent[p[-1]])
    return p[::-1]


def tolerance(ref, mass, dtype):
    """fp32: the framework's bound.  bf16: each weight is rounded by at most half a step
    (2^-8) before it meets its value, and the output by half a step again; the fp32 sums
    and exponentials add far less than 1e-5 of the mass."""
    if dtype == torch.float32:
        return torch.full_like(ref, helpers.F32_TOL)
    return 2.0 ** -8 * (mass + ref.abs()) * 1.01 + 1e-5 * (1 + mass)


def bf16_half_step(x):
    """Half the distance between the bf16 values around |x|."""
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -126))) - 8)


def pair_tolerance(q, k, ref, mass, scale):
    """bf16 with every weight as a sum hi + lo of two bf16 values, both cut off: lo misses less
    than 2^-7 of a rest that is less than 2^-7 of the weight, so 2^-14 of the mass.  The sums,
    counted as one fp32 cut-off (2^-23) for every 16 products and a few more within those: a
    score's d / 16 + 8 <= 16 of its products' absolute sum S, which change weights and their
    sum alike, and the output's n / 16 + 8 of the mass.  Then one rounding of the output."""
    s_abs = float((k.abs() @ q.double().abs()).max()) * scale
    part = 1.01 * 2.0 ** -14 + 2.0 ** -23 * (2 * 16 * s_abs + k.shape[0] / 16 + 8)
    err = part * mass
    return bf16_half_step(ref.abs() + err) + err


def cut_bf16(w):
    """fp32 values with the lower half of their bits 0."""
    return (w.float().view(torch.int32) & -65536).view(torch.float32)


def pair_attend(q, k, v, scale, lo=1.0):
    """The output in bf16 with weights hi + lo as in pair_tolerance, `lo` times the second."""
    s = (k @ q.double()) * scale
    w = torch.exp(s - s.max()).float()
    hi = cut_bf16(w)
    pair = hi.double() + lo * cut_bf16(w - hi).double()
    return ((pair @ v) / w.double().sum()).to(torch.bfloat16).double()


def random_parents(rng, T, reach=6):
    return [int(rng.integers(max(-1, i - reach), i)) if i else -1 for i in range(T)]


def kept_slots(score, keep, n_first, n_last):
    """Slots of the `keep` highest scores, the lower slot first among equals, ascending."""
    P = len(score)
    rank = []
    for s in range(P):
        x = float(score[s])
        guarded = s < n_first or s >= P - n_last
        rank.append((0 if guarded else 1, 1 if np.isnan(x) else 0, 0.0 if np.isnan(x) else -x, s))
    return sorted(r[3] for r in sorted(rank)[:keep])
