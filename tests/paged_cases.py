"""Small paged caches for the tests of the block-scaled cache and of attention with a
window: seeded numpy inputs, NaN (or the largest code) in every slot outside a context."""
from __future__ import annotations

import dataclasses

import numpy as np

from oracle import block_scaled as OB
from tests import gpu_cases as GC

import workloads as W


@dataclasses.dataclass
class Paged:
    kv: str                 # "bf16", "fp8_e4m3", "int8", "f32"
    lens: list
    tables: np.ndarray      # [S, MB], -1 past a context
    k: np.ndarray           # caches [NB, bs, Hkv, D] in storage
    v: np.ndarray
    ks: np.ndarray | None   # [NB, stride] or [Hkv] float32
    vs: np.ndarray | None

    @property
    def bs(self):
        return self.k.shape[1]

    def values(self, s, first=0, n=None):
        """float64 K, V of positions first .. first + n - 1 of sequence s."""
        n = self.lens[s] - first if n is None else n
        return tuple(OB.gather(c, sc, self.tables[s], first, n, self.kv).astype(np.float64)
                     for c, sc in ((self.k, self.ks), (self.v, self.vs)))

    def device(self):
        import torch
        d = {"tables": torch.from_numpy(self.tables).cuda(),
             "lens": torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
             "k": GC.to_torch(self.k, self.kv), "v": GC.to_torch(self.v, self.kv)}
        if self.ks is not None:
            d["ks"], d["vs"] = torch.from_numpy(self.ks).cuda(), torch.from_numpy(self.vs).cuda()
        return d


def bf16_bits(x):
    return W.f32_to_bf16_bits(np.asarray(x, dtype=np.float32))


def make(seed, kv, lens, hkv, d, bs, scales="block", stride=None, extra_blocks=3, mb=None,
         spread=1.0):
    """``scales``: "block", "head" or (f32 / bf16 caches) ignored; ``spread``: how many
    powers of e the scales of blocks differ by (one sigma)."""
    rng = np.random.default_rng(seed)
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + extra_blocks
    perm = rng.permutation(nb).astype(np.int32)
    mb = max(need + [1]) if mb is None else mb
    tables = np.full((len(lens), mb), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = perm[at:at + n]
        at += n
    shape = (nb, bs, hkv, d)
    dt, poison = GC.POISON[kv]
    caches = []
    for _ in range(2):
        if kv == "f32":
            x = rng.standard_normal(shape).astype(np.float32)
        elif kv == "bf16":
            x = bf16_bits(rng.standard_normal(shape))
        else:
            q = rng.standard_normal(shape).astype(np.float32) * OB.QMAX[kv] / 4
            x = OB.encode(q, kv)
        used = np.zeros((nb, bs), dtype=bool)
        for s, n in enumerate(lens):
            for i in range(need[s]):
                used[tables[s, i], : min(bs, n - i * bs)] = True
        x = x.astype(dt)
        x[~used] = poison
        caches.append(x)
    ks = vs = None
    if kv in OB.QMAX:
        stride = hkv if stride is None else stride
        shp = (hkv,) if scales == "head" else (nb, stride)
        ks, vs = (np.exp(spread * rng.standard_normal(shp)).astype(np.float32) * np.float32(4)
                  / OB.QMAX[kv] for _ in range(2))
    return Paged(kv, list(lens), tables, caches[0], caches[1], ks, vs)


# ---- error bounds ------------------------------------------------------------
# Half steps relative to the value: bf16 2^-8, fp16 2^-11, float32 2^-24.  The tensor cores
# accumulate in float32; 2^-23 per addition covers truncation.
def attention_bound(case, q, out, mag, reach, scale, q_f32, out_bf16, hi_lo, longest, e_p=None,
                    floor=None):
    """Elementwise bound on |kernel - out| ``[n, Hq, D]``; ``mag`` = A = sum p |v|, ``reach``
    = max over tokens of sum_d |q_d k_d|, ``longest`` the most tokens a query sees.

    z: 24 float32 steps on sum |q k| (the k-steps' additions, the scales' products, the
    exponent's argument), and q's split where q is float32 (bf16 hi + lo 2^-16, fp16 2^-22).
    p: hi + lo (bf16 2^-16, fp16 2^-22) or one value (bf16 2^-8, fp16 2^-11); ex2.approx and
    the V scale's product 2^-21.  Sums: a float32 step for each 16 tokens and 24 for warps and partitions.
    These act on numerator and denominator alike: twice their sum times A.

    8-bit caches: an fp16 weight below 2^-14 is off by up to 2^-25 where the largest weight
    is at least 1, that is by 2^-25 max(vs) in p |v| per unit code: 2^-25 qmax max(vs) a token
    (in decode the largest weight is at least 2^7, which only makes this smaller).

    INT8 with one fp16 weight (no hi + lo) carries code + 1152 (at most 1279) in both
    products: 16 float32 steps on sum |q| 1279 ks in z, and a step for each 16 tokens, twice
    (the sum and what is taken off), on 1279 max(vs) in the output.

    ``e_p`` and ``floor``, where given, take the place of the weights' relative term and of the
    2^-25 of a weight (8-bit caches).
    """
    codes = case.kv in OB.QMAX
    steps = longest / 16 + 24
    scale = abs(float(np.float32(scale)))
    dz = scale * reach * (24 * 2.0 ** -23 + (0 if not q_f32 else 2.0 ** (-22 if codes else -16)))
    extra = 0.0
    if codes:
        vs, ks = (float(x.max()) for x in (case.vs, case.ks))
        extra = longest * (2.0 ** -25 if floor is None else floor) * float(OB.QMAX[case.kv]) * vs
        if case.kv == "int8" and not hi_lo:
            dz = dz + 16 * 2.0 ** -23 * scale * 1279 * ks * np.abs(q).sum(-1)
            extra += 2 * steps * 2.0 ** -23 * 1279 * vs
    if e_p is None:
        e_p = (2.0 ** -22 if codes else 2.0 ** -16) if hi_lo else 2.0 ** (-11 if codes else -8)
    e = 2 * (dz[..., None] + e_p + 2.0 ** -21 + steps * 2.0 ** -23) * mag + extra
    return e + (2.0 ** -8 if out_bf16 else 2.0 ** -23) * (np.abs(out) + e)
