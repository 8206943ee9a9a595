"""The attention over a 4-bit cache in fp64 for whole tiles of rows at once,
for tests of long axes.  ``pool`` has ``lens``, ``Hkv``, ``D`` and
``values(name, b, h, n)`` (fp64 values, s, m, codes, which tokens have a
page)."""

from __future__ import annotations

import numpy as np

from oracle import u4


def round16(x: np.ndarray, dtype: str) -> np.ndarray:
    """fp64 rounded to bf16 or fp16 (by way of fp32), as fp64."""
    import torch
    t = torch.from_numpy(np.asarray(x, dtype=np.float64)).float()
    return t.to({"bf16": torch.bfloat16, "f16": torch.float16}[dtype]).double().numpy()


def tiles(pool, qv, new, scale, causal=True, window=0):
    """For each (sequence, KV head) with rows: a dict with the rows' indices
    ``at`` (two arrays: row of q, query head), ``o`` [R, D], ``lse`` [R], the
    weights ``w`` [R, L] and the keys' and values' ``kv, ks, km, vv, vs, vm,
    vc``, zero where a token has no page."""
    G, row = qv.shape[1] // pool.Hkv, 0
    for b, n in enumerate(new):
        L = max(pool.lens[b], 0)
        j = np.arange(L)
        pos = np.repeat(pool.lens[b] - n + np.arange(n), G)
        for h in range(pool.Hkv if n else 0):
            kv, ks, km, _, there = pool.values("k", b, h, L)
            vv, vs, vm, vc, _ = pool.values("v", b, h, L)
            for a in (kv, ks, km, vv, vs, vm):
                a[~there] = 0.0
            at = (np.repeat(row + np.arange(n), G), np.tile(h * G + np.arange(G), n))
            see = np.broadcast_to(there, (n * G, L)).copy()
            if causal:
                see &= j <= pos[:, None]
            if window:
                see &= j > pos[:, None] - window
            z = np.where(see, scale * (qv[at] @ kv.T), -np.inf)
            top = np.max(z, 1, initial=-np.inf)
            e = np.exp(z - np.where(np.isfinite(top), top, 0.0)[:, None])
            total = e.sum(1)
            w = e / np.where(total > 0, total, 1.0)[:, None]
            with np.errstate(divide="ignore"):
                lse = top + np.log(total)
            yield dict(at=at, o=w @ vv, lse=lse, w=w, see=see, kv=kv, ks=ks, km=km, vv=vv, vs=vs,
                       vm=vm, vc=vc)
        row += n


def score_error(t, qv, scale):
    """How far the kernel's scores of a tile's rows can be off [R]: fp32 sums
    of D products with codes as 16 + c, scaled, with a few roundings of their
    own (the largest over the keys that a row sees)."""
    mag, z = score_sums(t, qv, scale)
    dz = 2.0 ** -24 * ((qv.shape[-1] + 8) * mag + 8 * z)
    return np.max(np.where(t["see"], dz, 0.0), 1, initial=0.0)


def score_sums(t, qv, scale):
    """What a score's partial sums stay below, and the score's magnitude [R, L]."""
    aq = np.abs(qv[t["at"]]).sum(1)[:, None]
    mag = t["ks"] * (2 * 16 + 15) + np.abs(t["km"] - 16 * t["ks"])
    return abs(scale) * aq * mag, np.abs(scale * (qv[t["at"]] @ t["kv"].T))


def check_lse(pool, qv, lse, new, scale, causal=True, window=0):
    for t in tiles(pool, qv, new, scale, causal, window):
        got, seen = lse[t["at"]], np.isfinite(t["lse"])
        assert np.all(got[~seen] == -np.inf)
        bar = score_error(t, qv, scale) + 2.0 ** -20 * (1 + np.abs(t["lse"]))
        assert np.all(np.abs(got[seen] - t["lse"][seen]) <= bar[seen])


def outputs(pool, qv, new, scale, causal=True, window=0):
    """(out [T, q heads, D], lse [T, q heads]) in fp64."""
    T = sum(new)
    o, lse = np.zeros((T, qv.shape[1], pool.D)), np.full((T, qv.shape[1]), -np.inf)
    for t in tiles(pool, qv, new, scale, causal, window):
        o[t["at"]], lse[t["at"]] = t["o"], t["lse"]
    return o, lse


class HostPool:
    """Keys and values of some sequences in the 4-bit format, without a GPU."""

    def __init__(self, lens, Hkv, D, seed=0, keys=None, values=None):
        rng = np.random.default_rng(seed)
        self.lens, self.Hkv, self.D = list(lens), Hkv, D
        self._of = {}
        for b, n in enumerate(lens):
            for name, make in (("k", keys), ("v", values)):
                x = rng.standard_normal((max(n, 0), Hkv, D))
                if make is not None:
                    x = make(x, np.arange(max(n, 0))[:, None, None])
                self._of[name, b] = u4.encode(x)

    def values(self, name, b, h, n):
        c, p = self._of[name, b]
        c, p = c[:n, h].astype(np.float64), p[:n, h]
        s, m = u4.bits_value(p[:, 0]), u4.bits_value(p[:, 1])
        return m[:, None] + s[:, None] * c, s, m, c, np.ones(n, bool)


def by_position(x, t):
    """Values whose mean moves with their position, so that a share of the
    keys that is lost or weighted wrongly moves the result by about one."""
    return x + 2.0 * np.sin(t / 60.0)


def check_rows(pool, qv, out, lse, new, dtype, scale, causal=True, window=0, name=""):
    """Outputs and log sums of a call against fp64, with bars that an output of
    zeros or one without some of the keys cannot pass.

    What the roundings of single keys do to a result is a sum of independent
    terms of either sign, a_t at most each; it passes 7 sqrt(sum a_t^2) once in
    10^10 elements (Hoeffding).  The terms are
      the weight p s as an operand: w e_p s |c - 8|, e_p 2^-11 (bf16), 2^-20 (fp16)
      the score: 2 w |v - o| (exp, and the sum that it is divided by) times each of
        its roundings, which are fewer than D / 4 + 8 (eight for each product of 32),
        of 2^-23 of the largest partial sum at most; 2^-21 of the score's own size
    fp32 sums are charged in full: a step adds 32 keys in one product, and a wave
    walks every fourth one, so an accumulator is rounded fewer than n / 128 + 16
    times (16: the product's own sum, the waves and the chunks), each time by
    2^-23 of at most (2 72 + 15) sum(w s) (72: the codes' offset and the 8 taken
    off); the eight keys' shares of 8 s + m are added one by one.  Last, half a
    step of the output's type."""
    u = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    ep = {"bf16": 2.0 ** -11, "f16": 2.0 ** -20}[dtype]
    worst = 0.0
    for t in tiles(pool, qv, new, scale, causal, window):
        o, l = out[t["at"]], lse[t["at"]]
        none = ~t["see"].any(1)
        assert np.all(o[none] == 0) and np.all(l[none] == -np.inf), name
        nan, dz = np.isnan(t["lse"]), score_error(t, qv, scale)
        mag, z = score_sums(t, qv, scale)
        dz2 = (qv.shape[-1] / 4 + 8) * (2.0 ** -23 * mag) ** 2 + (2.0 ** -21 * z) ** 2
        assert np.isnan(o[nan]).all() and np.isnan(l[nan]).all(), name
        for r in np.flatnonzero(~none & ~nan):
            w, ro = t["w"][r][:, None], t["o"][r]
            vs, vm = t["vs"][:, None], t["vm"][:, None]
            single = w * w * ((ep * vs * (t["vc"] - 8)) ** 2 + 4 * dz2[r][:, None] * (t["vv"] - ro) ** 2)
            n = int(t["see"][r].sum())
            sums = ((n / 128 + 16) * 2.0 ** -23 * 159 * (w * vs).sum()
                    + (n / 16 + 32) * 2.0 ** -24 * (w * np.abs(8 * vs + vm)).sum())
            bar = u * np.abs(ro) + 7 * np.sqrt(single.sum(0)) + sums
            assert np.all(np.isfinite(o[r])), (name, r)
            off = np.abs(o[r] - ro)
            worst = max(worst, float((off / bar).max()))
            assert np.all(off <= bar), (name, r, float((off / bar).max()))
            assert abs(l[r] - t["lse"][r]) <= dz[r] + 2.0 ** -20 * (1 + abs(t["lse"][r])), (name, r)
    print(f"  {name}: worst error / bar {worst:.3f}", flush=True)
