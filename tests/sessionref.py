"""Plain 64-bit statements of the windowed-session operators, for their tests.

Nothing here calls the library: pools are read as bytes and opened with numpy,
the rotary angles are taken in extended precision, and the page operations run
on Python integers.
"""
from __future__ import annotations

import math

import numpy as np
import torch

import long_context_quantized_b200 as nf

BLOCK = 256


def open_nibbles(b):
    b = b.astype(np.int64)
    both = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], 128)
    return np.where(both > 7, both - 16, both).astype(np.float64)


def open_pool(kv):
    """K and V of every slot in fp64: two arrays [blocks][H][256][128]."""
    def np_of(t):
        return None if t is None else t.cpu().numpy() if t.dtype != torch.bfloat16 else t.float().cpu().numpy()
    kc, ks, vc, vs = (np_of(t) for t in (kv.k_codes, kv.k_scales, kv.v_codes, kv.v_scales))
    with np.errstate(invalid="ignore"):
        if kv.fmt == nf.NF_KV_BF16:
            return kc.astype(np.float64), vc.astype(np.float64)
        if kv.fmt == nf.NF_KV_K4V4:
            def rows(c, s):
                return open_nibbles(c) * np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, -1)
            return rows(kc, ks), rows(vc, vs)
        if kv.fmt == nf.NF_KV_F8:
            def rows8(c, s):
                x = torch.from_numpy(c).view(torch.float8_e4m3fn).float().numpy()
                return x.astype(np.float64) * s.astype(np.float64)[..., None]
            return rows8(kc, ks), rows8(vc, vs)
        k = kc.astype(np.float64) * ks.astype(np.float64)[..., None]
        if kv.fmt == nf.NF_KV_K8V8:
            return k, vc.astype(np.float64) * vs.astype(np.float64)[..., None]
        return k, open_nibbles(vc) * np.repeat(vs.astype(np.float64), 32, -1)


def visible(L, n_q, window, n_sink):
    """[n_q][L]: key t is seen by query j at P = L - n_q + j."""
    t, P = np.arange(L)[None], (L - n_q + np.arange(n_q))[:, None]
    return (t <= P) & ((t > P - window) | (t < n_sink))


def window_attention(kv, q, table, seqlens, window, n_sink, scale):
    """fp64 (out, lse, tol): tol is the part of the error bound that depends on
    the data, see tolerance()."""
    K, V = open_pool(kv)
    q = q.double().cpu().numpy()
    B, n_q, Hq, _ = q.shape
    G = Hq // kv.num_kv_heads
    out = np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    mag = np.zeros(q.shape)              # sum of weight x |v|
    spread = np.zeros((B, n_q, Hq, 1))   # keys / sum of exp(s - max), times max |v|
    dq = np.zeros((B, n_q, Hq, 1))       # scale x max|q| x max over keys of sum |k|
    dk = np.zeros((B, n_q, Hq, 1))       # scale x max over keys of sum |q k|
    for b, L in enumerate(seqlens):
        if L < n_q:
            continue
        see = visible(L, n_q, window, n_sink)
        some = np.nonzero(see.any(0))[0]  # keys no query sees are not even opened
        see = see[:, some]
        pages = np.asarray(table)[b][some // BLOCK]
        for h in range(kv.num_kv_heads):
            k, v = K[pages, h, some % BLOCK], V[pages, h, some % BLOCK]
            for j in range(n_q):
                kk, vv = k[see[j]], v[see[j]]
                for g in range(h * G, (h + 1) * G):
                    s = scale * (kk @ q[b, j, g])
                    m = s.max()
                    e = np.exp(s - m)
                    w = e / e.sum()
                    out[b, j, g] = w @ vv
                    lse[b, j, g] = m + math.log(e.sum())
                    mag[b, j, g] = w @ np.abs(vv)
                    spread[b, j, g] = len(s) / e.sum() * np.abs(vv).max()
                    dq[b, j, g] = scale * np.abs(q[b, j, g]).max() * np.abs(kk).sum(1).max()
                    dk[b, j, g] = scale * (np.abs(kk) @ np.abs(q[b, j, g])).max()
    return out, lse, dict(mag=mag, spread=spread, dq=dq, dk=dk, lift=value_lift(kv, G * n_q))


def value_lift(kv, rows):
    """9 to 32 rows of K8/V4, int8 and fp8 pools run on tcgen05, where a weight
    is multiplied by 2^(E - 15), E the exponent field of the key's largest V
    scale, and its value by the inverse: the largest 2^(15 - E) of the pool's
    slots.  1 for the other shapes."""
    if kv.fmt not in (nf.NF_KV_K8V4, nf.NF_KV_K8V8, nf.NF_KV_F8) or not 9 <= rows <= 32:
        return 1.0
    bits = kv.v_scales.view(torch.int16).cpu().numpy().astype(np.int64) & 0x7FFF
    field = bits >> 10
    if kv.fmt == nf.NF_KV_K8V4:
        field = field.max(-1)
    return float(2.0 ** (15 - max(1, int(field[(bits > 0).any(-1) if bits.ndim > field.ndim else bits > 0].min()))))


def decode_tolerance(parts):
    """Element-wise bound of the decode kernel's error before the last rounding.

    Each weight is rounded to fp16 and so is its product with the V scale: 2 x
    2^-11 relative, of sum w |v|.  A weight (or product) below fp16's normal
    range 2^-14 is off by at most 2^-25 instead, where the largest weight is at
    least 2^-4, so the row sum is at least sum exp(s - max) / 16: n 2^-25 16 /
    sum exp(s - max) x max|v|, twice (weight and product) -- times the lift 2^(15
    - E) that the tcgen05 form takes out of the weights.  The query's two
    digits leave 2^-16 max|q| per element, which moves a score by at most dq
    2^-16 and a normalised weight by twice that relatively.  fp32 sums and
    exponentials: 2^-15 covers 2^8 additions of half a step each, and the
    conversions."""
    return (2.0 ** -10 + 2 * 2.0 ** -16 * parts["dq"] + 2.0 ** -15) * parts["mag"] + parts["spread"] * 2.0 ** -20 * parts["lift"]


def prefill_tolerance(parts):
    """The same for the tcgen05 prefill: q (down to 2^-14 of its row's max exactly,
    below that by at most 2^-25) and the dequantised K (2^-11) are held in fp16, so a
    score moves by at most 2^-11 dk + 2^-25 dq, a normalised weight by twice that
    relatively; the weights and V are rounded to fp16 once each (2 x 2^-11); weights
    reach 2^8 and the running max is within 2^8 of the true one, so the largest
    weight is at least 1 and what fp16 loses at its bottom is n 2^-25 / sum exp(s -
    max).  fp32 sums and exponentials as above."""
    return ((2 * (2.0 ** -11 * parts["dk"] + 2.0 ** -25 * parts["dq"]) + 2.0 ** -10 + 2.0 ** -15) * parts["mag"]
            + parts["spread"] * 2.0 ** -24)


def check_out(out, ref, tol):
    """Element-wise: within tol, plus half a bf16 step (2^-8) of a bf16 result."""
    got = out.double().cpu().numpy()
    assert np.all(np.isfinite(got))
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    bound = tol + half * (np.abs(ref) + tol) + 1e-30
    bad = np.abs(got - ref) > bound
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - ref) / bound).max()))


def filled_pool(fmt, blocks, heads, seed=1, k_gain=1.0):
    """A pool with quantised normal values in every slot."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kv = nf.KVLayer.empty(fmt, blocks, heads)
    k, v = (torch.randn((1, blocks * BLOCK, heads, 128), generator=gen, device="cuda") for _ in range(2))
    table = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
    nf.nf_kv_append_quant(kv, k * k_gain, v, table, torch.zeros(1, dtype=torch.int32, device="cuda"))
    return kv


def make_table(seqlens, blocks, width=None, seed=0):
    rng = np.random.default_rng(seed)
    order = rng.permutation(blocks)
    need = [math.ceil(L / BLOCK) for L in seqlens]
    table = np.full((len(seqlens), width or max(1, max(need))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    assert at <= blocks
    return table


# ------------------------------------------------------------------ rotary
def rope_rows(x, positions, inv_freq, axis, layout, rot):
    """x [..., heads, 128] (float64) turned; positions [..., axes] ints."""
    a = positions[..., axis].astype(np.longdouble) * inv_freq.astype(np.longdouble)
    c, s = np.cos(a)[..., None, :], np.sin(a)[..., None, :]
    y = x.astype(np.longdouble).copy()
    half = rot // 2
    if layout == nf.NF_ROPE_PAIRS:
        i, j = slice(0, rot, 2), slice(1, rot, 2)
    else:
        i, j = slice(0, half), slice(half, rot)
    u, v = y[..., i].copy(), y[..., j].copy()
    y[..., i] = u * c - v * s
    y[..., j] = v * c + u * s
    return y


# ------------------------------------------------------------------ pages
class Pages:
    """The page state in plain Python."""

    def __init__(self, refs, table, lens=None):
        self.refs, self.table = [int(r) for r in refs], [[int(e) for e in row] for row in table]
        self.lens = None if lens is None else [int(n) for n in lens]

    def take(self):
        for i, r in enumerate(self.refs):
            if r == 0:
                self.refs[i] = 1
                return i
        return None

    def reserve(self, frm, to):
        for row, f, t in zip(self.table, frm, to):
            if t <= f or f < 0:
                continue
            for e in range(f // BLOCK, min(len(row), -(-t // BLOCK))):
                if row[e] < 0:
                    new = self.take()
                    if new is None:
                        return
                    row[e] = new

    def drop(self, block):
        if 0 <= block < len(self.refs) and self.refs[block] > 0:
            self.refs[block] -= 1

    def release(self, frm, to):
        for row, f, t in zip(self.table, frm, to):
            if f < 0 or f >= t:
                continue
            for e in range(len(row)):
                if e * BLOCK >= f and (e + 1) * BLOCK <= t and row[e] != -1:
                    self.drop(row[e])
                    row[e] = -1

    def fork(self, src, dst):
        """Returns the copies [(from, to)]."""
        pairs = [(i, s, d) for i, (s, d) in enumerate(zip(src, dst)) if s >= 0]
        good, copies = [], []
        n = len(self.table)
        for i, s, d in pairs:
            if not (0 <= s < n and 0 <= d < n) or s == d:
                continue
            if any(j != i and d in (s2, d2) for j, s2, d2 in pairs):
                continue
            L = self.lens[s]
            if not 0 <= L <= len(self.table[s]) * BLOCK:
                continue
            tail = self.table[s][L // BLOCK] if L % BLOCK else None
            if tail is not None and not 0 <= tail < len(self.refs):
                continue
            good.append((s, d, L, tail))
        after = []
        for s, d, L, tail in good:
            fresh = None
            if tail is not None:
                fresh = self.take()
                if fresh is None:
                    continue
                copies.append((tail, fresh))
            after.append((s, d, L, fresh))
        for s, d, L, fresh in after:
            new = self.table[s][:L // BLOCK]
            for b in new:
                if b >= 0:
                    self.refs[b] += 1
            if fresh is not None:
                new = new + [fresh]
            old = self.table[d]
            self.table[d] = new + [-1] * (len(old) - len(new))
            for b in old:
                if b != -1:
                    self.drop(b)
            self.lens[d] = L
        return copies

    def compact(self):
        """Returns the moves [(from, to)]."""
        live = sum(r != 0 for r in self.refs)
        src = [i for i in range(live, len(self.refs)) if self.refs[i] != 0]
        dst = [i for i in range(live) if self.refs[i] == 0]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        self.table = [[to.get(e, e if e < live else -1) for e in row] for row in self.table]
        return list(zip(src, dst))
