"""Plain fp64 CPU oracle for the quantized key/value cache and the attention over it.

TEST INFRASTRUCTURE ONLY, like gptq_oracle: only the tests may import it. It shares no code with
the CUDA library.

Sources (web pages, cited by title and section):
  [BLOG]  "GPTQ second-order quantization" blog: "Group-wise quantization" (one scale and zero point
          per group of values).

Readings taken (the pages have no cache):
  * The grid of a group is the layer quantizer's asymmetric min/max grid with its step rounded up to
    bfloat16: lo = min(0, min x), hi = max(0, max x), step = (hi - lo) / (2^bits - 1) (0: lo = -1,
    hi = 1), s = step rounded up to bf16, z = clamp(rint(-lo / s)), q = clamp(rint(x / s) + z), each
    step rounded once in float32. A value that is not finite, or a step that is not, gives the group
    a NaN scale and zero codes.
  * Codes of a row are packed like the weights': code d in bits bits * (d mod (32 / bits)) of word
    d // (32 / bits).
  * Attention of one query over tokens t: sum_t w_t v_t / sum_t w_t with w_t = exp(scale q . k_t),
    taken in fp64; no tokens give 0.
"""
from __future__ import annotations

import numpy as np


def bf16_up(x: np.ndarray) -> np.ndarray:
    """Positive float32 numbers rounded up to bfloat16 (as float32)."""
    bits = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return (((bits + 0xFFFF) >> 16) << 16).astype(np.uint32).view(np.float32)


def grid_quantize(x: np.ndarray, bits: int, group: int):
    """float32 x [..., dim] -> (codes uint8 [..., dim], scales float32 [..., dim / group] holding
    bf16 values, zeros uint8 [..., dim / group])."""
    x = np.asarray(x, np.float32)
    v = x.reshape(*x.shape[:-1], -1, group)
    top = np.float32(2 ** bits - 1)
    with np.errstate(all="ignore"):
        good = np.isfinite(v).all(-1)
        safe = np.where(good[..., None], v, np.float32(0))
        lo = np.minimum(safe.min(-1), np.float32(0))
        hi = np.maximum(safe.max(-1), np.float32(0))
        step = (hi - lo) / top
        flat = step == 0
        lo = np.where(flat, np.float32(-1), lo)
        step = np.where(flat, np.float32(2) / top, step)
        s = bf16_up(step)
        good &= np.isfinite(s)
        s = np.where(good, s, np.float32(1))
        z = np.clip(np.rint(-lo / s), 0, top)
        q = np.clip(np.rint(safe / s[..., None]) + z[..., None], 0, top)
    s = np.where(good, s, np.float32(np.nan))
    z = np.where(good, z, 0)
    q = np.where(good[..., None], q, 0)
    return q.reshape(x.shape).astype(np.uint8), s, z.astype(np.uint8)


def pack_rows(codes: np.ndarray, bits: int) -> np.ndarray:
    """uint8 codes [..., dim] -> uint32 words [..., dim * bits / 32]."""
    per = 32 // bits
    c = np.asarray(codes, np.uint32).reshape(*codes.shape[:-1], -1, per)
    words = np.zeros(c.shape[:-1], np.uint32)
    for i in range(per):
        words |= c[..., i] << np.uint32(bits * i)
    return words


def values(codes: np.ndarray, scales: np.ndarray, zeros: np.ndarray) -> np.ndarray:
    """s (q - z) in fp64."""
    group = codes.shape[-1] // scales.shape[-1]
    q = codes.astype(np.float64).reshape(*scales.shape, group)
    v = scales.astype(np.float64)[..., None] * (q - zeros.astype(np.float64)[..., None])
    return v.reshape(codes.shape)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float) -> np.ndarray:
    """One query [dim] over keys and values [tokens, dim], fp64."""
    if k.shape[0] == 0:
        return np.zeros(v.shape[-1])
    x = (k @ q.astype(np.float64)) * scale
    w = np.exp(x - x.max())
    return (w @ v) / w.sum()


def attend_bound(q, kc, ks, kz, vc, vs, vz, scale: float, image16: bool = False,
                 many_rows: bool = False):
    """One query [dim] over cached tokens: (the result, a bound on the error of a bf16 result of it),
    per dimension, for a kernel with fp32 sums and fp16 operands. The arithmetic written out, nothing
    measured. kc, vc: codes [tokens, dim]; ks, kz, vs, vz: their grids [tokens, groups].

    * The sums q . code take dim / 16 + 8 steps, each off by 2^-22 of the magnitudes it adds: x_t
      moves by (dim / 16 + 8) 2^-22 A_t, A_t = scale sum_groups s (sum |q| code + z sum |q|), or
      with `many_rows`, where the sums are those of q (code - z), A_t = scale sum |q k|. The score,
      the largest one, the logarithm of a scale and their differences are fp32 numbers: 2^-22 of
      their magnitudes. The exponential and the products around it add 2^-20. With `image16` the
      keys are fp16 images of s (code - z), off by 2^-12 each: x_t moves by 2^-12 scale sum |q k|
      more. Relative errors e_t of the weights move the result by sum p_t e_t |v_t - out| to first
      order, the rest being max e of that.
    * The operand of a token's weight is w s, per group of dimensions, rounded to fp16: by 2^-12 of
      itself, or by 2^-25 of a unit in which w S times the group's largest s / S is at least 2^6, S
      being a token's largest scale. A group of a token's values that are all zero does not count.
      With `image16` each value is an image too, off
      by 2^-12 of itself or 2^-32 of the largest (key images likewise), and one unit holds for all
      groups of a token. With `many_rows` (a shared prefix's own kernel) the values are images, off
      by 2^-12 of themselves or 2^-32 of the largest of their 32 tokens (their own where that one is
      2^13 and more above them), which the unit goes by, too; and where a row has several grids the
      keys are sums of two images, off by 2^-32 of the largest of their 32 tokens.
    * The sum over tokens runs in steps of 16 and is joined from parts: (tokens / 16 + 64) 2^-22 of
      sum p |v|. Each step adds codes and takes zero points out: 2^-22 of sum p s (code + z) more.
      A code enters as an fp16 subnormal, which the tensor core aligns as if it were 2^-14, that is
      2^10 codes: each of a step's 16 products is cut at 2^-24 of that and the step's largest
      weight, 16 * 2^-14 sum over steps of max p s. With `many_rows` the operands are normal.
    * The result is rounded to bf16: half a step, 2^-8 of the value that is rounded.
    """
    T, dim = kc.shape
    if T == 0:
        return np.zeros(dim), np.zeros(dim)
    G = ks.shape[1]
    q = q.astype(np.float64)
    k, v = values(kc, ks, kz), values(vc, vs, vz)
    x = (k @ q) * scale
    p = np.exp(x - x.max())
    p /= p.sum()
    out, mass = p @ v, p @ np.abs(v)
    aq = np.abs(q).reshape(G, -1)
    kq = scale * (np.abs(k) @ np.abs(q))
    if many_rows:
        A = kq
    else:
        A = scale * (ks.astype(np.float64) *
                     (np.einsum("tgd,gd->tg", kc.astype(np.float64).reshape(T, G, -1), aq) +
                      kz * aq.sum(-1))).sum(1)
    steps = (T / 16 + 64) * 2.0 ** -22
    logs = np.abs(np.log2(vs[vs > 0].astype(np.float64))).max() if (vs > 0).any() else 0.0
    e = (dim / 16 + 8) * 2.0 ** -22 * A + 2.0 ** -20 + \
        2.0 ** -22 * (np.abs(x) + np.abs(x.max()) + logs)
    if image16:
        e = (dim / 16 + 8) * 2.0 ** -22 * A.max() + 2.0 ** -20
        e += 2.0 ** -12 * kq.max() + 2.0 ** -32 * scale * np.abs(k).max() * np.abs(q).sum()
        bound = mass * (2 * e + 2.0 ** -11 + steps) + \
            2.0 ** -25 * p.max() * np.abs(v).sum(0) + 2.0 ** -32 * np.abs(v).max()
    else:
        z = np.repeat(vz.astype(np.float64), dim // G, 1)
        d = np.abs(vc - z)
        live_s = np.where(d.reshape(T, G, -1).any(-1), vs.astype(np.float64), 0.0)
        ps, top_s = p[:, None] * live_s, live_s.max(1)
        some = top_s > 0
        share = (live_s[some] / top_s[some, None]).max(0) if some.any() else np.zeros(G)
        unit = (p * top_s).max() * share                              # per group
        sums = np.einsum("tg,tgd->gd", ps, (vc + z).reshape(T, G, -1)).reshape(-1)
        def blocks(top):      # the largest of each token's 32, at most 2^13 times its own
            most = np.pad(top, (0, -T % 32)).reshape(-1, 32).max(1).repeat(32)[:T]
            return np.minimum(most, 2.0 ** 13 * top)
        if many_rows:
            if G > 1:
                tops = np.pad(np.abs(k).max(1), (0, -T % 32)).reshape(-1, 32).max(1).repeat(32)[:T]
                e += 2.0 ** -32 * scale * tops * np.abs(q).sum()
            bound = (p * e) @ np.abs(v - out) * (1 + 2 * (p * e).sum() + e[p > 2.0 ** -20].max())
        else:
            bound = 2 * e.max() * mass
        bound += mass * (2.0 ** -12 + steps) + 2.0 ** -22 * sums
        if not many_rows:
            step = np.pad(ps, ((0, -T % 16), (0, 0))).reshape(-1, 16, G).max(1)
            bound += 2.0 ** -10 * np.repeat(step.sum(0), dim // G)
        if many_rows:
            top = blocks(np.abs(v).max(1))
            live = top > 0
            bound += 2.0 ** -12 * mass + 2.0 ** -32 * (p @ top) + 2.0 ** -30 * (p * top).max() * \
                (np.abs(v)[live] / top[live, None]).sum(0)
        else:
            bound += 2.0 ** -31 * np.repeat(unit, dim // G) * d.sum(0)
    return out, bound + 2.0 ** -8 * (np.abs(out) + bound)
