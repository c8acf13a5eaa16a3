"""Plain CPU oracle of the scored router, its losses and gradients, and the
dropout beside the combine, from the formulas in ``include/moe.h``.

TEST INFRASTRUCTURE: shares no code with the HIP path and imports nothing from
it. Everything is float64 and follows the definitions one row at a time where
that is affordable; arrays are numpy.
"""
from __future__ import annotations

import dataclasses
import math

import numpy as np

__all__ = ["RouteSpec", "scores", "select", "balance_losses", "select_backward", "gate_backward", "philox4x32",
           "keep_mask", "combine_dropout", "dropout_backward"]

F32_MAX = float(np.finfo(np.float32).max)


@dataclasses.dataclass(frozen=True)
class RouteSpec:
    score: str = "softmax"
    groups: int = 1
    topk_groups: int = 1
    group_rule: str = "max"
    renormalise: bool = True
    scale: float = 1.0


def _clean(row):
    """float64 logits of one row; None in the places of -inf and NaN."""
    return [None if (math.isnan(v) or v == -math.inf) else min(float(v), F32_MAX) for v in row]


def scores(row, score):
    """Scores of one row (list of floats, None where out of the choice): sigmoid or softmax over the row."""
    live = [v for v in row if v is not None]
    if score == "sigmoid":
        return [0.0 if v is None else (1.0 / (1.0 + math.exp(-v)) if v >= -700 else math.exp(v)) for v in row]
    if not live:
        return [0.0] * len(row)
    m = max(live)
    z = [0.0 if v is None else math.exp(v - m) for v in row]
    tot = math.fsum(z)
    return [v / tot for v in z]


def select(logits, bias, k, spec: RouteSpec):
    """(topk_idx int32 [T][k], topk_w float64 [T][k]) by the definition."""
    T, E = logits.shape
    per = E // spec.groups
    idx = np.zeros((T, k), np.int32)
    w = np.zeros((T, k), np.float64)
    for t in range(T):
        l = _clean(logits[t])
        s = scores(l, spec.score)
        b = [0.0] * E if bias is None else [float(v) for v in bias]
        ok = [l[e] is not None and not math.isnan(b[e]) and b[e] != -math.inf for e in range(E)]
        c = [s[e] + b[e] if ok[e] else None for e in range(E)]
        if spec.topk_groups < spec.groups:
            gk = []
            for g in range(spec.groups):
                m = sorted((c[e] for e in range(g * per, (g + 1) * per) if ok[e]), reverse=True)
                gk.append(-math.inf if not m else (sum(m[:2]) if spec.group_rule == "top2" else m[0]))
                if not m:
                    gk[-1] = None
            order = sorted(range(spec.groups), key=lambda g: (gk[g] is None, -gk[g] if gk[g] is not None else 0.0, g))
            kept = set(order[:spec.topk_groups])
            ok = [ok[e] and e // per in kept for e in range(E)]
        live = sorted((e for e in range(E) if ok[e]), key=lambda e: (-c[e], -l[e], e))
        dead = [e for e in range(E) if not ok[e]]
        chosen = (live + dead)[:k]
        n = min(k, len(live))
        idx[t] = chosen
        if spec.renormalise and n:
            # ratios of scores, scaled so that none underflows: log s = l - log(1 + e^l), or l
            ls = [l[e] - (math.log1p(math.exp(l[e])) if l[e] < 30 else l[e]) if spec.score == "sigmoid" else l[e]
                  for e in chosen[:n]]
            z = [math.exp(v - max(ls)) for v in ls]
            w[t, :n] = [spec.scale * v / math.fsum(z) for v in z]
        else:
            w[t, :n] = [spec.scale * s[e] for e in chosen[:n]]
    return idx, w


def _shares(l, spec):
    """s_e / sum s of one cleaned row, without underflow."""
    if spec.score == "softmax":
        return scores(l, "softmax")
    live = [v for v in l if v is not None]
    if not live:
        return [0.0] * len(l)
    ls = [None if v is None else v - (math.log1p(math.exp(v)) if v < 30 else v) for v in l]
    m = max(v for v in ls if v is not None)
    z = [0.0 if v is None else math.exp(v - m) for v in ls]
    tot = math.fsum(z)
    return [v / tot for v in z]


def _lse(l):
    live = [v for v in l if v is not None]
    if not live:
        return None
    m = max(live)
    return m + math.log(math.fsum(math.exp(v - m) for v in live))


def balance_losses(logits, idx, seqs, spec: RouteSpec):
    """(losses [2], load [S][E]) for sequences seqs = offsets [S+1]."""
    T, E = logits.shape
    k = idx.shape[1]
    S = len(seqs) - 1
    load = np.zeros((S, E), np.int64)
    bal, filled, z, covered = 0.0, 0, 0.0, 0
    for s in range(S):
        a, b = seqs[s], seqs[s + 1]
        if b <= a:
            continue
        P = np.zeros(E)
        for t in range(a, b):
            for e in idx[t]:
                if 0 <= e < E:
                    load[s, e] += 1
            l = _clean(logits[t])
            P += np.array(_shares(l, spec))
            v = _lse(l)
            z += 0.0 if v is None else v * v
        n = b - a
        bal += E / (k * n * n) * float(np.dot(load[s], P))
        filled += 1
        covered += n
    return np.array([bal / filled if filled else 0.0, z / covered if covered else 0.0]), load


def select_backward(logits, idx, w, dw, spec: RouteSpec, dlosses=None, load=None, seqs=None):
    """dlogits [T][E] by the chain rule; w: the selection's weights (0 = slot out of the choice)."""
    T, E = logits.shape
    out = np.zeros((T, E))
    if dlosses is not None:
        S = len(seqs) - 1
        filled = sum(1 for s in range(S) if seqs[s + 1] > seqs[s])
        covered = max(0, seqs[S] - seqs[0])
    for t in range(T):
        l = _clean(logits[t])
        s = scores(l, spec.score)
        one_minus = [0.0 if v is None else scores([-v], "sigmoid")[0] for v in l]
        if dw is not None:
            k = idx.shape[1]
            on = [j for j in range(k) if w[t, j] != 0 and 0 <= idx[t, j] < E]
            D = math.fsum(w[t, j] * dw[t, j] for j in range(k) if w[t, j] != 0)
            for j in on:
                e = idx[t, j]
                g = w[t, j] * (dw[t, j] - (D / spec.scale if spec.renormalise else 0.0))
                out[t, e] += g * (one_minus[e] if spec.score == "sigmoid" else 1.0)
            if spec.score == "softmax" and not spec.renormalise:
                out[t] -= np.array(s) * D
        if dlosses is not None:
            sid = next((q for q in range(S) if seqs[q] <= t < seqs[q + 1]), None)
            if sid is None or all(v is None for v in l):
                continue
            n = seqs[sid + 1] - seqs[sid]
            k = idx.shape[1]
            g = dlosses[0] * E / (k * n * n * filled) * load[sid].astype(np.float64)
            q = np.array(_shares(l, spec))
            d = q * (g - float(np.dot(q, g)))
            if spec.score == "sigmoid":
                d = d * np.array(one_minus)
            out[t] += d + dlosses[1] * 2.0 * _lse(l) / covered * np.array(scores(l, "softmax"))
    return out


def gate_backward(x, wg, dl, dx_in=None):
    """(dx, dwg, dbias) in float64."""
    x, wg, dl = (np.asarray(v, np.float64) for v in (x, wg, dl))
    dx = dl @ wg
    if dx_in is not None:
        dx = dx + np.asarray(dx_in, np.float64)
    return dx, dl.T @ x, dl.sum(axis=0)


def philox4x32(counter, key, rounds=10):
    """Philox4x32 (Salmon et al., SC 2011) of one counter (4 words) and key (2 words), in Python integers."""
    c, k, M = list(counter), list(key), 2 ** 32
    for _ in range(rounds):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b // M) ^ c[1] ^ k[0], b % M, (a // M) ^ c[3] ^ k[1], a % M]
        k = [(k[0] + 0x9E3779B9) % M, (k[1] + 0xBB67AE85) % M]
    return c


def keep_mask(n, seed, offset, p):
    """Keep decisions of elements 0 .. n-1 (bool)."""
    thr = round(p * 65536)
    seed, offset = seed % 2 ** 64, offset % 2 ** 64  # the 64 bits of a signed value
    out = np.zeros(n, bool)
    for i in range((n + 7) // 8):
        words = philox4x32([i % 2 ** 32, i >> 32, offset % 2 ** 32, offset >> 32], [seed % 2 ** 32, seed >> 32])
        for j in range(8):
            if 8 * i + j < n:
                out[8 * i + j] = ((words[j // 2] >> (16 * (j % 2))) & 0xFFFF) >= thr
    return out


def _scale(p):
    thr = round(p * 65536)
    return 65536.0 / (65536 - thr) if thr < 65536 else 0.0


def combine_dropout(y, inv, w, residual, seed, offset, p):
    T, k = w.shape
    d = y.shape[1]
    s = np.zeros((T, d))
    for j in range(k):
        s += w[:, j:j + 1].astype(np.float64) * y[inv.reshape(T, k)[:, j]].astype(np.float64)
    keep = keep_mask(T * d, seed, offset, p).reshape(T, d)
    out = np.where(keep, s * _scale(p), 0.0)
    return out if residual is None else out + residual.astype(np.float64)


def dropout_backward(dout, seed, offset, p):
    keep = keep_mask(dout.size, seed, offset, p).reshape(dout.shape)
    return np.where(keep, dout.astype(np.float64) * _scale(p), 0.0)
