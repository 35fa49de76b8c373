"""fp64 definitions of the paged-cache calls and of the logit adjustment.

Written from the formulas in ``include/medusa_b200.h``: rotary positions with
their long-context scalings, attention of new tokens over a paged cache,
compaction of accepted rows inside the pages, and penalties, biases and masks
on the logits of tree nodes.  Plain loops over sequences, heads and nodes.
"""

from __future__ import annotations

import math

import numpy as np


def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_length=4096, beta_fast=32.0, beta_slow=1.0):
    """(radians per position of every pair, amplitude of cos and sin)."""
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling != "yarn":
        return f, 1.0

    def index(turns):
        """The pair (a real number) that makes that many turns over the original length."""
        return rot * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(index(beta_fast)), 0), min(math.ceil(index(beta_slow)), rot - 1)
    out = []
    for i, w in enumerate(f):
        ramp = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        out.append(w / factor * ramp + w * (1 - ramp))
    return np.array(out), 0.1 * math.log(factor) + 1.0


def rotate(x, positions, freq, amplitude, rot, layout):
    """x [N, heads, hd], positions [N]: the first rot dimensions of every head turned by position * freq."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        # the angle modulo a turn, from an exact product of the position and the frequency's high and low parts
        th = np.array([math.fmod(int(p) * float(freq[i]), 2 * math.pi) for p in positions])[:, None]
        c, s = np.cos(th) * amplitude, np.sin(th) * amplitude
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def gather_rows(pages, table_row, count):
    """Rows 0..count-1 of a sequence: pages [n_pages, Hkv, page, hd] -> [Hkv, count, hd]."""
    page = pages.shape[2]
    return np.stack([pages[table_row[r // page], :, r % page] for r in range(count)], 1) if count else \
        np.zeros((pages.shape[1], 0, pages.shape[3]))


def attention(q, k_pages, v_pages, table, lens, starts, scale, sees=None):
    """(out, mass) [N, H, hd]: softmax(scale q.k) v per query row, and the same with |v| (for error bounds).
    sees [T, T]: the tree's visibility, else causal chunks."""
    q = np.asarray(q, dtype=np.float64)
    N, H, hd = q.shape
    Hkv = k_pages.shape[1]
    out, mass = np.zeros((N, H, hd)), np.zeros((N, H, hd))
    for b, L in enumerate(lens):
        n = starts[b + 1] - starts[b]
        if n == 0:
            continue
        K, V = (gather_rows(p, table[b], L + n).astype(np.float64) for p in (k_pages, v_pages))
        for i in range(n):
            new = sees[i] if sees is not None else np.arange(n) <= i
            cols = np.concatenate([np.arange(L), L + np.flatnonzero(new)])
            for e in range(H):
                h = e // (H // Hkv)
                z = scale * (K[h, cols] @ q[starts[b] + i, e])
                p = np.exp(z - z.max())
                p /= p.sum()
                out[starts[b] + i, e] = p @ V[h, cols]
                mass[starts[b] + i, e] = p @ np.abs(V[h, cols])
    return out, mass


def accept(pages, table, lens, retrieve, best, accept_len):
    """pages [layers, n_pages, Hkv, page, hd] after the compaction."""
    out = pages.copy()
    page = pages.shape[3]
    for b, L in enumerate(lens):
        for j in range(accept_len[b] + 1):
            s, d = L + retrieve[best[b]][j], L + j
            out[:, table[b][d // page], :, d % page] = pages[:, table[b][s // page], :, s % page]
    return out


def adjust_logits(logits, tokens, parent, history=None, prompt_lens=None, repetition=None, presence=None, frequency=None,
                  bias=None, allowed=None):
    """logits [B, T, V]; history: a list of tokens per sequence; bias: a list of (id, value) per sequence;
    allowed [B, T, V] truth values."""
    z = np.array(logits, dtype=np.float64)
    B, T, V = z.shape
    for b in range(B):
        hist = list(history[b]) if history is not None else []
        cut = prompt_lens[b] if prompt_lens is not None else 0
        for i in range(T):
            path, node = [], i
            while node >= 0:
                path.append(tokens[b][node])
                node = parent[node]
            seen = [v for v in hist + path if 0 <= v < V]
            made = [v for v in hist[cut:] + path if 0 <= v < V]
            if repetition is not None:
                for v in set(seen):
                    z[b, i, v] = z[b, i, v] / repetition[b] if z[b, i, v] > 0 else z[b, i, v] * repetition[b]
            for v in set(made):
                if frequency is not None:
                    z[b, i, v] -= frequency[b] * made.count(v)
                if presence is not None:
                    z[b, i, v] -= presence[b]
            for v, x in (bias[b] if bias is not None else []):
                if 0 <= v < V:
                    z[b, i, v] += x
    if allowed is not None:
        z = np.where(allowed, z, -np.inf)
    return z
