"""The serving operators in fp64 on the CPU: rotation and append, attention of
packed prompts and of single tokens over a paged cache, logits processing.

Plain definitions; values the operators store in 16 bits are not rounded here
(the tests' tolerances count those roundings).  Each attention also returns
what its tolerance needs: the mean of |v| under the probabilities and the
largest sum of |q_i k_i| a query meets.
"""
import math

import torch


def rows(pages, table, n, page_size):
    """The first n cached rows of one sequence, [n][Hkv][D] (pages: [n_pages][Hkv][page_size][D])."""
    out = [pages[int(table[t // page_size]), :, t % page_size] for t in range(n)]
    return torch.stack(out) if out else pages.new_zeros((0, pages.shape[1], pages.shape[3]))


def attend(q, k, v, limit, scale):
    """q [n][Hq][D], k and v [m][Hkv][D]; query i sees keys j < limit[i].  Rows without keys are zero.
    Returns (out, mean |v|, largest sum |q_i k_i|), the last [n][Hq][1]."""
    n, hq, d = q.shape
    m, hkv = k.shape[:2]
    out = torch.zeros((n, hq, d), dtype=torch.float64)
    mag = torch.zeros_like(out)
    big = torch.zeros((n, hq, 1), dtype=torch.float64)
    q, k, v = q.double(), k.double(), v.double()
    for i in range(n):
        see = max(0, min(m, int(limit[i])))
        if see == 0:
            continue
        for h in range(hq):
            g = h // (hq // hkv)
            s = k[:see, g] @ q[i, h] * scale
            p = torch.exp(s - s.max())
            p = p / p.sum()
            out[i, h] = p @ v[:see, g]
            mag[i, h] = p @ v[:see, g].abs()
            big[i, h] = (k[:see, g].abs() @ q[i, h].abs()).max() * scale
    return out, mag, big


def rotate(x, pos, theta):
    """x [n][H][D] at positions pos [n]: pair (p, p + D/2) turned by pos * theta^(-2p/D)."""
    d = x.shape[-1]
    x = x.double()
    if not theta:
        return x
    out = torch.empty_like(x)
    for p in range(d // 2):
        a = torch.as_tensor(pos, dtype=torch.float64) * theta ** (-2.0 * p / d)
        c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
        out[..., p] = x[..., p] * c - x[..., p + d // 2] * s
        out[..., p + d // 2] = x[..., p + d // 2] * c + x[..., p] * s
    return out


def process(logits, history=None, history_lens=None, prompt_lens=None, repetition=None, frequency=None, presence=None,
            bias=None, mask=None):
    """(x [rows][vocab] fp64, the chosen id of each row by the definition in include/mk.h)."""
    x = logits.double().clone()
    R, V = x.shape
    best = []
    for r in range(R):
        if history is not None:
            n = history.shape[1] if history_lens is None else min(max(int(history_lens[r]), 0), history.shape[1])
            first = 0 if prompt_lens is None else int(prompt_lens[r])
            every, said = {}, {}
            for i, v in enumerate(history[r, :n].tolist()):
                if 0 <= v < V:
                    every[v] = every.get(v, 0) + 1
                    said[v] = said.get(v, 0) + (i >= first)
            for v in every:
                if repetition is not None:
                    rep = float(repetition[r])
                    x[r, v] = x[r, v] / rep if x[r, v] > 0 else x[r, v] * rep
                if said[v]:
                    x[r, v] -= (float(frequency[r]) * said[v] if frequency is not None else 0.0)
                    x[r, v] -= (float(presence[r]) if presence is not None else 0.0)
        if bias is not None:
            for i in range(int(bias[0][r]), int(bias[0][r + 1])):
                if 0 <= int(bias[1][i]) < V:
                    x[r, int(bias[1][i])] += float(bias[2][i])
        if mask is not None:
            row = mask[r if mask.shape[0] > 1 else 0].long()
            bits = (row[:, None] >> torch.arange(32)) & 1  # bit v % 32 of word v // 32
            x[r, bits.reshape(-1)[:V] == 0] = -math.inf
        choice, top = -1, -math.inf
        for v, value in enumerate(x[r].tolist()):
            if value > top:  # (a NaN is never larger)
                choice, top = v, value
        best.append(choice)
    return x, torch.tensor(best, dtype=torch.int32)
