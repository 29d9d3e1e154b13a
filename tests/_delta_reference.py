"""The gated delta rule and beam search in 64 bits on the CPU, for the tests."""
import math

import torch


def delta(q, k, v, g, beta, cu, scale, starts, eps=None):
    """Token after token.  starts: per sequence a float64 [Hv, D, D] state or None.

    Returns (out, final states, reach): with keys no longer than 1 and beta in [0, 1] a
    step never lengthens a row s of a state by more than what it writes,
        |s_t| <= a |s_{t-1}| + beta |v_t| |k_t| =: M_t  (per head and value dimension),
    and it carries an error of the state on no larger.  So errors of at most e M_t in
    every step add up to e E_t, E_t = a E_{t-1} + M_t, in a row's length and
    thereby in each of its elements, and to scale |q_t| e E_t in an output.  reach holds
    scale |q| M and scale |q| E per output, finals (S, E) per sequence."""
    T, Hk, D = q.shape
    Hv = v.shape[1]
    q, k, v, g, beta = (x.double() for x in (q, k, v, g, beta))
    if eps is not None:
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + eps) for x in (q, k))
    q, k = (x.repeat_interleave(Hv // Hk, 1) for x in (q, k))
    a = torch.exp(g.clamp(max=0))
    out = torch.zeros(T, Hv, D, dtype=torch.float64)
    rm, re, finals = torch.zeros_like(out), torch.zeros_like(out), []
    for b in range(len(cu) - 1):
        S = torch.zeros(Hv, D, D, dtype=torch.float64) if starts[b] is None else starts[b].clone()
        M = S.norm(dim=-1)
        E = torch.zeros_like(M)
        for t in range(int(cu[b]), int(cu[b + 1])):
            S = a[t][:, None, None] * S
            u = beta[t][:, None] * (v[t] - torch.einsum("hvk,hk->hv", S, k[t]))
            S = S + u[:, :, None] * k[t][:, None, :]
            M = a[t][:, None] * M + beta[t].abs()[:, None] * v[t].abs() * k[t].norm(dim=-1, keepdim=True)
            E = a[t][:, None] * E + M
            out[t] = scale * torch.einsum("hvk,hk->hv", S, q[t])
            reach = scale * q[t].norm(dim=-1, keepdim=True)
            rm[t], re[t] = reach * M, reach * E
        finals.append((S, E))
    return out, finals, (rm, re)


def select(logits, scores, W, k):
    """(tokens, parents, scores): one candidate after the other."""
    N, V = logits.shape
    x = logits.double()
    tokens, parents, best = [], [], []
    for r in range(N // W):
        cand = []
        for b in range(W):
            row, s = x[r * W + b], float(scores[r * W + b])
            top = row.max().item()
            if not math.isfinite(s) or not math.isfinite(top) or bool(row.isnan().any()):
                continue
            norm = top + math.log(float(torch.exp(row - top).sum()))
            order = torch.sort(row, descending=True, stable=True).indices[:k].tolist()
            cand += [(-(s + (float(row[t]) - norm)), b, i, t) for i, t in enumerate(order) if row[t] > -math.inf]
        cand.sort()
        cand = [(t, b, -m) for m, b, _, t in cand[:k]] + [(-1, -1, -math.inf)] * (k - len(cand))
        for to, i in ((tokens, 0), (parents, 1), (best, 2)):
            to.append([c[i] for c in cand])
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(parents, dtype=torch.int32), torch.tensor(
        best, dtype=torch.float64)


def beam_rows(parents, rows):
    new, source = [], []
    for p, r in zip(parents.tolist(), rows.tolist()):
        W = len(p)
        spare = [r[w] for w in range(W) if w not in p]
        n, s, seen = [], [], set()
        for x in p:
            if 0 <= x < W and x not in seen:
                seen.add(x)
                n.append(r[x])
                s.append(-1)
            else:
                n.append(spare.pop(0))
                s.append(r[x] if 0 <= x < W else -1)
        new.append(n)
        source.append(s)
    return torch.tensor(new, dtype=torch.int32), torch.tensor(source, dtype=torch.int32)
