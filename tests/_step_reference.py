"""The serving-step operators' definitions in 64 bits on the CPU, for the tests."""
import numpy as np
import torch


class Pool:
    """A page pool as plain Python lists (what step_tables / trim_pages keep on the device)."""

    def __init__(self, seq_lens, page_table, free_pages, num_free, bs):
        self.lens, self.table = [int(x) for x in seq_lens], [list(map(int, r)) for r in page_table]
        self.free, self.nf, self.bs = list(map(int, free_pages)), int(num_free), bs

    def _entries(self, rows):
        """(row, usable) of each entry: in range, a valid length, not named before."""
        M, seen, out = len(self.table[0]), set(), []
        for r in rows:
            r = int(r)
            ok = 0 <= r < len(self.lens) and 0 <= self.lens[r] <= M * self.bs
            out.append((r, ok and r not in seen, ok))
            if ok:
                seen.add(r)
        return out

    def grow(self, rows, new, T):
        bs, M = self.bs, len(self.table[0])
        nf0, cum, tokens, taken = self.nf, 0, 0, 0
        lens0 = list(self.lens)                # a row named twice: both entries see the length before the step
        bt, slots, pos, cu_q, cu_k, after_l, before_l = [], [-1] * T, [0] * T, [0], [0], [], []
        for (r, mine, valid), n in zip(self._entries(rows), map(int, new)):
            n = max(n, 0)
            start, tokens = tokens, tokens + n
            length = lens0[r] if valid else 0
            old, want = -(-length // bs), -(-(length + n) // bs)
            ok = mine and tokens <= T and want <= M
            need = want - old if ok else 0
            cum += need
            if need and cum > nf0:
                ok = False
            pages = list(self.table[r][:old]) if valid else []
            if ok:
                pages += [self.free[nf0 - 1 - (cum - need) - i] for i in range(need)]
                if need:
                    taken = max(taken, cum)
                    self.table[r][old:want] = pages[old:]
            after = length + n if ok else length
            if mine:
                self.lens[r] = after
            bt.append((pages + [-1] * M)[:M])
            for i in range(n):
                if start + i < T:
                    p = length + i
                    pos[start + i] = p
                    slots[start + i] = pages[p // bs] * bs + p % bs if ok else -1
            cu_q.append(min(tokens, T))
            cu_k.append(cu_k[-1] + after)
            after_l.append(after)
            before_l.append(length)
        self.nf = nf0 - taken
        return dict(block_table=bt, slot_mapping=slots, positions=pos, cu_seqlens_q=cu_q, cu_seqlens_k=cu_k,
                    cache_seqlens=after_l, context_lens=before_l)

    def trim(self, rows, keep):
        bs, back, room = self.bs, [], len(self.free) - self.nf
        for (r, mine, _), k in zip(self._entries(rows), map(int, keep)):
            if not mine:
                continue
            after = min(max(k, 0), self.lens[r])
            old, kept = -(-self.lens[r] // bs), -(-after // bs)
            if old > kept and len(back) + old - kept > room:
                room = -1                      # this and every later release is refused
                continue
            back += self.table[r][kept:old]
            self.table[r][kept:old] = [-1] * (old - kept)
            self.lens[r] = after
        for p in reversed(back):
            self.free[self.nf] = p
            self.nf += 1


def rope(x, positions, inv_freq, pair_axis, interleaved, scale):
    """x [N, H, D] rotated, float64."""
    y = x.double().clone()
    half = inv_freq.numel()
    pos = positions.double().reshape(-1, x.shape[0])
    axis = [0] * half if pair_axis is None else list(pair_axis)
    ang = torch.stack([pos[a] for a in axis], 1) * inv_freq.double()          # [N, half]
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    if interleaved:
        a, b = y[..., 0:2 * half:2].clone(), y[..., 1:2 * half:2].clone()
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = scale * (a * c - b * s), scale * (a * s + b * c)
    else:
        a, b = y[..., :half].clone(), y[..., half:2 * half].clone()
        y[..., :half], y[..., half:2 * half] = scale * (a * c - b * s), scale * (a * s + b * c)
    return y


def linear(q, k, v, g, cu, scale, starts):
    """Token after token.  starts: per sequence a float64 [Hkv, D, D] state or None.
    Returns (out, final states, weight): weight is scale * the sum of the absolute values of
    every term of an output, what a relative error of the terms is measured by."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    q, k, v = q.double(), k.double(), v.double()
    a = torch.exp(g.double().clamp(max=0))
    out, weight, finals = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64), []
    for b in range(len(cu) - 1):
        S = torch.zeros(Hkv, D, D, dtype=torch.float64) if starts[b] is None else starts[b].clone()
        A = S.abs()
        for t in range(int(cu[b]), int(cu[b + 1])):
            S = a[:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
            A = a[:, None, None] * A + v[t].abs()[:, :, None] * k[t].abs()[:, None, :]
            qg = q[t].view(Hkv, G, D)
            out[t] = scale * torch.einsum("hvk,hgk->hgv", S, qg).reshape(Hq, D)
            weight[t] = scale * torch.einsum("hvk,hgk->hgv", A, qg.abs()).reshape(Hq, D)
        finals.append((S, A))
    return out, finals, weight


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
