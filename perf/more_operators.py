"""Measured cases of the gated delta rule and of beam search.

A model whose linear layers follow the gated delta rule runs its prompts in chunks
(delta_attn_varlen_fwd) and its decode steps one token, or a few guessed ones, per
sequence (delta_attn_varlen_fwd with short sequences, delta_attn_decode), on the fp32
state cache that linear attention uses.  A beam search on top of it picks each
request's next tokens from the step's logits (beam_select), hands the beams' request
rows on to their successors (beam_rows), and copies the states and the cached keys and
values of beams that are continued more than once (copy_states, copy_kvcache).

Each operator is here in plain torch operations (own = False) and as the call a user
makes (own = True).
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # sixteen packed prompts of mixed length, some continuing from a cached state
        dict(name="delta_prompts_16", op="delta", B=16, lo=200, hi=4096, Hk=16, Hv=32, D=128, ctx=True, norm=True),
        # one long prompt: little parallelism over sequences
        dict(name="delta_long_32768", op="delta", B=1, lo=32768, hi=32768, Hk=16, Hv=16, D=128, ctx=False, norm=True),
        # many short odd prompts, four value heads to a key head, head_dim 64, keys normalised before
        dict(name="delta_short_96_d64", op="delta", B=96, lo=1, hi=150, Hk=4, Hv=16, D=64, ctx=True, norm=False),
        # a decode step with four guessed tokens behind the last one of 64 sequences
        dict(name="delta_guess_64x5", op="delta", B=64, lo=5, hi=5, Hk=16, Hv=32, D=128, ctx=True, norm=True),
        # one sequence's next token: latency only
        dict(name="delta_step_1", op="delta_step", B=1, Hk=16, Hv=32, D=128, norm=True),
        # a decode step of 256 sequences: the fp32 states are read and written once
        dict(name="delta_step_256", op="delta_step", B=256, Hk=16, Hv=32, D=128, norm=True),
        # one request with four beams: latency only
        dict(name="beam_select_1x4", op="select", R=1, W=4, V=32000, k=8, bf16=True, masked=False),
        # 64 requests of eight beams over a large vocabulary, bf16 logits, twice as many candidates as beams
        dict(name="beam_select_64x8", op="select", R=64, W=8, V=131072, k=16, bf16=True, masked=False),
        # odd sizes, fp32 logits, part of the vocabulary masked
        dict(name="beam_select_21x3_fp32", op="select", R=21, W=3, V=50021, k=6, bf16=False, masked=True),
        # one request's beams go on: latency only
        dict(name="beam_reorder_1x4", op="reorder", R=1, W=4, Hv=32, D=128, Hkv=8, Da=128, bs=256, prompt=400,
             made=37, v16=False),
        # 32 requests of eight beams: their states, and 300 cached tokens behind a shared prompt
        dict(name="beam_reorder_32x8", op="reorder", R=32, W=8, Hv=32, D=128, Hkv=8, Da=128, bs=256, prompt=1000,
             made=300, v16=False),
        # small pages and heads, an fp16 V / 16 cache beside the others
        dict(name="beam_reorder_13x5_d64", op="reorder", R=13, W=5, Hv=6, D=64, Hkv=2, Da=64, bs=16, prompt=77,
             made=90, v16=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta", "delta_step", "select", "select", "reorder"])
    if op == "delta" or op == "delta_step":
        D = rng.choice([64, 128])
        Hk = rng.choice([1, 2, 4, 8, 16])
        Hv = Hk * (rng.choice([1, 1, 2, 3, 4]) if Hk <= 8 else rng.choice([1, 2]))
        norm = rng.choice([False, True])
        if op == "delta_step":
            return dict(op=op, B=_log(rng, 1, 256), Hk=Hk, Hv=Hv, D=D, norm=norm)
        B = _log(rng, 1, 64)
        hi = _log(rng, 2, max(3, 16384 // B))
        return dict(op=op, B=B, lo=max(1, hi // rng.choice([1, 2, 20])), hi=hi, Hk=Hk, Hv=Hv, D=D,
                    ctx=rng.choice([False, True]), norm=norm)
    W = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if op == "select":
        R = _log(rng, 1, 256 // W)
        return dict(op=op, R=R, W=W, V=_log(rng, 1000, 150000), k=min(32, W * rng.choice([1, 2])),
                    bf16=rng.choice([False, True]), masked=rng.choice([False, True]))
    W = max(W, 2)
    D = rng.choice([64, 128])
    return dict(op=op, R=_log(rng, 1, 256 // W), W=W, Hv=rng.choice([2, 6, 16]), D=D, Hkv=rng.choice([1, 2, 8]),
                Da=rng.choice([64, 128]), bs=rng.choice([16, 64, 256]), prompt=_log(rng, 1, 1000),
                made=_log(rng, 1, 300), v16=rng.choice([False, True]))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _lens(case):
    # the lengths belong to the case: the packed tensors have one shape for every seed
    g = torch.Generator().manual_seed(29 + case["B"] + case["hi"])
    return torch.randint(case["lo"], case["hi"] + 1, (case["B"],), generator=g).tolist()


def prepare(case, seed):
    return {"delta": _prep_delta, "delta_step": _prep_delta, "select": _prep_select,
            "reorder": _prep_reorder}[case["op"]](case, seed)


EPS = 1e-6


def _prep_delta(c, seed):
    """Packed projections of a layer: q, k and v as views of one tensor, a decay and a write strength per token
    and value head."""
    g = _gen(seed)
    step = c["op"] == "delta_step"
    B, Hk, Hv, D = c["B"], c["Hk"], c["Hv"], c["D"]
    lens = [1] * B if step else _lens(c)
    T = sum(lens)
    qkv = _randn(g, T, 2 * Hk + Hv, D)
    if not c["norm"]:
        qkv[:, :2 * Hk] /= qkv[:, :2 * Hk].norm(dim=-1, keepdim=True)
    qkv = qkv.to(torch.bfloat16)
    # decays of a few to a few thousand tokens of memory over the heads, and tokens that reset the state
    rate = torch.exp(torch.linspace(math.log(1e-3), math.log(1.0), Hv, device=DEV))
    decay = -rate * torch.log1p(torch.exp(_randn(g, T, Hv) + 0.5))
    decay = torch.where(torch.rand(T, Hv, generator=g, device=DEV) < 0.002, decay - 30.0, decay)
    beta = 1 / (1 + torch.exp(-1.5 * _randn(g, T, Hv)))
    cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)
    state = _randn(g, B + 3, Hv, D, D) * 0.3
    slots = torch.randperm(B + 3, generator=g, device=DEV)[:B].to(torch.int32)
    ctx = None
    if not step and c["ctx"]:
        # a decode step's sequences all continue, prompts in part
        ctx = torch.full((B,), 100, device=DEV) if c["hi"] <= 16 else torch.arange(B, device=DEV) % 2 * 100
        ctx = ctx.to(torch.int32)
    return dict(c=c, q=qkv[:, :Hk], k=qkv[:, Hk:2 * Hk], v=qkv[:, 2 * Hk:], decay=decay, beta=beta, cu=cu,
                max_len=max(lens), state=state, slots=slots, ctx=ctx, scale=1.0 / math.sqrt(D),
                out=torch.empty(T, Hv, D, dtype=torch.bfloat16, device=DEV), ws=None)


def _prep_select(c, seed):
    g = _gen(seed)
    N, V = c["R"] * c["W"], c["V"]
    logits = _randn(g, N, V) * 2.5
    if c["masked"]:   # tokens that a grammar or a vocabulary mask rules out
        logits.masked_fill_(torch.rand(N, V, generator=g, device=DEV) < 0.3, -math.inf)
    # a few likely tokens per row, as a trained model has them
    likely = torch.randint(0, V, (N, 6), generator=g, device=DEV)
    logits.scatter_(1, likely, 9 + 2 * _randn(g, N, 6))
    logits = logits.to(torch.bfloat16 if c["bf16"] else torch.float32)
    scores = -20 - torch.rand(N, generator=g, device=DEV) * 3
    return dict(c=c, logits=logits, scores=scores, ws=None, kept=None)


def _prep_reorder(c, seed):
    """A beam search in the middle of its run: every request row has its pages and its state slot (slot = row)."""
    g = _gen(seed)
    R, W, bs = c["R"], c["W"], c["bs"]
    N = R * W
    length = c["prompt"] + c["made"]
    M = -(-length // bs) + 1
    used = M - 1
    pages = torch.randperm(N * used + 5, generator=g, device=DEV)[:N * used].to(torch.int32).view(N, used)
    rows = torch.randperm(N, generator=g, device=DEV).to(torch.int32).view(R, W)
    table = torch.cat([pages, torch.full((N, 1), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
    cache = lambda dt: _randn(g, N * used + 5, bs, c["Hkv"], c["Da"], dtype=dt)  # noqa: E731
    # better beams have more successors
    at = torch.rand(R, W, generator=g, device=DEV)
    parents = (at * at * W).to(torch.int32).clamp(max=W - 1)
    return dict(c=c, parents=parents, rows=rows, table=table,
                lens=torch.full((N,), length, dtype=torch.int32, device=DEV),
                first=torch.full((N,), c["prompt"], dtype=torch.int32, device=DEV),
                state=_randn(g, N, c["Hv"], c["D"], c["D"]), kc=cache(torch.bfloat16), vc=cache(torch.bfloat16),
                v16=cache(torch.float16) if c["v16"] else None, kept=None)


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    op = s["c"]["op"]
    if own:
        return {"delta": _own_delta, "delta_step": _own_delta_step, "select": _own_select,
                "reorder": _own_reorder}[op](s)
    return {"delta": _plain_delta, "delta_step": _plain_delta_step, "select": _plain_select,
            "reorder": _plain_reorder}[op](s)


def _own_delta(s):
    import attention_attn_varlen_gb300 as av
    c = s["c"]
    if s["ws"] is None:   # kept by the program from call to call
        n = av.delta_attn_workspace_size(c["B"], s["q"].shape[0], c["Hk"], c["Hv"], c["D"], s["max_len"])
        s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    av.delta_attn_varlen_fwd(s["q"], s["k"], s["v"], s["decay"], s["beta"], s["cu"], s["max_len"], s["scale"],
                             state_cache=s["state"], state_slots=s["slots"], context_lens=s["ctx"],
                             qk_norm_eps=EPS if c["norm"] else None, out=s["out"], workspace=s["ws"])
    return dict(out=s["out"], state=s["state"])


def _own_delta_step(s):
    import attention_attn_varlen_gb300 as av
    av.delta_attn_decode(s["q"], s["k"], s["v"], s["decay"], s["beta"], s["state"], s["slots"], s["scale"],
                         qk_norm_eps=EPS if s["c"]["norm"] else None, out=s["out"])
    return dict(out=s["out"], state=s["state"])


def _own_select(s):
    import attention_attn_varlen_gb300 as av
    c = s["c"]
    if s["kept"] is None:
        R, k = c["R"], c["k"]
        s["kept"] = (torch.empty(R, k, dtype=torch.int32, device=DEV), torch.empty(R, k, dtype=torch.int32, device=DEV),
                     torch.empty(R, k, dtype=torch.float32, device=DEV))
        s["ws"] = torch.empty(max(1, av.beam_select_workspace_size(R, c["W"], c["V"], k)), dtype=torch.uint8, device=DEV)
    tokens, parents, scores = av.beam_select(s["logits"], s["scores"], c["W"], c["k"], out=s["kept"], workspace=s["ws"])
    return dict(tokens=tokens, parents=parents, scores=scores)


def _own_reorder(s):
    import attention_attn_varlen_gb300 as av
    c = s["c"]
    if s["kept"] is None:
        s["kept"] = tuple(torch.empty(c["R"], c["W"], dtype=torch.int32, device=DEV) for _ in range(2))
    rows, source = av.beam_rows(s["parents"], s["rows"], out=s["kept"])
    av.copy_states(s["state"], source, rows)
    av.copy_kvcache(s["kc"], s["vc"], source, rows, s["table"], s["lens"], first_tokens=s["first"],
                    v16_cache=s["v16"])
    return dict(rows=rows, source=source, state=s["state"], k_cache=s["kc"], v_cache=s["vc"], v16_cache=s["v16"])


CHUNK = 64


def _normed(x, c):
    x = x.float()
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS) if c["norm"] else x


def _plain_delta(s):
    """Chunks of 64 tokens, all sequences side by side; S [B, Hv, Dv, Dk]."""
    c = s["c"]
    Hk, Hv, D, B = c["Hk"], c["Hv"], c["D"], c["B"]
    G, T = Hv // Hk, s["q"].shape[0]
    cu, slots = s["cu"].long(), s["slots"].long()
    L = cu[1:] - cu[:-1]
    S = s["state"][slots]
    if s["ctx"] is None:
        S = torch.zeros_like(S)
    else:
        S = torch.where((s["ctx"] > 0)[:, None, None, None], S, torch.zeros_like(S))
    qn, kn = _normed(s["q"], c), _normed(s["k"], c)
    i = torch.arange(CHUNK, device=DEV)
    low, eye = i[:, None] > i[None, :], torch.eye(CHUNK, device=DEV)
    # the blocks that each doubling of the triangular inverse fills: rows in the lower half of a pair, columns in
    # the upper one
    merges = [(i[:, None] // h == i[None, :] // h + 1) & (i[:, None] // (2 * h) == i[None, :] // (2 * h))
              for h in (1, 2, 4, 8, 16, 32)]
    out = torch.zeros(T + 1, Hv, D, dtype=torch.bfloat16, device=DEV)
    for at in range(0, s["max_len"], CHUNK):
        n = (L - at).clamp(0, CHUNK)                                        # tokens of this chunk
        real = i[None, :] < n[:, None]                                      # [B, C]
        tok = torch.where(real, cu[:-1, None] + at + i[None, :], torch.full_like(real, T, dtype=torch.int64))
        rows = tok.clamp(max=T - 1)
        mask = real[:, :, None, None]
        take = lambda x: torch.where(mask, x[rows].float(), 0.0).transpose(1, 2)  # noqa: E731  [B, H, C, D]
        q, k, v = take(qn).repeat_interleave(G, 1), take(kn).repeat_interleave(G, 1), take(s["v"])
        beta = torch.where(mask[..., 0], s["beta"][rows], 0.0).transpose(1, 2)               # [B, Hv, C]
        cum = torch.where(mask[..., 0], s["decay"][rows], 0.0).double().cumsum(1).transpose(1, 2)
        far = (cum[..., :, None] - cum[..., None, :]).clamp(max=0)
        far = torch.exp(far).float()                                        # e^{G_i - G_j} for j <= i
        first = torch.exp(cum).float()[..., None]
        A = torch.where(low, torch.matmul(k, k.transpose(-1, -2)) * far, 0.0) * beta[..., None]
        inv = eye.expand_as(A)
        for m in merges:                                                    # (I + A)^-1, blocks of 2, 4, .. 64
            inv = inv - torch.matmul(torch.matmul(inv, torch.where(m, A, 0.0)), inv)
        u = torch.matmul(inv, beta[..., None] * (v - first * torch.matmul(k, S.transpose(-1, -2))))
        p = torch.where(low | (eye > 0), torch.matmul(q, k.transpose(-1, -2)) * far, 0.0)
        o = torch.matmul(p, u) + first * torch.matmul(q, S.transpose(-1, -2))
        out[tok] = (o * s["scale"]).transpose(1, 2).to(torch.bfloat16)
        last = cum[..., -1:]                                                # (padding tokens add nothing)
        S = torch.exp(last).float()[..., None] * S
        S = S + torch.matmul(u.transpose(-1, -2), k * torch.exp(last - cum).float()[..., None])
    s["out"].copy_(out[:T])
    s["state"][slots] = S
    return dict(out=s["out"], state=s["state"])


def _plain_delta_step(s):
    c = s["c"]
    G, slots = c["Hv"] // c["Hk"], s["slots"].long()
    q, k = (_normed(s[x], c).repeat_interleave(G, 1) for x in ("q", "k"))
    S = torch.exp(s["decay"].double()).float()[..., None, None] * s["state"][slots]
    u = s["beta"][..., None] * (s["v"].float() - (S * k[..., None, :]).sum(-1))
    S = S + u[..., :, None] * k[..., None, :]
    s["out"].copy_((S * q[..., None, :]).sum(-1) * s["scale"])
    s["state"][slots] = S
    return dict(out=s["out"], state=s["state"])


def _plain_select(s):
    """In 64 bits: which candidate comes first may hang on the last digits."""
    c = s["c"]
    R, W, V, k = c["R"], c["W"], c["V"], c["k"]
    x = s["logits"].double()
    top = x.max(1, keepdim=True).values
    norm = top + torch.log(torch.exp(x - top).sum(1, keepdim=True))
    x = (s["scores"].double()[:, None] + (x - norm)).view(R, W * V)
    # equal scores: the lowest beam and token first
    best, at = (y[:, :k] for y in torch.sort(x, dim=1, descending=True, stable=True))
    i32 = torch.int32
    return dict(tokens=(at % V).to(i32), parents=(at // V).to(i32), scores=best.float())


def _plain_reorder(s):
    c = s["c"]
    R, W, bs = c["R"], c["W"], c["bs"]
    parents, rows = s["parents"].long(), s["rows"].long()
    w = torch.arange(W, device=DEV)
    # the first beam that goes on from a parent takes its row; the others take, in order, the rows of beams that
    # nobody goes on from
    same = (parents[:, :, None] == parents[:, None, :]) & (w[None, :] < w[:, None])
    first = ~same.any(2)
    dead = ~(parents[:, :, None] == w).any(1)
    order = torch.argsort(torch.where(dead, w, w + W), 1)                   # dead rows first, ascending
    place = torch.cumsum(~first, 1) - 1
    spare = torch.gather(rows, 1, torch.gather(order, 1, place.clamp(min=0)))
    taken = torch.gather(rows, 1, parents)
    new = torch.where(first, taken, spare)
    source = torch.where(first, torch.full_like(taken, -1), taken)
    # beams that need no copy copy their own rows onto themselves
    src, dst = torch.where(first, new, source).view(-1), new.view(-1)
    s["state"][dst] = s["state"][src]
    t = torch.arange(c["made"], device=DEV)[None, :] + s["first"].long()[src][:, None]
    slot = lambda r: torch.gather(s["table"].long()[r], 1, t // bs) * bs + t % bs  # noqa: E731
    a, b = slot(src).view(-1), slot(dst).view(-1)
    for x in (s["kc"], s["vc"]) + (() if s["v16"] is None else (s["v16"],)):
        flat = x.view(-1, c["Hkv"], c["Da"])
        flat[b] = flat[a]
    return dict(rows=new.to(torch.int32), source=source.to(torch.int32), state=s["state"], k_cache=s["kc"],
                v_cache=s["vc"], v16_cache=s["v16"])


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "select":
        n = c["R"] * c["W"] * c["V"]
        return {"bytes": n * (2 if c["bf16"] else 4) + 12 * c["R"] * c["k"], "flops": 3 * n}
    if c["op"] == "reorder":
        R, W = c["R"], c["W"]
        # beams that nobody goes on from: parent w is drawn with sqrt((w + 1) / W) - sqrt(w / W)
        spare = R * sum((1 - math.sqrt((w + 1) / W) + math.sqrt(w / W)) ** W for w in range(W))
        row = c["Hkv"] * c["Da"] * (6 if c["v16"] else 4)
        return {"bytes": 2 * spare * (c["Hv"] * c["D"] * c["D"] * 4 + c["made"] * row) + 16 * R * W, "flops": 0}
    B, Hk, Hv, D = c["B"], c["Hk"], c["Hv"], c["D"]
    step = c["op"] == "delta_step"
    T = B if step else B * (c["lo"] + c["hi"]) // 2
    states = B * Hv * D * D * 4
    moved = states * (2 if step or (c["ctx"] and c["hi"] <= 16) else 1.5 if c["ctx"] else 1)
    return {"bytes": T * (2 * (2 * Hk + 2 * Hv) * D + 8 * Hv) + moved, "flops": T * Hv * D * D * 6}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "reorder":
        return None                                          # whole numbers and copies only
    s = prepare(case, seed)
    return _exact_select(s) if case["op"] == "select" else _exact_delta(s)


def _exact_delta(s):
    """Token after token, no chunks."""
    c = s["c"]
    Hk, Hv, D, B = c["Hk"], c["Hv"], c["D"], c["B"]
    step = c["op"] == "delta_step"
    cu = s["cu"].long()
    L = cu[1:] - cu[:-1]
    state, slots = s["state"].double(), s["slots"].long()
    S = state[slots]
    if not step:
        S = S * (0 if s["ctx"] is None else (s["ctx"] > 0).double()[:, None, None, None])
    q, k, v = (s[x].double() for x in ("q", "k", "v"))
    if c["norm"]:
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS) for x in (q, k))
    a, b = torch.exp(s["decay"].double()), s["beta"].double()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    head = torch.arange(Hv, device=DEV) // (Hv // Hk)
    lens = L.tolist()
    for t in range(max(lens)):
        on = torch.tensor([i for i in range(B) if lens[i] > t], device=DEV)
        row = cu[:-1][on] + t
        old = S[on] * a[row][..., None, None]
        kt = k[row][:, head]
        miss = v[row] - torch.einsum("bhvk,bhk->bhv", old, kt)
        new = old + torch.einsum("bhv,bhk->bhvk", b[row][..., None] * miss, kt)
        out[row] = s["scale"] * torch.einsum("bhvk,bhk->bhv", new, q[row][:, head])
        S[on] = new
    state[slots] = S
    return dict(out=out, state=state)


def _exact_select(s):
    """Scores alone: one best candidate after the other."""
    c = s["c"]
    R, W = c["R"], c["W"]
    best = torch.empty(R, c["k"], dtype=torch.float64, device=DEV)
    for r in range(R):
        x = s["logits"][r * W:(r + 1) * W].double()
        x = (x - torch.logsumexp(x, 1, keepdim=True) + s["scores"][r * W:(r + 1) * W, None].double()).view(-1)
        for i in range(c["k"]):
            at = x.argmax()
            best[r, i] = x[at]
            x[at] = -math.inf
    return dict(tokens=None, parents=None, scores=best)
