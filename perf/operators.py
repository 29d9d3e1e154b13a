"""Measured cases of the serving-step operators.

One serving step of a model with attention layers and linear-attention layers
uses them in this order: the page tables grow on the GPU by the step's new
tokens (step_tables; trim_pages takes rejected tokens back), every attention
layer rotates its q and k and stores k and v into the paged cache
(rope_store_kvcache), every linear-attention layer runs a prompt in chunks
(linear_attn_varlen_fwd) or one token per sequence (linear_attn_decode) on its
fp32 state cache.

Each operator is here in plain torch operations (own = False) and as the call a
user makes (own = True).
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
        # a decode step of 64 running requests: latency only
        dict(name="tables_decode_64", op="tables", B=64, R=96, M=64, bs=256, new_max=1, T=64),
        # chunked prefill mixed with decode: 300 requests, up to 512 new tokens each
        dict(name="tables_mixed_300", op="tables", B=300, R=512, M=129, bs=16, new_max=512, T=90000),
        # a whole batch of prompts admitted at once, long rows of small pages
        dict(name="tables_admit_4096", op="tables", B=4096, R=4096, M=512, bs=32, new_max=2048, T=4700000),
        # one decode step's q/k/v of 64 requests, 32/8 heads
        dict(name="rope_decode_64", op="rope", N=64, Hq=32, Hkv=8, D=128, rot=128, axes=1, inter=False, bs=256,
             v16=False, far=131072),
        # the prefix-cache step's 8,503 new tokens, positions with three axes, V / 16 kept too
        dict(name="rope_step_8503_3axes", op="rope", N=8503, Hq=32, Hkv=8, D=128, rot=128, axes=3, inter=False,
             bs=256, v16=True, far=32768),
        # small heads, neighbouring pairs, half of the head rotated, positions near a million
        dict(name="rope_partial_1237_d64", op="rope", N=1237, Hq=16, Hkv=16, D=64, rot=32, axes=1, inter=True, bs=16,
             v16=False, far=1000000),
        # a prompt pass of 32,768 tokens
        dict(name="rope_prompt_32768", op="rope", N=32768, Hq=32, Hkv=8, D=128, rot=128, axes=1, inter=False, bs=256,
             v16=False, far=32768),
        # sixteen packed prompts of mixed length, some continuing from a cached state
        dict(name="linear_prompts_16", op="linear", B=16, lo=200, hi=4096, Hq=32, Hkv=32, D=128, ctx=True),
        # one long prompt: little parallelism over sequences
        dict(name="linear_long_32768", op="linear", B=1, lo=32768, hi=32768, Hq=16, Hkv=16, D=128, ctx=False),
        # many short odd prompts, shared key/value heads, head_dim 64
        dict(name="linear_short_96_gqa", op="linear", B=96, lo=1, hi=150, Hq=16, Hkv=4, D=64, ctx=True),
        # one sequence's next token: latency only
        dict(name="linear_step_1", op="linear_step", B=1, Hq=32, Hkv=32, D=128),
        # a decode step of 256 sequences: the fp32 states are read and written once
        dict(name="linear_step_256", op="linear_step", B=256, Hq=32, Hkv=32, D=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "rope", "linear", "linear", "linear_step"])
    if op == "tables":
        B = _log(rng, 1, 4096)
        new_max = rng.choice([1, 4, _log(rng, 1, 1024)])
        bs = rng.choice([16, 32, 64, 256])
        M = max(-(-(new_max + 64) // bs) + 1, _log(rng, 4, 512))
        return dict(op=op, B=B, R=B + rng.randrange(0, 100), M=M, bs=bs, new_max=new_max,
                    T=B * new_max + rng.randrange(0, 300))
    if op == "rope":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 8])
        G = rng.choice([1, 3, 4, 8])
        axes = rng.choice([1, 1, 3])
        rot = rng.choice([D, D, D // 2])
        return dict(op=op, N=_log(rng, 1, 16384), Hq=Hkv * G, Hkv=Hkv, D=D, rot=rot, axes=axes,
                    inter=rng.choice([False, False, True]), bs=rng.choice([16, 64, 256]),
                    v16=rng.choice([False, True]), far=_log(rng, 100, 1000000))
    D = rng.choice([64, 128])
    Hkv = rng.choice([2, 4, 16, 32])
    Hq = Hkv * (rng.choice([1, 1, 2, 4]) if Hkv <= 8 else 1)
    if op == "linear_step":
        return dict(op=op, B=_log(rng, 1, 256), Hq=Hq, Hkv=Hkv, D=D)
    B = _log(rng, 1, 64)
    hi = _log(rng, 1, max(2, 16384 // B))
    return dict(op=op, B=B, lo=max(1, hi // rng.choice([1, 2, 20])), hi=hi, Hq=Hq, Hkv=Hkv, D=D,
                ctx=rng.choice([False, True]))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _lens(case):
    # the lengths belong to the case: the packed tensors have one shape for every seed
    g = torch.Generator().manual_seed(17 + case["B"] + case["hi"])
    return torch.randint(case["lo"], case["hi"] + 1, (case["B"],), generator=g).tolist()


def prepare(case, seed):
    return {"tables": _prep_tables, "rope": _prep_rope, "linear": _prep_linear,
            "linear_step": _prep_linear_step}[case["op"]](case, seed)


def _prep_tables(c, seed):
    """A page pool in the middle of a run: R request rows, B of them in this step."""
    g = torch.Generator().manual_seed(int(seed))
    B, R, M, bs = c["B"], c["R"], c["M"], c["bs"]
    rows = torch.randperm(R, generator=g)[:B]
    new = torch.randint(1, c["new_max"] + 1, (B,), generator=g)
    new = torch.where(torch.cumsum(new, 0) <= c["T"], new, torch.zeros_like(new))
    lens = torch.randint(0, M * bs - c["new_max"] + 1, (R,), generator=g)
    used = (lens + bs - 1) // bs
    total = int(used.sum())
    F = R * M + 8
    pages = torch.randperm(F, generator=g).to(torch.int32)
    table = torch.full((R, M), -1, dtype=torch.int32)
    fill = torch.arange(M)[None, :] < used[:, None]
    table[fill] = pages[:total]
    free = torch.full((F,), -1, dtype=torch.int32)
    free[:F - total] = pages[total:]
    i32 = torch.int32
    return dict(c=c, rows=rows.to(i32).to(DEV), new=new.to(i32).to(DEV), lens=lens.to(i32).to(DEV), table=table.to(DEV),
                free=free.to(DEV), nfree=torch.tensor([F - total], dtype=i32, device=DEV), kept=None)


def _prep_rope(c, seed):
    g = _gen(seed)
    N, Hq, Hkv, D, bs = c["N"], c["Hq"], c["Hkv"], c["D"], c["bs"]
    # q, k and v are views of the projection's packed output
    qkv = _randn(g, N, Hq + 2 * Hkv, D)
    nb = -(-(N + N // 4 + 1) // bs)
    cache = lambda dt: _randn(g, nb, bs, Hkv, D, dtype=dt)  # noqa: E731
    slots = torch.randperm(nb * bs, generator=g, device=DEV)[:N].to(torch.int64)
    start = torch.randint(0, c["far"], (1,), generator=g, device=DEV)
    if c["axes"] == 1:
        pos = (start + torch.arange(N, device=DEV)).to(torch.int32)
        axis = None
    else:
        # time advances slowly, height and width walk over image grids of 24 columns
        i = torch.arange(N, device=DEV)
        pos = torch.stack([start + i // 576, start + (i // 24) % 24, start + i % 24]).to(torch.int32)
        h = c["rot"] // 2
        axis = [0] * (h - 2 * (3 * h // 8)) + [1] * (3 * h // 8) + [2] * (3 * h // 8)
    half = c["rot"] // 2
    inv = (500000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).to(torch.float32).to(DEV)
    return dict(c=c, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], pos=pos, axis=axis, inv=inv,
                axis_t=torch.tensor(axis or [0] * half, device=DEV), kc=cache(torch.bfloat16),
                vc=cache(torch.bfloat16), v16=cache(torch.float16) if c["v16"] else None, slots=slots,
                q_out=torch.empty(N, Hq, D, dtype=torch.bfloat16, device=DEV))


def _decays(Hkv):
    # a geometric range of memory lengths over the heads: about 1 to 256 tokens
    h = torch.arange(1, Hkv + 1, dtype=torch.float64)
    return (-(2.0 ** (-8.0 * h / Hkv))).to(torch.float32).to(DEV)


def _prep_linear(c, seed):
    g = _gen(seed)
    lens = _lens(c)
    T, B, Hq, Hkv, D = sum(lens), c["B"], c["Hq"], c["Hkv"], c["D"]
    qkv = _randn(g, T, Hq + 2 * Hkv, D)
    cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)
    state = torch.randn(B + 3, Hkv, D, D, generator=g, device=DEV, dtype=torch.float32)
    slots = torch.randperm(B + 3, generator=g, device=DEV)[:B].to(torch.int32)
    ctx = (torch.arange(B, device=DEV) % 2 * 100).to(torch.int32) if c["ctx"] else None
    return dict(c=c, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], cu=cu, max_len=max(lens),
                g=_decays(Hkv), state=state, slots=slots, ctx=ctx, scale=1.0 / math.sqrt(D),
                out=torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV), ws=None)


def _prep_linear_step(c, seed):
    g = _gen(seed)
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    qkv = _randn(g, B, Hq + 2 * Hkv, D)
    state = torch.randn(B + 3, Hkv, D, D, generator=g, device=DEV, dtype=torch.float32)
    slots = torch.randperm(B + 3, generator=g, device=DEV)[:B].to(torch.int32)
    return dict(c=c, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], g=_decays(Hkv), state=state,
                slots=slots, scale=1.0 / math.sqrt(D), out=torch.empty(B, Hq, D, dtype=torch.bfloat16, device=DEV))


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    op = s["c"]["op"]
    if own:
        return {"tables": _own_tables, "rope": _own_rope, "linear": _own_linear, "linear_step": _own_linear_step}[op](s)
    return {"tables": _plain_tables, "rope": _plain_rope, "linear": _plain_linear,
            "linear_step": _plain_linear_step}[op](s)


def _own_tables(s):
    import attention_attn_varlen_gb300 as av
    c = s["c"]
    if s["kept"] is None:   # buffers that the program keeps from step to step
        ws = torch.empty(av.lib().attn_step_tables_workspace_size(c["B"]), dtype=torch.uint8, device=DEV)
        s["kept"] = av.StepTables.empty(c["B"], c["M"], c["T"], DEV), ws
    t, ws = s["kept"]
    av.step_tables(s["rows"], s["new"], s["lens"], s["table"], s["free"], s["nfree"], c["bs"], c["T"], out=t,
                   workspace=ws)
    # the step's tokens are taken back: the pool is as before
    av.trim_pages(s["rows"], t.context_lens, s["lens"], s["table"], s["free"], s["nfree"], c["bs"], workspace=ws)
    return dict(block_table=t.block_table, slot_mapping=t.slot_mapping, positions=t.positions, cu_q=t.cu_seqlens_q,
                cu_k=t.cu_seqlens_k, cache_seqlens=t.cache_seqlens, context_lens=t.context_lens, lens=s["lens"],
                table=s["table"], free=s["free"], nfree=s["nfree"])


def _own_rope(s):
    import attention_attn_varlen_gb300 as av
    c = s["c"]
    av.rope_store_kvcache(s["q"], s["k"], s["v"], s["pos"], s["inv"], s["kc"], s["vc"], s["slots"],
                          pair_axis=s["axis"], interleaved=c["inter"], q_out=s["q_out"], v16_cache=s["v16"])
    return dict(q=s["q_out"], k_cache=s["kc"], v_cache=s["vc"], v16_cache=s["v16"])


def _own_linear(s):
    import attention_attn_varlen_gb300 as av
    if s["ws"] is None:   # kept by the program, as for the other calls
        c = s["c"]
        n = av.linear_attn_workspace_size(c["B"], c["Hq"], c["Hkv"], c["D"], s["max_len"])
        s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    av.linear_attn_varlen_fwd(s["q"], s["k"], s["v"], s["g"], s["cu"], s["max_len"], s["scale"],
                              state_cache=s["state"], state_slots=s["slots"], context_lens=s["ctx"], out=s["out"],
                              workspace=s["ws"])
    return dict(out=s["out"], state=s["state"])


def _own_linear_step(s):
    import attention_attn_varlen_gb300 as av
    av.linear_attn_decode(s["q"], s["k"], s["v"], s["g"], s["state"], s["slots"], s["scale"], out=s["out"])
    return dict(out=s["out"], state=s["state"])


def _plain_tables(s):
    c = s["c"]
    bs, T, M, B = c["bs"], c["T"], c["M"], c["B"]
    i32 = torch.int32
    rows = s["rows"].long()
    new, lens, table, free = s["new"].long(), s["lens"], s["table"], s["free"]
    ctx = lens[rows].long()
    nfree = s["nfree"].long()
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    before, want = (ctx + bs - 1) // bs, (ctx + new + bs - 1) // bs
    need = want - before
    cum = torch.cumsum(need, 0)
    ok = ((need == 0) | (cum <= nfree)) & (want <= M)
    after = torch.where(ok, want, before)
    total = torch.where(ok, ctx + new, ctx)
    j = torch.arange(M, device=DEV)[None, :]
    place = nfree - 1 - (cum - need)[:, None] - (j - before[:, None])
    fresh = (j >= before[:, None]) & (j < after[:, None])
    own_rows = torch.where(fresh, free[place.clamp(0, free.numel() - 1)], table[rows])
    block_table = torch.where(j < after[:, None], own_rows, torch.full_like(own_rows, -1))
    table[rows] = own_rows
    lens[rows] = total.to(i32)
    taken = torch.where(ok, cum, torch.zeros_like(cum)).max()
    s["nfree"].sub_(taken.to(i32))
    cu_q = torch.cat([zero, torch.cumsum(new, 0)])
    cu_k = torch.cat([zero, torch.cumsum(total, 0)])
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu_q[1:], t, right=True)
    inside = b < B
    b = b.clamp(max=B - 1)
    pos = ctx[b] + t - cu_q[b]
    page = block_table[b, (pos // bs).clamp(max=M - 1)].long()
    slot = torch.where(inside & ok[b], page * bs + pos % bs, torch.full_like(pos, -1))
    positions = torch.where(inside, pos, torch.zeros_like(pos)).to(i32)
    # take the step's tokens back: pages return in the order that restores the list
    freed = after - before
    cumf = torch.cumsum(freed, 0)
    nf = s["nfree"].long()
    place = nf + cumf[-1] - 1 - ((cumf - freed)[:, None] + j - before[:, None])
    give = (j >= before[:, None]) & (j < after[:, None])
    grown = torch.cat([free, free[:1]])
    grown[torch.where(give, place, torch.full_like(place, free.numel()))] = own_rows
    free.copy_(grown[:-1])
    table[rows] = torch.where(give, torch.full_like(own_rows, -1), own_rows)
    lens[rows] = ctx.to(i32)
    s["nfree"].add_(cumf[-1].to(i32))
    return dict(block_table=block_table, slot_mapping=slot, positions=positions, cu_q=cu_q.to(i32), cu_k=cu_k.to(i32),
                cache_seqlens=total.to(i32), context_lens=ctx.to(i32), lens=lens, table=table, free=free,
                nfree=s["nfree"])


def _plain_rotate(x, cos, sin, rot, inter):
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([u, w], -1).flatten(-2) if inter else torch.cat([u, w], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rope(s):
    c = s["c"]
    pos = s["pos"].double()
    pos = pos[:, None] if c["axes"] == 1 else pos[s["axis_t"]].T
    angle = pos * s["inv"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    s["q_out"].copy_(_plain_rotate(s["q"], cos, sin, c["rot"], c["inter"]))
    k = _plain_rotate(s["k"], cos, sin, c["rot"], c["inter"]).to(torch.bfloat16)
    s["kc"].view(-1, c["Hkv"], c["D"])[s["slots"]] = k
    s["vc"].view(-1, c["Hkv"], c["D"])[s["slots"]] = s["v"]
    if s["v16"] is not None:
        s["v16"].view(-1, c["Hkv"], c["D"])[s["slots"]] = (s["v"].float() / 16).to(torch.float16)
    return dict(q=s["q_out"], k_cache=s["kc"], v_cache=s["vc"], v16_cache=s["v16"])


CHUNK = 128


def _plain_linear(s):
    """Chunks of 128 tokens, all sequences side by side; S [B, Hkv, Dv, Dk]."""
    c = s["c"]
    Hq, Hkv, D, B = c["Hq"], c["Hkv"], c["D"], c["B"]
    G, T = Hq // Hkv, s["q"].shape[0]
    g = s["g"].double()
    cu, slots = s["cu"].long(), s["slots"].long()
    L = cu[1:] - cu[:-1]
    S = s["state"][slots]
    if s["ctx"] is None:
        S = torch.zeros_like(S)
    else:
        S = torch.where((s["ctx"] > 0)[:, None, None, None], S, torch.zeros_like(S))
    i = torch.arange(CHUNK, device=DEV)
    d = i[:, None] - i[None, :]
    decay = torch.where(d >= 0, torch.exp(d.clamp(min=0) * g[:, None, None]), torch.zeros((), device=DEV).double())
    decay = decay.float()                                                   # [Hkv, C, C]
    first = torch.exp((i + 1) * g[:, None]).float()                         # [Hkv, C]
    out = torch.zeros(T + 1, Hq, D, dtype=torch.bfloat16, device=DEV)
    for at in range(0, s["max_len"], CHUNK):
        n = (L - at).clamp(0, CHUNK)                                        # tokens of this chunk
        real = i[None, :] < n[:, None]                                      # [B, C]
        tok = torch.where(real, cu[:-1, None] + at + i[None, :], torch.full_like(real, T, dtype=torch.int64))
        rows = tok.clamp(max=T - 1)
        mask = real[:, :, None, None]
        q = torch.where(mask, s["q"][rows].float(), 0.0).view(B, CHUNK, Hkv, G, D).permute(0, 2, 3, 1, 4)
        k = torch.where(mask, s["k"][rows].float(), 0.0).transpose(1, 2)    # [B, Hkv, C, D]
        v = torch.where(mask, s["v"][rows].float(), 0.0).transpose(1, 2)
        p = torch.matmul(q, k.transpose(-1, -2)[:, :, None]) * decay[None, :, None]
        o = torch.matmul(p, v[:, :, None])
        o = o + first[None, :, None, :, None] * torch.matmul(q, S.transpose(-1, -2)[:, :, None])
        o = (o * s["scale"]).permute(0, 3, 1, 2, 4).reshape(B, CHUNK, Hq, D)
        out[tok] = o.to(torch.bfloat16)
        left = (n[:, None] - 1 - i[None, :]).clamp(min=0)                   # steps from token i to the chunk's end
        w = torch.exp(left[:, None, :] * g[None, :, None]).float()          # [B, Hkv, C]
        S = torch.exp(n[:, None] * g[None, :]).float()[:, :, None, None] * S
        S = S + torch.matmul(v.transpose(-1, -2), k * w[..., None])
    s["out"].copy_(out[:T])
    s["state"][slots] = S
    return dict(out=s["out"], state=s["state"])


def _plain_linear_step(s):
    c = s["c"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    slots = s["slots"].long()
    S = s["state"][slots]
    k, v = s["k"].float(), s["v"].float()
    S = torch.exp(s["g"].double()).float()[None, :, None, None] * S + v[..., :, None] * k[..., None, :]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    o = torch.matmul(q, S.transpose(-1, -2)) * s["scale"]
    s["out"].copy_(o.view(B, Hq, D))
    s["state"][slots] = S
    return dict(out=s["out"], state=s["state"])


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "tables":
        B, M, T = c["B"], c["M"], c["T"]
        pages = -(-M // 2) + 1                               # of a request, on average
        new = -(-c["new_max"] // (2 * c["bs"])) + 1
        # lists of requests, offsets and lengths; the table rows; the tokens; the pages taken and given back
        return {"bytes": B * (16 + 8 + 20) + 4 * B * (M + pages) + 12 * T + 24 * B * new, "flops": 0}
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "rope":
        N = c["N"]
        row = 2 * (2 * Hq + 4 * Hkv) * D + (2 * Hkv * D if c["v16"] else 0) + 8 + 4 * c["axes"]
        return {"bytes": N * row, "flops": N * (Hq + Hkv) * c["rot"] * 3}
    B = c["B"]
    T = B if c["op"] == "linear_step" else B * (c["lo"] + c["hi"]) // 2
    states = B * Hkv * D * D * 4
    moved = 2 * states if c["op"] == "linear_step" else states * (1.5 if c["ctx"] else 1)
    return {"bytes": T * 2 * (2 * Hq + 2 * Hkv) * D + moved, "flops": T * D * D * 2 * (Hq + Hkv)}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "tables":
        return None                                          # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    return _exact_linear(s) if case["op"] == "linear" else _exact_linear_step(s)


def _exact_rope(s):
    c = s["c"]
    rot, half = c["rot"], c["rot"] // 2
    # each pair as a complex number times exp(i angle)
    p = s["pos"].double().reshape(c["axes"], -1)
    angle = torch.stack([p[s["axis_t"][i]] * float(s["inv"][i]) for i in range(half)], 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def rotated(x):
        y = x.double().clone()
        if c["inter"]:
            z = torch.complex(y[..., 0:rot:2].contiguous(), y[..., 1:rot:2].contiguous()) * turn
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        else:
            z = torch.complex(y[..., :half].contiguous(), y[..., half:rot].contiguous()) * turn
            y[..., :half], y[..., half:rot] = z.real, z.imag
        return y

    def stored(cache, rows):
        y = cache.double().view(-1, c["Hkv"], c["D"])
        y[s["slots"]] = rows
        return y.view(cache.shape)

    v = s["v"].double()
    return dict(q=rotated(s["q"]), k_cache=stored(s["kc"], rotated(s["k"])), v_cache=stored(s["vc"], v),
                v16_cache=None if s["v16"] is None else stored(s["v16"], v / 16))


def _exact_linear(s):
    """Every visible pair (i, j <= i) of a sequence, weighted by exp((i - j) g): no chunks, no running state."""
    c = s["c"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    cu = s["cu"].tolist()
    if sum((cu[b + 1] - cu[b]) ** 2 for b in range(c["B"])) * Hq * D * 2 > 2e13:
        return None
    g = s["g"].double()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    state = s["state"].double()
    for b in range(c["B"]):
        lo, n, slot = cu[b], cu[b + 1] - cu[b], int(s["slots"][b])
        start = state[slot].clone()
        if s["ctx"] is None or int(s["ctx"][b]) == 0:
            start.zero_()
        k, v = (s[x][lo:lo + n].double().transpose(0, 1) for x in ("k", "v"))         # [Hkv, n, D]
        j = torch.arange(n, device=DEV, dtype=torch.float64)
        for h in range(Hkv):
            q = s["q"][lo:lo + n, h * G:(h + 1) * G].double().transpose(0, 1)          # [G, n, D]
            for a in range(0, n, 2048):
                e = min(n, a + 2048)
                far = j[a:e, None] - j[None, :e]
                p = q[:, a:e] @ k[h, :e].T
                p = torch.where(far >= 0, p * torch.exp(far.clamp(min=0) * g[h]), 0.0)
                o = p @ v[h, :e] + torch.exp((j[a:e, None] + 1) * g[h]) * (q[:, a:e] @ start[h].T)
                out[lo + a:lo + e, h * G:(h + 1) * G] = (o * s["scale"]).transpose(0, 1)
        w = torch.exp((n - 1 - j)[None, :] * g[:, None])
        state[slot] = torch.exp(n * g)[:, None, None] * start + torch.einsum("hnv,hnk->hvk", v, k * w[..., None])
    return dict(out=out, state=state)


def _exact_linear_step(s):
    c = s["c"]
    G = c["Hq"] // c["Hkv"]
    state = s["state"].double()
    a = torch.exp(s["g"].double())
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        slot = int(s["slots"][b])
        new = a[:, None, None] * state[slot] + torch.einsum("hv,hk->hvk", s["v"][b].double(), s["k"][b].double())
        state[slot] = new
        out[b] = s["scale"] * torch.einsum("hvk,hk->hv", new.repeat_interleave(G, 0), s["q"][b].double())
    return dict(out=out, state=state)
