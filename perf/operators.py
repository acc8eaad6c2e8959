"""Cases that time libkda's latent attention and RMS norm calls beside their plain form.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges, ``prepare(case, seed)`` makes what a
program has in hand before the call, ``run(state)`` is one call, ``work(case)`` counts what it cannot do without
and ``exact(case, seed)`` is the same result from the definition in 64 bits. With ``own`` true ``run`` makes the
library's calls, else the plain form in elementary torch operations.
"""
import math
import random

import torch

own = False

HEAD = 128          # channels per head of the expanded keys and values
LATENT = 512        # channels of the latent vector
GROUP = 128         # values that share one scale of the 8-bit output
E4M3_MAX = 448.0
EPS = 1e-5
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a prompt of 8K tokens at the library's 32 heads
        dict(name="prefill_8k_h32", op="prefill", tokens=8192, history=0, seqs=1, heads=32, shared=64, causal=True),
        # a serving batch: nine ragged prompts, each continuing a history already expanded, no shared key part
        dict(name="prefill_packed_history_h16", op="prefill", tokens=2777, history=11003, seqs=9, heads=16, shared=0,
             causal=True),
        # a training step on one 8K sequence
        dict(name="train_bwd_8k_h16", op="backward", tokens=8192, history=0, seqs=1, heads=16, shared=64, causal=True),
        # a training step on packed documents of odd lengths
        dict(name="train_bwd_packed_h8", op="backward", tokens=4099, history=0, seqs=6, heads=8, shared=64, causal=True),
        # a large decode batch, ragged lengths, idle slots among them (256 sequences x 32 heads as the decode benchmark)
        dict(name="decode_n256_h32", op="decode", seqs=256, drafted=1, heads=32, shared=64, longest=8192, page=64),
        # one user far into a 128K context
        dict(name="decode_n1_h32_128k", op="decode", seqs=1, drafted=1, heads=32, shared=64, longest=131072, page=64),
        # a few short sequences that check three drafted tokens each: latency counts
        dict(name="decode_n4_h16_drafted3", op="decode", seqs=4, drafted=3, heads=16, shared=64, longest=333, page=16),
        # the norm in front of a layer in training, with the residual's addition
        dict(name="norm_16k_4096", op="norm", rows=16384, width=4096, dtype="bf16", residual=True, bits8=False),
        # the norm in front of 8-bit projections in a decode step
        dict(name="norm_8bit_256_4096", op="norm", rows=256, width=4096, dtype="bf16", residual=True, bits8=True),
        # its backward pass in training
        dict(name="norm_bwd_8k_4096", op="norm_bwd", rows=8192, width=4096, dtype="bf16", residual=True),
        # the latents of a prompt into the cache's pages, and those of one decode step
        dict(name="append_prompt_8k", op="append", tokens=8192, shared=64, page=64),
        dict(name="append_decode_256", op="append", tokens=256, shared=64, page=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "backward", "backward", "decode", "decode", "decode", "norm", "norm",
                     "norm_bwd", "append"])
    shared = rng.choice([64, 64, 0])
    if op in ("prefill", "backward"):
        heads = rng.choice([1, 3, 4, 8, 16, 32])
        tokens = _log_int(rng, 16, 8192 if heads <= 16 else 5000)
        seqs = min(tokens, _log_int(rng, 1, 16))
        history = 0 if op == "backward" or rng.random() < 0.5 else _log_int(rng, 1, 4096)
        return dict(op=op, tokens=tokens, history=history, seqs=seqs, heads=heads, shared=shared,
                    causal=rng.random() < 0.8)
    if op == "decode":
        seqs = _log_int(rng, 1, 256)
        return dict(op=op, seqs=seqs, drafted=rng.choice([1, 1, 1, 2, 4]), heads=rng.choice([8, 16, 20, 32, 64, 128]),
                    shared=shared, longest=_log_int(rng, 8, min(131072, 800000 // seqs)),
                    page=rng.choice([16, 32, 64, 80, 128]))
    if op == "append":
        return dict(op=op, tokens=_log_int(rng, 1, 16384), shared=shared, page=rng.choice([16, 32, 64, 80, 128]))
    width = 128 * _log_int(rng, 2, 64)
    if op == "norm":
        bits8 = rng.random() < 0.5
        return dict(op=op, rows=_log_int(rng, 1, 16384), width=width, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    residual=rng.random() < 0.7, bits8=bits8)
    return dict(op=op, rows=_log_int(rng, 1, 8192), width=width, dtype=rng.choice(["bf16", "bf16", "f32"]),
                residual=rng.random() < 0.7)


def _split(total, parts, least, tag):
    """``total`` into ``parts`` ragged lengths of at least ``least``, the same ones for the same numbers."""
    r = random.Random("%d %d %s" % (total, parts, tag))
    w = [r.uniform(0.1, 1.0) for _ in range(parts)]
    room = total - least * parts
    cut = [0] + [int(room * sum(w[:i + 1]) / sum(w)) for i in range(parts - 1)] + [room]
    return [least + cut[i + 1] - cut[i] for i in range(parts)]


def _lengths(case):
    """(new tokens, keys) of each sequence of a packed case."""
    new = _split(case["tokens"], case["seqs"], 1, "new")
    old = _split(case["history"], case["seqs"], 0, "old")
    return new, [a + b for a, b in zip(new, old)]


def _decode_lengths(case):
    """Cached tokens of each sequence, the drafted ones included; with many sequences one slot in 32 is idle."""
    r = random.Random("%d %d lens" % (case["seqs"], case["longest"]))
    lens = [r.randint(max(1, case["longest"] // 4), case["longest"]) for _ in range(case["seqs"])]
    lens[0] = case["longest"]
    return [0 if i % 32 == 31 else max(n, case["drafted"]) for i, n in enumerate(lens)]


def _pairs(case):
    """Visible (query, key) pairs of a packed case."""
    if not case["causal"]:
        return sum(a * b for a, b in zip(*_lengths(case)))
    return sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(*_lengths(case)))


def work(case):
    op = case["op"]
    if op in ("prefill", "backward"):
        H, R, T = case["heads"], case["shared"], case["tokens"]
        Tk, dqk = T + case["history"], HEAD + case["shared"]
        q, o, kv, r = T * H * dqk * 2, T * H * HEAD * 2, 2 * Tk * H * HEAD * 2, Tk * R * 2
        if op == "prefill":
            return {"bytes": q + kv + r + o + T * H * 4, "flops": 2 * _pairs(case) * H * (dqk + HEAD)}
        return {"bytes": 2 * (q + kv + r) + 2 * o + T * H * 4, "flops": 2 * _pairs(case) * H * (3 * dqk + 2 * HEAD)}
    if op == "decode":
        n, w = sum(_decode_lengths(case)), LATENT + case["shared"]
        rows = case["seqs"] * case["drafted"] * case["heads"]
        return {"bytes": n * w * 2 + rows * (w * 2 + LATENT * 2 + 4),
                "flops": 2 * n * case["drafted"] * case["heads"] * (w + LATENT)}
    if op == "append":
        return {"bytes": case["tokens"] * ((LATENT + case["shared"]) * 4 + 8), "flops": 4 * case["tokens"] * LATENT}
    n, e = case["rows"] * case["width"], 2 if case["dtype"] == "bf16" else 4
    if op == "norm":
        out = n + case["rows"] * (case["width"] // GROUP) * 4 if case["bits8"] else n * e
        return {"bytes": n * e * (3 if case["residual"] else 1) + out + case["width"] * 4, "flops": 5 * n}
    return {"bytes": n * e * (4 if case["residual"] else 3) + 2 * case["width"] * 4, "flops": 10 * n}


# ------------------------------------------------------------------------------------------ inputs

def _gen(case, seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(gen, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)


def _offsets(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)


def prepare(case, seed):
    g, op = _gen(case, seed), case["op"]
    s = {"case": case, "op": op}
    if op in ("prefill", "backward"):
        H, R, T, Tk = case["heads"], case["shared"], case["tokens"], case["tokens"] + case["history"]
        new, keys = _lengths(case)
        s.update(cu_q=_offsets(new), cu_k=_offsets(keys), longest_q=max(new), longest_k=max(keys),
                 causal=case["causal"], scale=(HEAD + R) ** -0.5)
        s["q"] = _normal(g, 1, T, H, HEAD + R, std=1.5)
        # keys and values leave the up-projection of the latent as one tensor, and are views of it
        s["kv"] = _normal(g, 1, Tk, H, 2 * HEAD)
        s["r"] = _normal(g, 1, Tk, R) if R else None
        if op == "backward":
            s["dout"] = _normal(g, 1, T, H, HEAD)
            out, lse = _attend(s)
            s["out"], s["lse"] = out.to(torch.bfloat16), lse
        return s
    if op == "decode":
        N, W, page = case["seqs"], LATENT + case["shared"], case["page"]
        lens = _decode_lengths(case)
        per = [-(-n // page) for n in lens]
        width = max(max(per), 1)
        total = sum(per) + 1
        order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)    # pages as an allocator leaves them
        first = torch.tensor([0] + per, dtype=torch.int64).cumsum(0)[:-1].to(DEV)
        col = torch.arange(width, device=DEV)
        used = col[None] < torch.tensor(per, device=DEV)[:, None]
        s["table"] = torch.where(used, order[(first[:, None] + col[None]).clamp(max=total - 1)], 0).to(torch.int32)
        s["lens"] = torch.tensor(lens, dtype=torch.int32).to(DEV)
        s["cache"] = _normal(g, total, page, W)
        s["q"] = _normal(g, N, case["drafted"], case["heads"], W)
        s["scale"] = (HEAD + case["shared"]) ** -0.5
        s["longest"] = max(lens)
        return s
    if op == "append":
        T, R, page = case["tokens"], case["shared"], case["page"]
        # one projection gives latent and shared key part side by side
        s["x"] = _normal(g, T, LATENT + R, std=2.0)
        s["weight"] = _normal(g, LATENT, dtype=torch.float32, std=0.1) + 1.0
        pages = -(-T // page) + 8
        s["cache"] = torch.zeros(pages, page, LATENT + R, dtype=torch.bfloat16, device=DEV)
        order = torch.randperm(pages, generator=g, device=DEV)
        t = torch.arange(T, device=DEV)
        s["slots"] = order[t // page] * page + t % page
        return s
    dt, rows, width = TYPES[case["dtype"]], case["rows"], case["width"]
    s["weight"] = _normal(g, width, dtype=torch.float32, std=0.1) + 1.0
    s["x"] = _normal(g, rows, width, dtype=dt)
    s["res"] = _normal(g, rows, width, dtype=dt, std=2.0) if case["residual"] else None
    if op == "norm_bwd":
        s["dy"] = _normal(g, rows, width, dtype=dt)
    return s


# ---------------------------------------------------------------------------------------- plain forms

def _pad(x, cu, longest):
    """Packed rows [1, T, ...] as [N, longest, ...], zeros behind each sequence."""
    at = torch.arange(longest, device=x.device)
    rows = (cu[:-1, None] + at[None]).clamp(max=x.shape[1] - 1).long()
    valid = at[None] < (cu[1:] - cu[:-1])[:, None]
    y = x[0][rows].float()
    return torch.where(valid.reshape(valid.shape + (1,) * (y.dim() - 2)), y, 0.0)


def _pack(y, cu, total):
    """The inverse of _pad: [N, longest, ...] to [1, total, ...]."""
    at = torch.arange(y.shape[1], device=y.device)
    valid = at[None] < (cu[1:] - cu[:-1])[:, None]
    rows = torch.where(valid, (cu[:-1, None] + at[None]).long(), total).reshape(-1)
    flat = torch.zeros((total + 1,) + y.shape[2:], dtype=y.dtype, device=y.device)
    return flat.index_copy(0, rows, y.reshape((-1,) + y.shape[2:]))[None, :total]


def _seen(s):
    """[N, 1, Lq, Lk]: which keys a query attends to."""
    lq, lk = s["cu_q"][1:] - s["cu_q"][:-1], s["cu_k"][1:] - s["cu_k"][:-1]
    i = torch.arange(s["longest_q"], device=DEV)[None, :, None]
    j = torch.arange(s["longest_k"], device=DEV)[None, None, :]
    seen = (j < lk[:, None, None]) & (i < lq[:, None, None])
    if s["causal"]:
        seen = seen & (j <= i + (lk - lq)[:, None, None])
    return seen[:, None]


def _operands(s):
    """q, [k, r] and v in 32 bits as [N, H, L, D]."""
    H = s["q"].shape[2]
    q = _pad(s["q"], s["cu_q"], s["longest_q"]).transpose(1, 2)
    kv = _pad(s["kv"], s["cu_k"], s["longest_k"]).transpose(1, 2)
    k, v = kv[..., :HEAD], kv[..., HEAD:]
    if s["r"] is not None:
        r = _pad(s["r"], s["cu_k"], s["longest_k"])[:, None].expand(-1, H, -1, -1)
        k = torch.cat([k, r], -1)
    return q, k, v


def _softmax(x):
    """exp(x - max), its sums and the log of the sums of exp(x); rows without a value give zeros and -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    return p, total, (m + torch.log(total))[..., 0]


def _attend(s):
    q, k, v = _operands(s)
    p, total, lse = _softmax((q @ k.transpose(-1, -2) * s["scale"]).masked_fill(~_seen(s), -math.inf))
    out = (p @ v) / torch.where(total == 0.0, 1.0, total)
    T = s["q"].shape[1]
    return _pack(out.transpose(1, 2), s["cu_q"], T), _pack(lse.transpose(1, 2), s["cu_q"], T)


def _attend_backward(s):
    q, k, v = _operands(s)
    seen = _seen(s)
    lse = _pad(s["lse"], s["cu_q"], s["longest_q"]).transpose(1, 2)[..., None]
    p = torch.exp((q @ k.transpose(-1, -2) * s["scale"]).masked_fill(~seen, -math.inf) - torch.where(lse == -math.inf, 0.0, lse))
    do = _pad(s["dout"], s["cu_q"], s["longest_q"]).transpose(1, 2)
    dv = p.transpose(-1, -2) @ do
    dp = do @ v.transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * s["scale"]
    del dp, p
    dq, dk = ds @ k, ds.transpose(-1, -2) @ q
    T, Tk, b = s["q"].shape[1], s["kv"].shape[1], torch.bfloat16
    got = {"dq": _pack(dq.transpose(1, 2), s["cu_q"], T).to(b),
           "dk": _pack(dk[..., :HEAD].transpose(1, 2), s["cu_k"], Tk).to(b),
           "dv": _pack(dv.transpose(1, 2), s["cu_k"], Tk).to(b)}
    if s["r"] is not None:
        got["dk_shared"] = _pack(dk[..., HEAD:].sum(1), s["cu_k"], Tk).to(b)
    return got


def _decode(s):
    N, Tq, H, W = s["q"].shape
    page, longest = s["cache"].shape[1], s["longest"]
    j = torch.arange(longest, device=DEV)
    rows = s["table"][:, j // page].long() * page + (j % page)[None]
    c = s["cache"].reshape(-1, W)[rows].float()                                     # [N, longest, W]
    t = torch.arange(Tq, device=DEV)[None, :, None, None]
    seen = j[None, None, None] < (s["lens"][:, None, None, None] - (Tq - 1) + t)
    x = (s["q"].float().reshape(N, Tq * H, W) @ c.transpose(1, 2) * s["scale"]).reshape(N, Tq, H, longest)
    p, total, lse = _softmax(x.masked_fill(~seen, -math.inf))
    out = (p.reshape(N, Tq * H, longest) @ c[..., :LATENT]).reshape(N, Tq, H, LATENT)
    return (out / torch.where(total == 0.0, 1.0, total)).to(torch.bfloat16), lse


def _norm(s, bits8):
    h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["x"].dtype)
    f = h.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * s["weight"]
    if not bits8:
        return y.to(h.dtype), h
    y = y.reshape(y.shape[0], -1, GROUP)
    scale = y.abs().amax(-1) / E4M3_MAX
    q = y / torch.where(scale == 0.0, 1.0, scale)[..., None]
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).reshape(h.shape), scale, h


def _norm_backward(s):
    h, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    g = dy * s["weight"]
    dx = r * (g - h * (r * r) * (g * h).mean(-1, keepdim=True))
    if s["res"] is not None:
        dx = dx + s["res"].float()
    return dx.to(s["x"].dtype), (dy * h * r).sum(0)


def _append(s):
    c = s["x"][:, :LATENT].float()
    y = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["weight"]
    rows = torch.cat([y.to(torch.bfloat16), s["x"][:, LATENT:]], -1)
    s["cache"].view(-1, rows.shape[1]).index_copy_(0, s["slots"], rows)
    return s["cache"]


# ------------------------------------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if own:
        import kimi_delta_attention_25_b200 as kda
        if op == "prefill":
            return kda.latent_fwd(s["q"], s["kv"][..., :HEAD], s["kv"][..., HEAD:], s["r"], cu_seqlens=s["cu_q"],
                                  cu_seqlens_k=s["cu_k"], causal=s["causal"], scale=s["scale"])
        if op == "backward":
            g = kda.latent_bwd(s["q"], s["kv"][..., :HEAD], s["kv"][..., HEAD:], s["r"], s["out"], s["lse"], s["dout"],
                               cu_seqlens=s["cu_q"], cu_seqlens_k=s["cu_k"], causal=s["causal"], scale=s["scale"])
            return {name: t for name, t in g.items() if t is not None}
        if op == "decode":
            return kda.latent_decode_step(s["q"], s["cache"], s["table"], s["lens"], scale=s["scale"])
        if op == "append":
            return kda.latent_append(s["x"][:, :LATENT], s["x"][:, LATENT:] if s["case"]["shared"] else None, s["cache"],
                                     s["slots"], weight=s["weight"], eps=EPS)
        if op == "norm":
            if s["case"]["bits8"]:
                return kda.rms_norm_e4m3(s["x"], s["weight"], residual=s["res"], eps=EPS)
            return kda.rms_norm(s["x"], s["weight"], residual=s["res"], eps=EPS)
        return kda.rms_norm_bwd(s["dy"], s["x"], s["weight"], dh=s["res"], eps=EPS)
    if op == "prefill":
        out, lse = _attend(s)
        return out.to(torch.bfloat16), lse
    if op == "backward":
        return _attend_backward(s)
    if op == "decode":
        return _decode(s)
    if op == "append":
        return _append(s)
    if op == "norm":
        return _norm(s, s["case"]["bits8"])
    return _norm_backward(s)


# ------------------------------------------------------------------------------- 64 bits, by definition

def _round_e4m3(x):
    """To the nearest value of e4m3 (4 significant bits, exponents from -6, multiples of 2^-9 below), ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_attention(case, s):
    """Sequence by sequence and head by head: softmax over the visible keys, and the chain rule through it."""
    H, R = case["heads"], case["shared"]
    T, Tk, d = case["tokens"], case["tokens"] + case["history"], torch.float64
    z = lambda *shape: torch.zeros(*shape, dtype=d, device=DEV)  # noqa: E731
    out, lse = z(1, T, H, HEAD), z(1, T, H)
    dq, dk, dv, dr = z(1, T, H, HEAD + R), z(1, Tk, H, HEAD), z(1, Tk, H, HEAD), z(1, Tk, max(R, 1))
    a = b = 0
    for n, m in zip(*_lengths(case)):
        shift = m - n
        hidden = torch.arange(m, device=DEV)[None] > torch.arange(n, device=DEV)[:, None] + shift
        for h in range(H):
            q, k = s["q"][0, a:a + n, h].to(d), s["kv"][0, b:b + m, h, :HEAD].to(d)
            v = s["kv"][0, b:b + m, h, HEAD:].to(d)
            x = q[:, :HEAD] @ k.T
            if R:
                x += q[:, HEAD:] @ s["r"][0, b:b + m].to(d).T
            x *= s["scale"]
            if case["causal"]:
                x.masked_fill_(hidden, -math.inf)
            total = torch.logsumexp(x, 1)
            p = x.sub_(total[:, None]).exp_()
            out[0, a:a + n, h], lse[0, a:a + n, h] = p @ v, total
            if case["op"] == "backward":
                do = s["dout"][0, a:a + n, h].to(d)
                dv[0, b:b + m, h] = p.T @ do
                dp = do @ v.T
                dx = dp.sub_((dp * p).sum(1, keepdim=True)).mul_(p).mul_(s["scale"])
                dq[0, a:a + n, h, :HEAD], dk[0, b:b + m, h] = dx @ k, dx.T @ q[:, :HEAD]
                if R:
                    dq[0, a:a + n, h, HEAD:] = dx @ s["r"][0, b:b + m].to(d)
                    dr[0, b:b + m] += dx.T @ q[:, HEAD:]
        a, b = a + n, b + m
    if case["op"] == "prefill":
        return out, lse
    return {"dq": dq, "dk": dk, "dv": dv, **({"dk_shared": dr} if R else {})}


def _exact_decode(case, s):
    N, Tq, H, W = s["q"].shape
    page, d = case["page"], torch.float64
    out = torch.zeros(N, Tq, H, LATENT, dtype=d, device=DEV)
    lse = torch.full((N, Tq, H), -math.inf, dtype=d, device=DEV)
    for n, length in enumerate(_decode_lengths(case)):
        if not length:
            continue
        pages = s["table"][n, :-(-length // page)].long()
        c = s["cache"][pages].reshape(-1, W)[:length].to(d)
        for t in range(Tq):
            upto = length - Tq + t + 1
            x = s["q"][n, t].to(d) @ c[:upto].T * s["scale"]
            lse[n, t] = torch.logsumexp(x, 1)
            out[n, t] = torch.softmax(x, 1) @ c[:upto, :LATENT]
    return out, lse


def exact(case, seed):
    s, op, d = prepare(case, seed), case["op"], torch.float64
    if op in ("prefill", "backward"):
        return _exact_attention(case, s)
    if op == "decode":
        return _exact_decode(case, s)
    w = s["weight"].to(d)
    if op == "append":
        c = s["x"][:, :LATENT].to(d)
        cache = torch.zeros(s["cache"].shape, dtype=d, device=DEV)
        flat = cache.view(-1, cache.shape[-1])
        flat[s["slots"], :LATENT] = c / (c.square().mean(1, keepdim=True) + EPS).sqrt() * w
        flat[s["slots"], LATENT:] = s["x"][:, LATENT:].to(d)
        return cache
    if op == "norm":
        h = s["x"].to(d) + (0.0 if s["res"] is None else s["res"].to(d))
        hr = h.to(s["x"].dtype).to(d)                  # the sum is kept, and normalised, in the inputs' type
        y = hr / (hr.square().mean(1, keepdim=True) + EPS).sqrt() * w
        if not case["bits8"]:
            return y, hr
        scale = y.reshape(y.shape[0], -1, GROUP).abs().amax(-1) / E4M3_MAX
        wide = scale.repeat_interleave(GROUP, 1)
        return _round_e4m3(y / torch.where(wide == 0.0, 1.0, wide)), scale, hr
    h, dy = s["x"].to(d), s["dy"].to(d)
    rms = (h.square().mean(1, keepdim=True) + EPS).sqrt()
    unit = h / rms
    g = dy * w
    dx = (g - unit * (g * unit).mean(1, keepdim=True)) / rms
    return dx + (0.0 if s["res"] is None else s["res"].to(d)), (dy * unit).sum(0)
