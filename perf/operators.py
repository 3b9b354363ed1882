"""Workloads of the operators for sampling several answers to a prompt and learning from them.

  packed   causal grouped-query attention over packed sequences of different lengths: forward (prompts), or forward
           and backward (training on the sampled answers)
  prefix   one decode step of a batch whose sequences share their prompts' keys and values, group by group
  policy   clipped policy loss with a KL term on the logits, with its gradient

Head layouts are those of this repository's workloads (6, 10 over 5, 12 and 13 heads of 128) and grouped ones;
the vocabulary is its 32768, or an odd one.
"""
import random

import torch

own = False

HD = 128
HEADS = [(6, 6), (10, 5), (12, 12), (13, 13), (8, 2), (4, 1)]
LARGEST_PAIRS = 12 * 8192 * 8192  # heads x padded score entries of the largest packed case


def _lens(count, lo, hi, seed):
    """`count` lengths in lo..hi, spread evenly over their logarithm."""
    r = random.Random(seed)
    return [max(lo, min(hi, int(round(lo * (hi / lo) ** r.random())))) for _ in range(count)]


def _split(total, parts):
    """`total` sequences over `parts` groups of uneven sizes (at least one each)."""
    r = random.Random(total * 1009 + parts)
    cuts = sorted(r.sample(range(1, total), parts - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def listed():
    return [
        # one short prompt: the wait before the first sampled token
        {"name": "prompt, one of 47", "op": "packed", "n": 1, "lo": 47, "hi": 47, "lens_seed": 0, "heads": 6, "kv_heads": 6, "window": -1, "train": False},
        # a batch of prompts of very different lengths, grouped heads, the sliding window of the d20_gqa layers
        {"name": "prompts, 24 ragged, window", "op": "packed", "n": 24, "lo": 30, "hi": 2000, "lens_seed": 1, "heads": 10, "kv_heads": 5, "window": 1024, "train": False},
        # one long document read whole
        {"name": "prompt, one of 8192", "op": "packed", "n": 1, "lo": 8192, "hi": 8192, "lens_seed": 0, "heads": 12, "kv_heads": 12, "window": -1, "train": False},
        # a handful of short answers: a fine-tuning micro-batch
        {"name": "train, 5 short", "op": "packed", "n": 5, "lo": 12, "hi": 180, "lens_seed": 2, "heads": 8, "kv_heads": 2, "window": -1, "train": True},
        # a training micro-batch of packed sampled answers with their prompts, d24's heads
        {"name": "train, 20 ragged", "op": "packed", "n": 20, "lo": 200, "hi": 2048, "lens_seed": 3, "heads": 12, "kv_heads": 12, "window": -1, "train": True},
        # four samples of one short prompt, a few tokens in
        {"name": "decode, 4 over 210", "op": "prefix", "groups": 1, "batch": 4, "lo": 210, "hi": 210, "T_max": 64, "own_lo": 5, "own_hi": 20, "lens_seed": 4, "heads": 6, "kv_heads": 6, "window": -1},
        # sixteen samples of one prompt, some hundred tokens in
        {"name": "decode, 16 over 2048", "op": "prefix", "groups": 1, "batch": 16, "lo": 2048, "hi": 2048, "T_max": 512, "own_lo": 40, "own_hi": 500, "lens_seed": 5, "heads": 12, "kv_heads": 12, "window": -1},
        # a rollout batch: eight prompts of different lengths, uneven numbers of samples, grouped heads
        {"name": "decode, 128 over 8 prompts", "op": "prefix", "groups": 8, "batch": 128, "lo": 300, "hi": 4000, "T_max": 1024, "own_lo": 20, "own_hi": 1000, "lens_seed": 6, "heads": 10, "kv_heads": 5, "window": -1},
        # many samples over one very long shared context
        {"name": "decode, 64 over 32000", "op": "prefix", "groups": 1, "batch": 64, "lo": 32000, "hi": 32000, "T_max": 256, "own_lo": 10, "own_hi": 250, "lens_seed": 7, "heads": 12, "kv_heads": 12, "window": -1},
        # the tokens of one short answer
        {"name": "policy, 29 rows", "op": "policy", "rows": 29, "vocab": 32768, "pad": 0, "dtype": "bf16", "masked": 0.0, "beta": 0.04},
        # one row chunk of a training micro-batch, a third of it prompt tokens that carry no loss
        {"name": "policy, 8192 rows", "op": "policy", "rows": 8192, "vocab": 32768, "pad": 0, "dtype": "bf16", "masked": 0.33, "beta": 0.04},
        # full-precision logits of an odd vocabulary in padded rows, no reference policy
        {"name": "policy, 2000 rows of 50257", "op": "policy", "rows": 2000, "vocab": 50257, "pad": 47, "dtype": "f32", "masked": 0.1, "beta": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["packed", "prefix", "policy"])
    if op == "packed":
        H, Hk = rng.choice(HEADS)
        n = _log(rng, 1, 96)
        train = rng.random() < 0.5
        most = int((LARGEST_PAIRS / (n * H * (3 if train else 1))) ** 0.5)  # the padded scores fit
        hi = _log(rng, 1, max(1, min(8192, most, 24000 // n)))
        return {"op": "packed", "n": n, "lo": _log(rng, 1, hi), "hi": hi, "lens_seed": rng.randrange(1 << 20), "heads": H,
                "kv_heads": Hk, "window": rng.choice([-1, -1, _log(rng, 1, 2048)]), "train": train}
    if op == "prefix":
        H, Hk = rng.choice(HEADS)
        B = _log(rng, 1, 128)
        groups = min(B, _log(rng, 1, 16))
        hi = _log(rng, 1, 32000 // groups if groups > 1 else 32000)
        T = _log(rng, 1, 1024)
        return {"op": "prefix", "groups": groups, "batch": B, "lo": _log(rng, 1, hi), "hi": hi, "T_max": T,
                "own_lo": 1, "own_hi": T, "lens_seed": rng.randrange(1 << 20), "heads": H, "kv_heads": Hk,
                "window": rng.choice([-1, -1, _log(rng, 1, 4096)])}
    V = rng.choice([32768, _log(rng, 100, 65000)])
    return {"op": "policy", "rows": _log(rng, 1, min(8192, (1 << 27) // V)), "vocab": V, "pad": rng.choice([0, rng.randrange(1, 64)]),
            "dtype": rng.choice(["bf16", "f32"]), "masked": round(rng.random() * 0.6, 3), "beta": rng.choice([0.0, 0.04, 0.1])}


# ------------------------------------------------------------------ inputs

def _normed(g, *shape):
    """Query and key vectors as the model's QK normalisation leaves them: RMS 1 per head."""
    x = torch.randn(*shape, generator=g, device="cuda")
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "packed":
        H, Hk = case["heads"], case["kv_heads"]
        lens = _lens(case["n"], case["lo"], case["hi"], case["lens_seed"])
        total = sum(lens)
        # q, k and v are the column ranges of one projection's output, as the block makes them
        qkv = torch.cat([_normed(g, total, H + Hk, HD), torch.randn(total, Hk, HD, generator=g, device="cuda")], 1)
        s["qkv"] = qkv.bfloat16().view(total, (H + 2 * Hk) * HD)
        s["cu"] = torch.tensor(_cu(lens), dtype=torch.int32, device="cuda")
        s["max_len"] = max(lens)
        if case["train"]:
            s["dout"] = torch.randn(total, H * HD, generator=g, device="cuda").bfloat16()
    elif case["op"] == "prefix":
        H, Hk, B, T = case["heads"], case["kv_heads"], case["batch"], case["T_max"]
        plens = _lens(case["groups"], case["lo"], case["hi"], case["lens_seed"])
        sizes = _split(B, case["groups"])
        P = sum(plens)
        s["kp"] = _normed(g, P, Hk, HD).bfloat16().view(P, Hk * HD)
        s["vp"] = torch.randn(P, Hk * HD, generator=g, device="cuda").bfloat16()
        s["k"] = _normed(g, B, T, Hk, HD).bfloat16()
        s["v"] = torch.randn(B, T, Hk, HD, generator=g, device="cuda").bfloat16()
        s["q"] = _normed(g, B, H, HD).bfloat16()
        own_lens = _lens(B, case["own_lo"], case["own_hi"], case["lens_seed"] + 1)
        for name, v in (("lens", own_lens), ("cu_prefix", _cu(plens)), ("cu_group", _cu(sizes))):
            s[name] = torch.tensor(v, dtype=torch.int32, device="cuda")
        s["max_prefix"], s["max_group"] = max(plens), max(sizes)
    else:
        N, V = case["rows"], case["vocab"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        z = torch.empty(N, V + case["pad"], dtype=dt, device="cuda")
        z.normal_(0.0, 2.0, generator=g)
        s["logits"] = z[:, :V]
        s["actions"] = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
        # sampled tokens are likely ones: their logits stand above the rest
        z[torch.arange(N, device="cuda"), s["actions"].long()] = (6 + 3 * torch.randn(N, generator=g, device="cuda")).to(dt)
        logp = torch.log_softmax(s["logits"].float(), -1).gather(1, s["actions"].long()[:, None])[:, 0]
        s["old"] = logp + 0.2 * torch.randn(N, generator=g, device="cuda")
        s["ref"] = logp + 0.5 * torch.randn(N, generator=g, device="cuda")
        s["adv"] = torch.randn(N, generator=g, device="cuda")
        kept = torch.rand(N, generator=g, device="cuda") >= case["masked"]
        s["weights"] = kept.float() / N
    return s


# ------------------------------------------------------------------ one pass

def _views(s):
    H, Hk = s["heads"], s["kv_heads"]
    return s["qkv"][:, :H * HD], s["qkv"][:, H * HD:(H + Hk) * HD], s["qkv"][:, (H + Hk) * HD:]


def _packed_own(s):
    import gpt_transformer_block_b200 as gb
    H, Hk, W = s["heads"], s["kv_heads"], s["window"]
    q, k, v = _views(s)
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.empty(H, q.shape[0], dtype=torch.float32, device=q.device)
    gb.gptb_packed_attention(q, k, v, s["cu"], o, lse, H, Hk, W)
    if not s["train"]:
        return {"o": o, "lse": lse}
    dqkv = torch.empty_like(s["qkv"])
    dq, dk, dv = dqkv[:, :H * HD], dqkv[:, H * HD:(H + Hk) * HD], dqkv[:, (H + Hk) * HD:]
    ws = torch.empty(gb.gptb_packed_attention_workspace_bytes(q.shape[0], H), dtype=torch.uint8, device=q.device)
    gb.gptb_packed_attention_backward(q, k, v, o, s["dout"], lse, s["cu"], dq, dk, dv, H, Hk, W, ws)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _packed_plain(s):
    H, Hk, W, L = s["heads"], s["kv_heads"], s["window"], s["max_len"]
    G, n, cu = H // Hk, s["n"], s["cu"].long()
    total = s["qkv"].shape[0]
    pos = torch.arange(L, device="cuda")
    row = (cu[:-1, None] + pos).clamp(max=total - 1)                       # [n, L] rows of the padded batch
    real = pos < (cu[1:] - cu[:-1])[:, None]
    at = torch.arange(total, device="cuda")
    seq = torch.searchsorted(cu, at, right=True) - 1                       # a packed row's place in the padded batch
    place = at - cu[seq]

    def pad(x, heads):                                                     # [total, heads*HD] -> [n, heads, L, HD]
        return x[row].float().view(n, L, heads, HD).transpose(1, 2)

    def pack(x, heads):                                                    # back
        return x.transpose(1, 2)[seq, place].reshape(total, heads * HD)

    q, k, v = _views(s)
    q, k, v = pad(q, H).reshape(n, Hk, G * L, HD), pad(k, Hk), pad(v, Hk)
    back = pos[:, None] - pos
    seen = (back >= 0) & (back <= W if W >= 0 else True)
    seen = (seen & real[:, None, :])[:, None, None]                        # [n, 1, 1, L, L]
    scale = HD ** -0.5
    p = (q @ k.transpose(2, 3)).mul_(scale).view(n, Hk, G, L, L).masked_fill_(~seen, float("-inf"))
    m = p.amax(-1, keepdim=True)
    p = p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    p = p.div_(l).view(n, Hk, G * L, L)
    o = p @ v
    lse = (m + l.log()).view(n, H, L).transpose(1, 2)[seq, place].t().contiguous()
    out = {"o": pack(o.view(n, H, L, HD), H).bfloat16(), "lse": lse}
    if s["train"]:
        do = pad(s["dout"], H) * real[:, None, :, None]                    # padding rows have no gradient
        do = do.reshape(n, Hk, G * L, HD)
        p = torch.where(real[:, None, None, :, None], p.view(n, Hk, G, L, L), 0.0).view(n, Hk, G * L, L)
        out["dv"] = pack(p.transpose(2, 3) @ do, Hk).bfloat16()
        ds = (do @ v.transpose(2, 3)).sub_((do * o.nan_to_num()).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        out["dq"] = pack((ds @ k).view(n, H, L, HD), H).bfloat16()
        out["dk"] = pack(ds.transpose(2, 3) @ q, Hk).bfloat16()
    return out


def _prefix_own(s):
    import gpt_transformer_block_b200 as gb
    H, Hk, B = s["heads"], s["kv_heads"], s["batch"]
    o = torch.empty_like(s["q"])
    lse = torch.empty(B, H, dtype=torch.float32, device="cuda")
    ws = torch.empty(gb.gptb_prefix_decode_workspace_bytes(B, H, Hk), dtype=torch.uint8, device="cuda")
    gb.gptb_prefix_decode_attention(s["q"], s["kp"], s["vp"], s["cu_prefix"], s["cu_group"], s["k"], s["v"], s["lens"], o, lse,
                                    H, Hk, s["window"], ws)
    return {"o": o, "lse": lse}


def _prefix_plain(s):
    H, Hk, B, T, W = s["heads"], s["kv_heads"], s["batch"], s["T_max"], s["window"]
    G, n, P, S = H // Hk, s["groups"], s["max_prefix"], s["max_group"]
    cp, cg, lens = s["cu_prefix"].long(), s["cu_group"].long(), s["lens"].long()
    scale = HD ** -0.5
    seq = torch.arange(B, device="cuda")
    group = torch.searchsorted(cg, seq, right=True) - 1
    slot = seq - cg[group]
    plen = (cp[1:] - cp[:-1])[group]                                       # [B]
    newest = plen + lens - 1
    # scores over the prefixes, group by group: [n, Hk, S*G, P] -> [B, Hk, G, P]
    row = (cp[:-1, None] + torch.arange(P, device="cuda")).clamp(max=s["kp"].shape[0] - 1)
    kp = s["kp"][row].float().view(n, P, Hk, HD).transpose(1, 2)
    vp = s["vp"][row].float().view(n, P, Hk, HD).transpose(1, 2)
    q = s["q"].float()
    mate = (cg[:-1, None] + torch.arange(S, device="cuda")).clamp(max=B - 1)
    qg = q[mate].view(n, S, Hk, G, HD).transpose(1, 2).reshape(n, Hk, S * G, HD)
    sp = (qg @ kp.transpose(2, 3)).mul_(scale).view(n, Hk, S, G, P)
    at = torch.arange(P, device="cuda")
    oldest = newest - W if W >= 0 else torch.zeros_like(newest)
    off = (at >= (cp[1:] - cp[:-1])[:, None, None]) | (at < oldest[mate][:, :, None])   # [n, S, P]
    sp.masked_fill_(off[:, None, :, None], float("-inf"))
    # scores over each sequence's own keys: [B, Hk, G, T]
    ko, vo = s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)
    so = (q.view(B, Hk, G, HD) @ ko.transpose(2, 3)).mul_(scale)
    at = torch.arange(T, device="cuda")
    off = (at >= lens[:, None]) | (plen[:, None] + at < oldest[:, None])
    so.masked_fill_(off[:, None, None], float("-inf"))
    m = torch.maximum(sp.amax(-1).transpose(1, 2)[group, slot], so.amax(-1))           # [B, Hk, G]
    mg = m[mate].transpose(1, 2)                                           # [n, Hk, S, G]
    pp, po = sp.sub_(mg[..., None]).exp_(), so.sub_(m[..., None]).exp_()
    l = pp.sum(-1).transpose(1, 2)[group, slot] + po.sum(-1)
    o = (pp.view(n, Hk, S * G, P) @ vp).view(n, Hk, S, G, HD).transpose(1, 2)[group, slot] + po @ vo
    return {"o": (o / l[..., None]).view(B, H, HD).bfloat16(), "lse": (m + l.log()).view(B, H)}


CLIP = 0.2


def _policy_own(s):
    import gpt_transformer_block_b200 as gb
    z = s["logits"]
    dz = torch.empty(z.shape, dtype=z.dtype, device="cuda")
    logp = torch.empty(z.shape[0], dtype=torch.float32, device="cuda")
    stats = torch.empty(3, dtype=torch.float32, device="cuda")
    ws = torch.empty(gb.gptb_policy_loss_workspace_bytes(z.shape[0]), dtype=torch.uint8, device="cuda")
    gb.gptb_policy_loss(z, s["actions"], s["weights"], s["adv"], s["old"], s["ref"] if s["beta"] else None, CLIP, CLIP,
                        s["beta"], dz, logp, stats, ws)
    return {"dlogits": dz, "logp": logp, "stats": stats}


def _policy_plain(s):
    z, a, w, beta = s["logits"].float(), s["actions"].long()[:, None], s["weights"], s["beta"]
    m = z.amax(-1, keepdim=True)
    p = (z - m).exp_()
    l = p.sum(-1, keepdim=True)
    # the ratio is held against the clip borders: 64 bits from here to the row's coefficient
    lp = (z.gather(1, a).double() - m.double() - l.double().log())[:, 0]
    A, r = s["adv"].double(), (lp - s["old"].double()).exp()
    c = r.clamp(1 - CLIP, 1 + CLIP)
    d = s["ref"].double() - lp if beta else torch.zeros_like(lp)
    k = d.exp() - d - 1
    live = w != 0
    kept = r * A <= c * A
    g = torch.where(live, w * (beta * (1 - d.exp()) - torch.where(kept, r * A, 0.0)), 0.0).float()
    dz = p.div_(l).mul_(-g[:, None])
    dz.scatter_add_(1, a, g[:, None])
    loss = (w * (beta * k - torch.minimum(r * A, c * A)))[live].sum()
    stats = torch.stack([loss, (w * k)[live].sum(), (w * (~kept).double())[live].sum()])
    return {"dlogits": dz.to(s["logits"].dtype), "logp": torch.where(live, lp, 0.0).float(), "stats": stats.float()}


def run(state):
    if own:
        return {"packed": _packed_own, "prefix": _prefix_own, "policy": _policy_own}[state["op"]](state)
    return {"packed": _packed_plain, "prefix": _prefix_plain, "policy": _policy_plain}[state["op"]](state)


# ------------------------------------------------------------------ the least a pass needs

def _pairs(n, W):
    """Visible (query, key) pairs of one causal sequence of n tokens, window W."""
    if W < 0 or W >= n:
        return n * (n + 1) // 2
    return (W + 1) * (W + 2) // 2 + (n - W - 1) * (W + 1)


def work(case):
    if case["op"] == "packed":
        H, Hk = case["heads"], case["kv_heads"]
        lens = _lens(case["n"], case["lo"], case["hi"], case["lens_seed"])
        N, pairs = sum(lens), sum(_pairs(n, case["window"]) for n in lens)
        fwd = N * HD * 2 * (2 * H + 2 * Hk) + N * H * 4
        if not case["train"]:
            return {"bytes": fwd, "flops": 4 * HD * H * pairs}
        return {"bytes": fwd + N * HD * 2 * (2 * H + 2 * Hk), "flops": 14 * HD * H * pairs}
    if case["op"] == "prefix":
        H, Hk, W = case["heads"], case["kv_heads"], case["window"]
        plens, sizes = _lens(case["groups"], case["lo"], case["hi"], case["lens_seed"]), _split(case["batch"], case["groups"])
        own_lens, b, rows, pairs = _lens(case["batch"], case["own_lo"], case["own_hi"], case["lens_seed"] + 1), 0, 0, 0
        for p, n in zip(plens, sizes):
            far = 0
            for m in own_lens[b:b + n]:
                first = max(0, p + m - 1 - W) if W >= 0 else 0             # the oldest visible position
                far = max(far, p - min(p, first))
                rows += m - max(0, first - p)
                pairs += p + m - first
            rows += far                                                    # a prefix row is read once for its group
            b += n
        return {"bytes": rows * Hk * HD * 4 + case["batch"] * H * (HD * 4 + 4), "flops": 4 * HD * H * pairs}
    z = 2 if case["dtype"] == "bf16" else 4
    N, V = case["rows"], case["vocab"]
    return {"bytes": int((2 - case["masked"]) * N * V * z) + N * 24, "flops": 8 * N * V * (1 - case["masked"])}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "packed":
        return _packed_exact(s)
    if case["op"] == "prefix":
        return _prefix_exact(s)
    return _policy_exact(s)


def _packed_exact(s):
    H, Hk, W = s["heads"], s["kv_heads"], s["window"]
    N = s["qkv"].shape[0]
    x = s["qkv"].double().view(N, H + 2 * Hk, HD)
    new = lambda heads: torch.zeros(N, heads, HD, dtype=torch.float64, device="cuda")  # noqa: E731
    o, dq, dk, dv = new(H), new(H), new(Hk), new(Hk)
    lse = torch.zeros(H, N, dtype=torch.float64, device="cuda")
    cu = s["cu"].tolist()
    for a, b in zip(cu, cu[1:]):
        i = torch.arange(b - a, device="cuda")
        hidden = i[None] > i[:, None]
        if W >= 0:
            hidden |= i[:, None] - i[None] > W
        for h in range(H):
            kv = h // (H // Hk)
            q, k, v = x[a:b, h], x[a:b, H + kv], x[a:b, H + Hk + kv]
            sc = torch.einsum("id,jd->ij", q, k) / HD ** 0.5
            sc[hidden] = -torch.inf
            lse[h, a:b] = torch.logsumexp(sc, 1)
            pr = torch.softmax(sc, 1)
            o[a:b, h] = pr @ v
            if s["train"]:
                do = s["dout"][a:b].double().view(b - a, H, HD)[:, h]
                dv[a:b, kv] += pr.T @ do
                dp = do @ v.T
                ds = pr * (dp - (pr * dp).sum(1, keepdim=True)) / HD ** 0.5
                dq[a:b, h] = ds @ k
                dk[a:b, kv] += ds.T @ q
    out = {"o": o.view(N, -1), "lse": lse}
    if s["train"]:
        out |= {"dq": dq.view(N, -1), "dk": dk.view(N, -1), "dv": dv.view(N, -1)}
    return out


def _prefix_exact(s):
    H, Hk, B, W = s["heads"], s["kv_heads"], s["batch"], s["window"]
    o = torch.zeros(B, H, HD, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, H, dtype=torch.float64, device="cuda")
    cp, cg, lens = s["cu_prefix"].tolist(), s["cu_group"].tolist(), s["lens"].tolist()
    for g in range(len(cg) - 1):
        kp = s["kp"][cp[g]:cp[g + 1]].double().view(-1, Hk, HD)
        vp = s["vp"][cp[g]:cp[g + 1]].double().view(-1, Hk, HD)
        for b in range(cg[g], cg[g + 1]):
            k = torch.cat([kp, s["k"][b, :lens[b]].double()])
            v = torch.cat([vp, s["v"][b, :lens[b]].double()])
            if W >= 0:
                k, v = k[-(W + 1):], v[-(W + 1):]
            q = s["q"][b].double().view(Hk, H // Hk, HD)
            sc = torch.einsum("kgd,jkd->kgj", q, k) / HD ** 0.5
            lse[b] = torch.logsumexp(sc, -1).view(H)
            o[b] = torch.einsum("kgj,jkd->kgd", torch.softmax(sc, -1), v).reshape(H, HD)
    return {"o": o, "lse": lse}


def _policy_exact(s):
    N, V = s["logits"].shape
    dz = torch.zeros(N, V, dtype=torch.float64, device="cuda")
    logp = torch.zeros(N, dtype=torch.float64, device="cuda")
    loss = kl = clipped = 0.0
    A, w, old, ref = (s[n].double() for n in ("adv", "weights", "old", "ref"))
    live = w != 0
    for i in range(0, N, 1024):                                            # rows at a time, for memory
        j = slice(i, min(N, i + 1024))
        lz = torch.log_softmax(s["logits"][j].double(), -1)
        hot = torch.zeros_like(lz).scatter_(1, s["actions"][j].long()[:, None], 1.0)
        lp = (lz * hot).sum(-1)
        ratio = torch.exp(lp - old[j])
        plain, capped = ratio * A[j], torch.clip(ratio, 1 - CLIP, 1 + CLIP) * A[j]
        slope = torch.where(plain <= capped, -plain, torch.zeros_like(plain))
        k = torch.zeros_like(lp)
        if s["beta"]:
            k = torch.expm1(ref[j] - lp) - (ref[j] - lp)
            slope = slope - s["beta"] * torch.expm1(ref[j] - lp)
        wj = torch.where(live[j], w[j], torch.zeros_like(lp))
        loss = loss + (wj * (s["beta"] * k - torch.minimum(plain, capped))).sum()
        kl, clipped = kl + (wj * k).sum(), clipped + wj[plain > capped].sum()
        dz[j] = (wj * slope)[:, None] * (hot - lz.exp())
        logp[j] = torch.where(live[j], lp, torch.zeros_like(lp))
    return {"dlogits": dz, "logp": logp, "stats": torch.stack([loss, kl, clipped])}
