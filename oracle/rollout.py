"""fp64 oracle for sampling several answers to a prompt and learning from them
— TEST INFRASTRUCTURE ONLY (same rules as the rest of ``oracle``): attention
over packed sequences (forward, backward), one decode step over a shared prompt
and the sequence's own cache, and the clipped policy loss with a KL term.

Sources: the causal, windowed, grouped-query attention is that of
``oracle.model`` (apidog.com/fr "Comment Entraîner Votre Propre ChatGPT Pour
50€ ?", § "Comment nanochat fonctionne" › 5), applied to one sequence at a time.
The loss is the clipped surrogate of J. Schulman et al., "Proximal Policy
Optimization Algorithms" (2017), with the estimator exp(d) - d - 1,
d = lp_ref - lp, of the KL divergence from the reference policy (J. Schulman,
"Approximating KL Divergence", 2020).

Besides its results every attention function returns bounds of the error that
rounding P and dS to bf16, as a matrix unit wants them, and o (from which D is
formed) may cause: u = 2^-8 per rounding, relative.
"""
import numpy as np

U = 2.0 ** -8  # half a step of bf16, relative


def _visible(n, window):
    i = np.arange(n)
    m = i[None, :] <= i[:, None]
    if window is not None and window >= 0:
        m &= i[:, None] - i[None, :] <= window
    return m


def _softmax(s):
    m = s.max(-1, keepdims=True)
    e = np.exp(s - m)
    z = e.sum(-1, keepdims=True)
    return e / z, (m + np.log(z))[..., 0]


def packed_attention(q, k, v, cu, window, dout=None):
    """q, dout [N,H,hd]; k, v [N,Hkv,hd]; cu offsets -> dict of o, lse [H,N] (with dout: dq, dk, dv) and ``err``, the
    bound of each one's rounding error.  Rows outside the sequences stay 0."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    N, H, hd = q.shape
    Hk = k.shape[1]
    G, scale = H // Hk, 1.0 / np.sqrt(hd)
    out = {"o": np.zeros_like(q), "lse": np.zeros((H, N))}
    err = {"o": np.zeros_like(q)}
    if dout is not None:
        dout = np.asarray(dout, dtype=np.float64)
        for n, x in (("dq", q), ("dk", k), ("dv", v)):
            out[n], err[n] = np.zeros_like(x), np.zeros_like(x)
    for a, b in zip(cu[:-1], cu[1:]):
        a, b = int(a), int(b)
        if a == b:
            continue
        seen = _visible(b - a, window)
        for h in range(H):
            kv = h // G
            Q, K, V = q[a:b, h], k[a:b, kv], v[a:b, kv]
            P, lse = _softmax(np.where(seen, Q @ K.T * scale, -np.inf))
            o = P @ V
            out["o"][a:b, h], out["lse"][h, a:b] = o, lse
            eo = U * (P @ np.abs(V)) + U * np.abs(o)
            err["o"][a:b, h] = eo
            if dout is None:
                continue
            dO = dout[a:b, h]
            dP = dO @ V.T
            D = (dO * o).sum(-1, keepdims=True)
            dS = P * (dP - D) * scale
            out["dq"][a:b, h] = dS @ K
            out["dk"][a:b, kv] += dS.T @ Q
            out["dv"][a:b, kv] += P.T @ dO
            eS = U * np.abs(dS) + P * (np.abs(dO) * eo).sum(-1, keepdims=True) * scale
            err["dq"][a:b, h] = eS @ np.abs(K)
            err["dk"][a:b, kv] += eS.T @ np.abs(Q)
            err["dv"][a:b, kv] += U * P.T @ np.abs(dO)
    for n in ("dq", "dk", "dv"):
        if n in out:
            err[n] += U * np.abs(out[n])
    out["err"] = err
    return out


def prefix_decode(q, k_prefix, v_prefix, cu_prefix, cu_group, k_cache, v_cache, lens, window):
    """q [B,H,hd]; k_prefix, v_prefix [rows,Hkv,hd]; k_cache, v_cache [B,T,Hkv,hd] -> o, lse [B,H], bound of o's error."""
    q, k_prefix, v_prefix, k_cache, v_cache = (np.asarray(x, dtype=np.float64) for x in
                                               (q, k_prefix, v_prefix, k_cache, v_cache))
    B, H, hd = q.shape
    T, Hk = k_cache.shape[1], k_cache.shape[2]
    o, lse, err = np.zeros_like(q), np.full((B, H), -np.inf), np.zeros_like(q)
    for b in range(B):
        n = int(lens[b])
        if n < 0 or n > T:
            continue
        a = e = 0
        for g in range(len(cu_group) - 1):
            if cu_group[g] <= b < cu_group[g + 1]:
                a, e = int(cu_prefix[g]), int(cu_prefix[g + 1])
        K = np.concatenate([k_prefix[a:e], k_cache[b, :n]])
        V = np.concatenate([v_prefix[a:e], v_cache[b, :n]])
        first = max(0, len(K) - 1 - window) if window is not None and window >= 0 else 0
        if len(K) == first:
            continue
        for h in range(H):
            kv = h // (H // Hk)
            P, lse[b, h] = _softmax(K[first:, kv] @ q[b, h] / np.sqrt(hd))
            o[b, h] = P @ V[first:, kv]
            err[b, h] = U * (P @ np.abs(V[first:, kv])) + U * np.abs(o[b, h])
    return o, lse, err


def token_logprobs(z, tokens):
    z = np.asarray(z, dtype=np.float64)
    z = z - z.max(-1, keepdims=True)  # (first: z - lse loses lse where a whole row is the type's lowest value)
    return z[np.arange(len(z)), tokens] - np.log(np.exp(z).sum(-1))


def policy_loss(z, actions, weights, adv, lp_old, lp_ref, clip_lo, clip_hi, beta):
    """-> loss, KL, clipped weight, lp [N], dz [N,V], the coefficient g [N] and the ratios' distances from the clip borders."""
    z = np.asarray(z, dtype=np.float64)
    N, V = z.shape
    lp_all = np.zeros(N)
    dz, g = np.zeros_like(z), np.zeros(N)
    gap = np.full(N, np.inf)
    loss = kl = clipped = 0.0
    for i in range(N):
        w, A = float(weights[i]), float(adv[i])
        if w == 0.0 or not 0 <= actions[i] < V:
            continue
        p, _ = _softmax(z[i][None])
        lp = token_logprobs(z[i][None], [actions[i]])[0]
        r = np.exp(lp - float(lp_old[i]))
        lo, hi = 1.0 - clip_lo, 1.0 + clip_hi
        un, cl = r * A, min(max(r, lo), hi) * A
        d = float(lp_ref[i]) - lp if lp_ref is not None else 0.0
        k = np.exp(d) - d - 1.0
        slope = (-un if un <= cl else 0.0) + beta * (1.0 - np.exp(d))
        loss += w * (-min(un, cl) + beta * k)
        kl += w * k
        clipped += w if un > cl else 0.0
        g[i] = w * slope
        dz[i] = -g[i] * p[0]
        dz[i, actions[i]] += g[i]
        lp_all[i] = lp
        gap[i] = min(abs(r - lo), abs(r - hi))
    return loss, kl, clipped, lp_all, dz, g, gap
