"""Inputs of the rollout operators' tests (no method arithmetic here)."""
import numpy as np
import torch

BF = torch.bfloat16


def normed(g, *shape):
    """Vectors of RMS 1, as the QK normalisation leaves them."""
    x = torch.randn(*shape, generator=g)
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True))).to(BF)


def offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def packed(lens, H, Hk, seed=0, pad=0, junk=float("nan")):
    """qkv [total + pad, (H + 2 Hk) * 128] and dout on the device (rows behind the last sequence hold `junk`), cu."""
    g = torch.Generator().manual_seed(seed)
    n = int(sum(lens))
    qkv = torch.cat([normed(g, n, H + Hk, 128), torch.randn(n, Hk, 128, generator=g).to(BF)], 1).view(n, (H + 2 * Hk) * 128)
    dout = torch.randn(n, H * 128, generator=g).to(BF)
    if pad:
        qkv = torch.cat([qkv, torch.full((pad, qkv.shape[1]), junk, dtype=BF)])
        dout = torch.cat([dout, torch.full((pad, dout.shape[1]), junk, dtype=BF)])
    return qkv.cuda(), dout.cuda(), torch.tensor(offsets(lens)).cuda()


def qkv_views(qkv, H, Hk):
    return qkv[:, :H * 128], qkv[:, H * 128:(H + Hk) * 128], qkv[:, (H + Hk) * 128:]


def heads(t, n):
    """[rows, n*128] device tensor -> fp64 numpy [rows, n, 128]."""
    return t.double().cpu().numpy().reshape(t.shape[0], n, 128)


def prefix_case(plens, sizes, lens, T, H, Hk, seed=0, extra=0, junk=float("nan")):
    """Inputs of a shared-prefix decode step on the device; cache rows from lens[b] on hold `junk`; `extra` sequences
    at the end belong to no group."""
    g = torch.Generator().manual_seed(seed)
    B, P = sum(sizes) + extra, int(sum(plens))
    assert len(lens) == B
    d = {"q": normed(g, B, H, 128), "kp": normed(g, P, Hk, 128).view(P, Hk * 128),
         "vp": torch.randn(P, Hk * 128, generator=g).to(BF),
         "k": normed(g, B, T, Hk, 128), "v": torch.randn(B, T, Hk, 128, generator=g).to(BF)}
    for b, n in enumerate(lens):
        if 0 <= n < T:
            d["k"][b, n:] = junk
            d["v"][b, n:] = junk
    d = {n: t.cuda() for n, t in d.items()}
    d |= {n: torch.tensor(x, dtype=torch.int32).cuda() for n, x in
          (("cp", offsets(plens)), ("cg", offsets(sizes)), ("lens", np.array(lens, dtype=np.int32)))}
    return d


def policy_case(N, V, dtype, seed=0, pad=0, offset=0, masked=0.25):
    """Logits [N, V] whose rows start `offset` elements into rows of V + pad, and the per-row arrays, on the device."""
    g = torch.Generator().manual_seed(seed)
    z = (2.0 * torch.randn(N, V + pad, generator=g)).to(dtype).cuda()
    z = z[:, offset:offset + V]
    a = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    z[torch.arange(N), a.long()] += 5.0
    lp = torch.log_softmax(z.double(), -1).cpu()[torch.arange(N), a.long()]
    old = lp + 0.2 * torch.randn(N, generator=g)
    r = (lp - old).exp()  # no ratio next to a clip border (1 - 0.2, 1 + 0.3)
    old[torch.minimum((r - 0.8).abs(), (r - 1.3).abs()) < 1e-3] += 0.01
    w = torch.rand(N, generator=g) / N * (torch.rand(N, generator=g) >= masked)
    d = {"z": z, "a": a, "w": w, "A": torch.randn(N, generator=g),
         "old": old.float(), "ref": (lp + 0.5 * torch.randn(N, generator=g)).float()}
    return {n: t.cuda() for n, t in d.items()}
