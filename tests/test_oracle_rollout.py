"""Pins of oracle/rollout.py, CPU only: packed attention against the model's
attention on each sequence alone, torch's scaled_dot_product_attention with
autograd and central differences; the shared-prefix decode step against the
plain decode step on the concatenated cache; the policy loss against torch
autograd written from its definition, differences, and its special cases."""
import numpy as np
import pytest
import torch

from oracle import decode as od
from oracle import model as om
from oracle import rollout as orl


def _packed(seed, lens, H=4, Hk=2, hd=8):
    rng = np.random.default_rng(seed)
    n = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    return (rng.standard_normal((n, H, hd)), rng.standard_normal((n, Hk, hd)), rng.standard_normal((n, Hk, hd)), cu,
            rng.standard_normal((n, H, hd)))


@pytest.mark.parametrize("window", [-1, 0, 3, 100])
def test_each_sequence_is_the_models_attention_on_it_alone(window):
    q, k, v, cu, _ = _packed(1, [5, 0, 1, 12, 7])
    r = orl.packed_attention(q, k, v, cu, window)
    for a, b in zip(cu[:-1], cu[1:]):
        if a < b:
            o, lse = om.attention_forward(q[None, a:b], k[None, a:b], v[None, a:b], window)
            assert np.allclose(r["o"][a:b], o[0], atol=1e-12)
            assert np.allclose(r["lse"][:, a:b], lse[0], atol=1e-12)


@pytest.mark.parametrize("window", [-1, 2])
def test_packed_gradients_match_autograd(window):
    q, k, v, cu, do = _packed(2, [6, 1, 9])
    r = orl.packed_attention(q, k, v, cu, window, do)
    tq, tk, tv = (torch.tensor(x, requires_grad=True) for x in (q, k, v))
    seq = np.searchsorted(cu, np.arange(len(q)), side="right")
    i = np.arange(len(q))
    mask = (seq[:, None] == seq[None]) & (i[None] <= i[:, None])
    if window >= 0:
        mask &= i[:, None] - i[None] <= window
    o = torch.nn.functional.scaled_dot_product_attention(
        tq.transpose(0, 1), tk.repeat_interleave(2, 1).transpose(0, 1), tv.repeat_interleave(2, 1).transpose(0, 1),
        attn_mask=torch.tensor(mask)).transpose(0, 1)
    (o * torch.tensor(do)).sum().backward()
    assert np.allclose(r["o"], o.detach().numpy(), atol=1e-12)
    for n, t in (("dq", tq), ("dk", tk), ("dv", tv)):
        assert np.allclose(r[n], t.grad.numpy(), atol=1e-11)


def test_packed_gradients_match_differences():
    q, k, v, cu, do = _packed(3, [4, 5], H=2, Hk=1, hd=4)
    r = orl.packed_attention(q, k, v, cu, 2, do)
    f = lambda: (orl.packed_attention(q, k, v, cu, 2)["o"] * do).sum()  # noqa: E731
    for n, x in (("dq", q), ("dk", k), ("dv", v)):
        num = np.zeros_like(x)
        for at in np.ndindex(*x.shape):
            keep = x[at]
            x[at] = keep + 1e-5
            up = f()
            x[at] = keep - 1e-5
            num[at] = (up - f()) / 2e-5
            x[at] = keep
        assert np.allclose(r[n], num, atol=1e-8)


@pytest.mark.parametrize("window", [-1, 0, 4, 9, 1000])
def test_prefix_decode_is_the_plain_decode_step_on_the_joined_cache(window):
    rng = np.random.default_rng(4)
    H, Hk, hd, T = 4, 2, 8, 6
    cp, cg = [0, 7, 7, 12], [0, 2, 3, 5]  # the second prompt is empty; sequence 5 has none
    B = 6
    lens = [1, 6, 3, 2, 5, 4]
    q = rng.standard_normal((B, H, hd))
    kp, vp = rng.standard_normal((2, 12, Hk, hd))
    k, v = rng.standard_normal((2, B, T, Hk, hd))
    o, lse, _ = orl.prefix_decode(q, kp, vp, cp, cg, k, v, lens, window)
    for b, (a, e) in enumerate([(0, 7), (0, 7), (7, 7), (7, 12), (7, 12), (0, 0)]):
        K, V = (np.concatenate([x[a:e], y[b, :lens[b]]])[None] for x, y in ((kp, k), (vp, v)))
        ro, rl = od.decode_attention(q[b:b + 1], K, V, [K.shape[1]], window)
        assert np.allclose(o[b], ro[0], atol=1e-12) and np.allclose(lse[b], rl[0], atol=1e-12)


def _policy(seed, N=12, V=9, beta=0.1):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((N, V)) * 2
    a = rng.integers(0, V, N)
    lp = orl.token_logprobs(z, a)
    w = rng.random(N) * (rng.random(N) > 0.2)
    return z, a, w, rng.standard_normal(N), lp + 0.3 * rng.standard_normal(N), lp + 0.5 * rng.standard_normal(N), 0.2, 0.3, beta


@pytest.mark.parametrize("beta", [0.0, 0.1])
def test_policy_loss_matches_autograd(beta):
    z, a, w, A, old, ref, lo, hi, _ = args = _policy(5, beta=beta)
    args = args[:8] + (beta,)
    loss, kl, clipped, lp, dz, _, _ = orl.policy_loss(*args)
    t = torch.tensor(z, requires_grad=True)
    tl = torch.log_softmax(t, -1)[torch.arange(len(a)), torch.tensor(a)]
    r = (tl - torch.tensor(old)).exp()
    s = torch.minimum(r * torch.tensor(A), r.clamp(1 - lo, 1 + hi) * torch.tensor(A))
    d = torch.tensor(ref) - tl
    k = d.exp() - d - 1
    ref_loss = (torch.tensor(w) * (-s + beta * k)).sum()
    ref_loss.backward()
    assert np.isclose(loss, ref_loss.item(), atol=1e-12) and np.isclose(kl, (torch.tensor(w) * k).sum().item())
    assert np.allclose(dz, t.grad.numpy(), atol=1e-12)
    assert np.allclose(lp[w != 0], tl.detach().numpy()[w != 0], atol=1e-12)


def test_policy_gradient_matches_differences():
    z, *rest = _policy(6, N=5, V=6)
    *_, dz, _, gap = orl.policy_loss(z, *rest)
    assert gap.min() > 1e-3  # no ratio next to a clip border
    for at in np.ndindex(*z.shape):
        keep = z[at]
        z[at] = keep + 1e-6
        up = orl.policy_loss(z, *rest)[0]
        z[at] = keep - 1e-6
        num = (up - orl.policy_loss(z, *rest)[0]) / 2e-6
        z[at] = keep
        assert np.isclose(dz[at], num, atol=1e-8)


def test_policy_special_cases():
    z, a, w, A, old, ref, lo, hi, beta = _policy(7)
    lp = orl.token_logprobs(z, a)
    # on-policy without KL: the plain policy gradient, nothing clipped, loss -sum w A
    loss, kl, clipped, _, dz, g, _ = orl.policy_loss(z, a, w, A, lp, None, lo, hi, 0.0)
    assert np.isclose(loss, -(w * A).sum()) and kl == 0 and clipped == 0 and np.allclose(g, -w * A)
    # the reference policy itself: no KL and no gradient from it
    assert np.isclose(orl.policy_loss(z, a, w, A * 0, lp, lp, lo, hi, 0.5)[0], 0.0)
    # rows sum to zero, weightless rows and rows without a valid action are zero
    assert np.allclose(dz.sum(-1), 0, atol=1e-12) and np.all(dz[w == 0] == 0)
    a2 = a.copy()
    a2[np.flatnonzero(w)[0]] = z.shape[1]
    assert np.all(orl.policy_loss(z, a2, w, A, lp, None, lo, hi, 0.0)[4][np.flatnonzero(w)[0]] == 0)
    # a ratio past the upper border with a positive advantage is clipped, with a negative one it is not
    one = lambda adv: orl.policy_loss(z[:1], a[:1], [1.0], [adv], lp[:1] - 1.0, None, lo, hi, 0.0)  # noqa: E731
    assert one(1.0)[2] == 1.0 and np.all(one(1.0)[4] == 0) and np.isclose(one(1.0)[0], -(1 + hi))
    assert one(-1.0)[2] == 0.0 and np.isclose(one(-1.0)[0], np.e)
