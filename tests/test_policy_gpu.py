"""The policy loss and the tokens' log-probabilities through the C ABI against
the fp64 oracle.  Tolerances: lp within e = 2e-5 (the sum of exponentials: at
most 100 additions in a row and 20 across threads, each off by 2^-24, the
exponentials by 2^-21 with their rounded arguments: 1.3e-5 in all); dz within
what that changes of g and of the softmax, 4 e |g| (onehot + p) with g's
magnitude w (|r A| + beta (1 + exp d)), plus half a step of its type; the sums
within 4 e of the sum of their terms' magnitudes.  No input has a ratio within
1e-4 of a clip border."""
import numpy as np
import pytest
import torch

from oracle import rollout as orl
from rollout_inputs import policy_case

pytestmark = pytest.mark.gpu

E = 2e-5


def call(gb, d, lo=0.2, hi=0.3, beta=0.1, ref=True, out="new"):
    z = d["z"]
    n = z.shape[0]
    dz = {"new": torch.full(z.shape, 7.0, dtype=z.dtype, device="cuda"), "same": z, None: None}[out] if isinstance(out, (str, type(None))) else out
    logp, stats = torch.full((n,), 7.0, device="cuda"), torch.full((3,), 7.0, device="cuda")
    ws = torch.full((gb.gptb_policy_loss_workspace_bytes(n),), 255, dtype=torch.uint8, device="cuda")
    gb.gptb_policy_loss(z, d["a"], d["w"], d["A"], d["old"], d["ref"] if ref else None, lo, hi, beta, dz, logp, stats, ws)
    return dz, logp, stats


def check(gb, d, lo=0.2, hi=0.3, beta=0.1, ref=True, out="new"):
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    z, a, w, A, old, rf = f(d["z"]), d["a"].cpu().numpy(), f(d["w"]), f(d["A"]), f(d["old"]), f(d["ref"])
    loss, kl, clipped, lp, rz, g, gap = orl.policy_loss(z, a, w, A, old, rf if ref else None, lo, hi, beta)
    assert gap.min() > 1e-4
    half = torch.finfo(d["z"].dtype).eps / 2
    dz, logp, stats = call(gb, d, lo, hi, beta, ref, out)
    live = (w != 0) & (a >= 0) & (a < z.shape[1])
    assert np.abs(f(logp) - lp).max() <= E + 2e-7 * np.abs(lp).max()
    assert torch.all(logp[torch.tensor(~live)] == 0)
    if dz is not None:
        got = f(dz)
        r, d_ = np.exp(lp - old), (rf - lp) if ref else np.zeros_like(lp)
        big = np.abs(w) * (np.abs(r * A) + beta * (1 + np.exp(d_)))
        p = np.exp(z - z.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        p[np.arange(len(a))[live], a[live]] += 1
        slack = 4 * E * big[:, None] * p + half * np.abs(rz) + 1e-38
        assert np.all(np.abs(got - rz) <= slack * 1.02), (np.abs(got - rz) / slack).max()
        assert np.all(got[~live] == 0)
    r, d_ = np.exp(lp - old), (rf - lp) if ref else np.zeros_like(lp)
    terms = (np.abs(w) * (np.abs(r * A) + np.abs(A) + beta * (np.exp(d_) + np.abs(d_) + 1)))[live].sum()
    s = f(stats)
    assert abs(s[0] - loss) <= 4 * E * terms + 2.0 ** -24 * abs(loss)
    assert abs(s[1] - kl) <= 4 * E * (np.abs(w) * (np.exp(d_) + np.abs(d_) + 1))[live].sum()
    assert abs(s[2] - clipped) <= 1e-6 * np.abs(w).sum()
    return dz, logp, stats


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,V,pad,offset", [(1, 1, 0, 0), (3, 7, 0, 0), (9, 64, 0, 0), (40, 1000, 24, 0), (17, 4099, 0, 0),
                                            (5, 4096, 3, 1), (6, 32768, 0, 0), (4, 50257, 47, 0), (3, 70001, 0, 0),
                                            (3, 140000, 8, 8)])
def test_policy_loss(cuda_lib, dtype, N, V, pad, offset):
    check(cuda_lib, policy_case(N, V, dtype, seed=N + V, pad=pad, offset=offset, masked=0.0 if N < 4 else 0.25))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_rows(cuda_lib, dtype):
    """More rows than the persistent grid has CTAs, most of them without weight in the second case."""
    check(cuda_lib, policy_case(1500, 520, dtype, seed=1))
    check(cuda_lib, policy_case(1500, 520, dtype, seed=2, masked=0.95))


@pytest.mark.parametrize("beta,ref", [(0.0, False), (0.0, True), (0.5, True)])
def test_without_and_with_the_kl_term(cuda_lib, beta, ref):
    check(cuda_lib, policy_case(30, 300, torch.float32, seed=3), beta=beta, ref=ref)


@pytest.mark.parametrize("lo,hi", [(0.0, 0.0), (1.0, 10.0)])
def test_clip_borders(cuda_lib, lo, hi):
    check(cuda_lib, policy_case(30, 300, torch.float32, seed=4), lo=lo, hi=hi)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,pad,offset", [(1024, 0, 0), (333, 0, 0), (333, 30, 5), (32768, 8, 0)])
def test_gradient_over_the_logits_and_none_at_all(cuda_lib, dtype, V, pad, offset):
    gb = cuda_lib
    d = policy_case(8, V, dtype, seed=5, pad=pad, offset=offset)
    dz, logp, stats = check(gb, d)
    # vectors are cut at the gradient's alignment, so where it lies otherwise than the logits the sums are taken in
    # another order: each result is within E of the exact one, two of them within 2 E of each other
    alike = offset == 0
    same = torch.equal if alike else lambda x, y: bool((x - y).abs().max() <= 2 * E)
    _, lp0, st0 = call(gb, d, out=None)
    assert same(lp0, logp) and same(st0, stats)
    over, lp1, st1 = check(gb, d, out="same")  # overwrites the logits
    assert over is d["z"] and torch.equal(lp1, lp0) and torch.equal(st1, st0)
    assert not alike or torch.equal(over, dz)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_rows_elsewhere_aligned_than_the_logits(cuda_lib, dtype):
    gb = cuda_lib
    d = policy_case(6, 901, dtype, seed=6, pad=11, offset=0)
    for pad, offset in ((0, 0), (7, 3), (11, 8)):
        box = torch.full((6, 901 + pad), 7.0, dtype=dtype, device="cuda")
        check(gb, d, out=box[:, offset:offset + 901])
        assert torch.all(box[:, :offset] == 7.0) and torch.all(box[:, offset + 901:] == 7.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_that_do_not_count_are_not_read(cuda_lib, dtype):
    """NaN logits, advantages and ratios in rows of weight 0; actions outside the vocabulary are reported."""
    gb = cuda_lib
    d = policy_case(12, 200, dtype, seed=7, masked=0.0)
    base = {n: t.clone() for n, t in d.items()}
    off = torch.tensor([0, 5, 11], device="cuda")
    d["w"][off] = 0
    base["w"][off] = 0
    for n in ("z", "A", "old", "ref"):
        d[n][off] = float("nan")
    for x, y in zip(call(gb, d), call(gb, base)):
        assert torch.equal(x, y) and bool(torch.isfinite(x.float()).all())
    d["a"][5] = -1  # in a row without weight: nothing to report
    call(gb, d)
    assert gb.gptb_device_error() == 0
    for bad in (-1, 200, 2 ** 31 - 1):
        base["a"][3] = bad
        dz, logp, stats = check(gb, base)
        assert gb.gptb_device_error() == gb.ERR_BAD_INPUT
        assert torch.all(dz[3] == 0) and logp[3] == 0


def test_logits_of_minus_infinity(cuda_lib):
    """Forbidden tokens: probability and gradient 0."""
    gb = cuda_lib
    for dtype in (torch.bfloat16, torch.float32):
        d = policy_case(6, 5000, dtype, seed=8, masked=0.0)
        gone = torch.rand(5000, device="cuda") < 0.7
        gone[:2048] = True  # whole strips of a thread
        gone[d["a"].long()] = False
        d["z"][:, gone] = float("-inf")
        lp = torch.log_softmax(d["z"].double(), -1)[torch.arange(6), d["a"].long()]
        d["old"], d["ref"] = (lp + 0.1).float(), (lp - 0.2).float()
        dz, logp, _ = call(gb, d)
        assert torch.all(dz[:, gone] == 0) and bool(torch.isfinite(dz).all())
        assert (logp.double() - lp).abs().max() <= E + 2e-7 * lp.abs().max()
        assert dz.double().sum(-1).abs().max() <= 2 ** -8 * dz.double().abs().sum(-1).max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,V", [(1, 5), (700, 333), (20, 32768)])
def test_token_logprobs(cuda_lib, dtype, N, V):
    gb = cuda_lib
    d = policy_case(N, V, dtype, seed=9)
    logp = torch.full((N,), 7.0, device="cuda")
    gb.gptb_token_logprobs(d["z"], d["a"], logp)
    want = orl.token_logprobs(d["z"].double().cpu().numpy(), d["a"].cpu().numpy())
    assert np.abs(logp.double().cpu().numpy() - want).max() <= E + 2e-7 * np.abs(want).max()
    assert gb.gptb_device_error() == 0


def test_policy_captured_step(cuda_lib):
    gb = cuda_lib
    d = policy_case(64, 900, torch.bfloat16, seed=10)
    torch.cuda.synchronize()
    call(gb, d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call(gb, d)
    new = policy_case(64, 900, torch.bfloat16, seed=11)
    for n in d:
        d[n].copy_(new[n])
    for _ in range(2):
        graph.replay()
    for x, y in zip(outs, call(gb, new)):
        assert torch.equal(x, y)


def test_policy_no_rows(cuda_lib):
    gb = cuda_lib
    d = policy_case(1, 8, torch.float32)
    _, _, stats = call(gb, {n: t[:0] for n, t in d.items()})
    assert torch.all(stats == 0)
    gb.gptb_token_logprobs(d["z"][:0], d["a"][:0], torch.empty(0, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [600, 40001])
def test_logits_of_the_types_lowest_and_large_ones(cuda_lib, dtype, V):
    """Rows masked with the type's lowest value, in part and whole (a uniform softmax), and logits around 1e4."""
    gb = cuda_lib
    d = policy_case(5, V, dtype, seed=12, masked=0.0)
    low = torch.finfo(dtype).min
    a = d["a"].long()
    d["z"][0] = low
    keep = d["z"][1].clone()
    d["z"][1, : V // 2] = low
    d["z"][1, a[1]] = keep[a[1]]
    d["z"][2] = low
    d["z"][2, a[2]] = 1.0
    d["z"][3] += 1e4
    d["z"][4] = float("-inf")
    d["z"][4, a[4]] = low
    lp = torch.log_softmax(d["z"].double(), -1)[torch.arange(5), a]
    d["old"], d["ref"] = (lp + 0.05).float(), (lp - 0.1).float()
    check(gb, d)
