"""The policy loss and the tokens' log-probabilities on rows with large finite
logits: the usual mask fills, in part of a row and in all of it, in what a CTA
holds and in what it does not, and rows whose values lie far from zero but close
to each other.  Tolerances: those of test_policy_gpu.py; far from zero the
exponent (z - m) log2(e) is rounded twice, at most 88 * 1.45 * 2^-23 = 1.6e-5 in
base 2 where the exponential is not 0, next to the 4 E = 8e-5 that an element of
the gradient is allowed."""
import numpy as np
import pytest
import torch

from oracle import rollout as orl
from rollout_inputs import policy_case
from test_policy_gpu import E, check

pytestmark = pytest.mark.gpu


def on_policy(d):
    """Old and reference log-probabilities next to the logits' own."""
    rows = torch.arange(d["z"].shape[0], device="cuda")
    lp = torch.log_softmax(d["z"].double(), -1)[rows, d["a"].long()]
    d["old"], d["ref"] = (lp + 0.05).float(), (lp - 0.1).float()


def check_all(gb, d):
    on_policy(d)
    z, a = d["z"].clone(), d["a"]
    check(gb, d)
    check(gb, d, out="same")
    d["z"] = z
    logp = torch.full((z.shape[0],), 7.0, device="cuda")
    gb.gptb_token_logprobs(z, a, logp)
    want = orl.token_logprobs(z.double().cpu().numpy(), a.cpu().numpy())
    assert np.abs(logp.double().cpu().numpy() - want).max() <= E + 2e-7 * np.abs(want).max()
    assert gb.gptb_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,pad,offset", [(600, 0, 0), (4099, 5, 3), (33001, 0, 0), (140000, 8, 8)])
@pytest.mark.parametrize("fill", [-1e4, -1e6, -1e9, -3e9, -1e10, -1e20, -1e30, -9e37])
def test_rows_masked_with_a_large_fill(cuda_lib, dtype, V, pad, offset, fill):
    """Row 0: all but the action; 1: the first half, so whole strips of a thread; 2: the second half, what a long row's
    CTA does not hold; 3: the whole row, a uniform softmax; 4: nine of ten, at random."""
    d = policy_case(5, V, dtype, seed=20, pad=pad, offset=offset, masked=0.0)
    z, a = d["z"], d["a"].long()
    keep = z[torch.arange(5), a].clone()
    z[0] = fill
    z[1, : V // 2] = fill
    z[2, V // 2:] = fill
    z[3] = fill
    z[4, torch.rand(V, generator=torch.Generator().manual_seed(21)).cuda() < 0.9] = fill
    for i in (0, 1, 2, 4):
        z[i, a[i]] = keep[i]
    check_all(cuda_lib, d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [600, 140001])
@pytest.mark.parametrize("top", [1e6, 3e9, 1e10, 1e20, 1e30, 9e37])
def test_rows_whose_largest_logits_are_far_from_zero(cuda_lib, dtype, V, top):
    """The action and some others at `top`: early, late, everywhere; the last row has its `top` after -top."""
    d = policy_case(4, V, dtype, seed=22, masked=0.0)
    z, a = d["z"], d["a"].long()
    z[0, :3] = top
    z[1, V - 3:] = top
    z[2, ::7] = top
    z[3, : V - 5] = -top
    z[torch.arange(4), a] = top
    check_all(cuda_lib, d)


@pytest.mark.parametrize("V", [600, 140001])
@pytest.mark.parametrize("base", [2.0 ** 19, -(2.0 ** 21), 2.0 ** 25, -(2.0 ** 28), 2.0 ** 29, 2.0 ** 31])
def test_close_logits_far_from_zero(cuda_lib, V, base):
    """fp32 rows around `base` whose neighbours a few steps of the type apart count for one another."""
    d = policy_case(3, V, torch.float32, seed=23, masked=0.0)
    step = max(2.0 ** -2, abs(base) * 2.0 ** -23)
    k = torch.randint(0, 12, (3, V), generator=torch.Generator().manual_seed(24)).cuda()
    d["z"] = (base - step * k.double()).float()
    d["z"][torch.arange(3), d["a"].long()] = base
    check_all(cuda_lib, d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("z_a", [-2000.0, float("-inf")])
def test_reference_without_its_term(cuda_lib, dtype, z_a):
    """beta 0 with a reference (the KL is only watched): an action that the policy has all but given up gives the loss,
    the gradient and the clipped weight of a call without reference."""
    gb = cuda_lib
    d = policy_case(6, 700, dtype, seed=25, masked=0.0)
    d["z"][2, d["a"][2].long()] = z_a
    lp = torch.log_softmax(d["z"].double(), -1)[torch.arange(6), d["a"].long()]
    d["old"] = (lp.clamp(min=-3000.0) + 0.05).float()
    out = []
    for ref in (d["ref"], None):
        dz, logp, stats = torch.empty_like(d["z"]), torch.empty(6, device="cuda"), torch.empty(3, device="cuda")
        ws = torch.empty(gb.gptb_policy_loss_workspace_bytes(6), dtype=torch.uint8, device="cuda")
        gb.gptb_policy_loss(d["z"], d["a"], d["w"], d["A"], d["old"], ref, 0.2, 0.3, 0.0, dz, logp, stats, ws)
        out.append((dz, logp, stats))
    (dz, logp, stats), (dz0, logp0, stats0) = out
    assert bool(torch.isfinite(dz).all()) and torch.equal(dz, dz0) and torch.equal(logp, logp0)
    assert bool(torch.isfinite(stats[0])) and stats[0] == stats0[0] and stats[2] == stats0[2]
    assert stats[1] == float("inf") and stats0[1] == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [333, 4099, 50257])
@pytest.mark.parametrize("pad,offset", [(0, 0), (30, 5), (11, 8)])
def test_where_the_gradient_goes_changes_no_result(cuda_lib, dtype, V, pad, offset):
    """No gradient, one in an array of its own, in rows that lie otherwise, over the logits: the same bits (vectors are
    cut at the logits' alignment, whatever the gradient's is)."""
    gb = cuda_lib
    d = policy_case(7, V, dtype, seed=26, pad=pad, offset=offset)
    n = d["z"].shape[0]

    def call(dz):
        logp, stats = torch.full((n,), 7.0, device="cuda"), torch.full((3,), 7.0, device="cuda")
        ws = torch.empty(gb.gptb_policy_loss_workspace_bytes(n), dtype=torch.uint8, device="cuda")
        gb.gptb_policy_loss(d["z"], d["a"], d["w"], d["A"], d["old"], d["ref"], 0.2, 0.3, 0.1, dz, logp, stats, ws)
        return logp, stats

    want = call(None)
    grads = [torch.full((n, V), 7.0, dtype=dtype, device="cuda"),
             torch.full((n, V + 9), 7.0, dtype=dtype, device="cuda")[:, 3:V + 3],
             torch.full((n, V + 8), 7.0, dtype=dtype, device="cuda")[:, 7:V + 7], d["z"]]
    for dz in grads:  # (the last call overwrites the logits)
        for x, y in zip(call(dz), want):
            assert torch.equal(x, y)
    for dz in grads[1:]:
        assert torch.equal(dz, grads[0])
