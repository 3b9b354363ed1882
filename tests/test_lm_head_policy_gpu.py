"""model.lm_head_policy and lm_head_logprobs on layouts and rows that the run of
all operators together (test_rollout_gpu.py) does not have."""
import pytest
import torch

from gpt_transformer_block_b200 import model

pytestmark = pytest.mark.gpu

N, D, V = 300, 256, 640


def inputs(seed=0):
    g = torch.Generator().manual_seed(seed)
    x = {"h": torch.randn(N, D, generator=g).bfloat16(), "w_lm": (torch.randn(V, D, generator=g) * 0.1).bfloat16(),
         "actions": torch.randint(0, V, (N,), generator=g, dtype=torch.int32), "weights": torch.rand(N, generator=g) / N,
         "advantages": torch.randn(N, generator=g)}
    x = {n: t.cuda() for n, t in x.items()}
    x["logp_old"] = model.lm_head_logprobs(x["h"], x["w_lm"], x["actions"])
    x["logp_ref"] = x["logp_old"] - 0.1
    return x


def run(x, dh=None, dw=None, **kw):
    dh = torch.full((N, D), 7.0, dtype=torch.bfloat16, device="cuda") if dh is None else dh
    dw = torch.zeros(V, D, device="cuda") if dw is None else dw
    stats, logp = model.lm_head_policy(**x, clip_lo=0.2, clip_hi=0.2, beta=0.05, dh=dh, dw_lm=dw, **kw)
    return stats, logp, dh, dw


def same(got, want):
    """The same results, dw up to the order of its N fp32 sums."""
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a, b)
    assert (got[3] - want[3]).abs().max() <= N * 2.0 ** -23 * float(want[3].abs().max())


def test_column_ranges_of_wider_arrays(cuda_lib):
    x = inputs()
    want = run(x)
    wide = {n: torch.full((x[n].shape[0], 2 * D), float("nan"), dtype=torch.bfloat16, device="cuda") for n in ("h", "w_lm")}
    y = dict(x)
    for n, t in wide.items():
        t[:, D:] = x[n]
        y[n] = t[:, D:]
    dh, dw = torch.full((N, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.zeros(V, D + 4, device="cuda")
    same(run(y, dh[:, :D], dw[:, :D], rows_per_chunk=128), run(x, rows_per_chunk=128))
    assert torch.all(dh[:, D:] == 7.0) and torch.all(dw[:, D:] == 0)
    assert torch.equal(model.lm_head_logprobs(y["h"], y["w_lm"], x["actions"]), want[1])
    assert cuda_lib.gptb_device_error() == 0


def test_refused_before_any_launch(cuda_lib):
    x = inputs()
    for bad in (dict(h=x["h"].float()), dict(w_lm=x["w_lm"][:, :D - 8]), dict(logp_ref=x["logp_ref"].cpu())):
        dh, dw = torch.full((N, D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.zeros(V, D, device="cuda")
        with pytest.raises(ValueError):
            run(x | bad, dh, dw)
        assert torch.all(dh == 7.0) and torch.all(dw == 0)
    with pytest.raises(ValueError):
        run(x, dw=torch.zeros(V, D, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), 3e38])
def test_rows_without_weight_reach_no_gradient(cuda_lib, junk):
    """Rows of weight 0 (prompt tokens, padding behind the last sequence, which packed attention leaves as it was) may
    hold anything: dw and the other rows are those of a call with zeros there, dh is 0 in them."""
    x = inputs(seed=1)
    dead = torch.zeros(N, dtype=torch.bool, device="cuda")
    dead[[0, 7, 130, N - 1]] = True
    dead[200:260] = True
    x["weights"][dead] = 0
    clean, dirty = dict(x), dict(x)
    clean["h"], dirty["h"] = x["h"].clone(), x["h"].clone()
    clean["h"][dead], dirty["h"][dead] = 0, junk
    for n in ("advantages", "logp_old", "logp_ref"):
        dirty[n] = x[n].clone()
        dirty[n][dead] = float("nan")
    for chunk in (8192, 64):
        want, got = run(clean, rows_per_chunk=chunk), run(dirty, rows_per_chunk=chunk)
        assert bool(torch.isfinite(got[3]).all()) and torch.all(got[2][dead] == 0) and torch.all(got[1][dead] == 0)
        same(got, want)
    assert cuda_lib.gptb_device_error() == 0


def test_gradient_over_the_rows_themselves(cuda_lib):
    """dh in the place of h: the same results, dw's product reads h first."""
    x = inputs(seed=2)
    x["weights"][::5] = 0
    for chunk in (8192, 64):
        want = run(x, rows_per_chunk=chunk)
        y = dict(x, h=x["h"].clone())
        same(run(y, dh=y["h"], rows_per_chunk=chunk), want)
