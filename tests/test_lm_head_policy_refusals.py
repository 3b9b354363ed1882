"""model.lm_head_policy and lm_head_logprobs without a GPU: the calls that they
refuse, by ValueError before anything is launched, and that every launch of a
call is made with the tensors' device as the current one."""
import types

import pytest
import torch

from gpt_transformer_block_b200 import model

BF = torch.bfloat16
N, D, V = 10, 16, 24


def good():
    i32, f32 = (lambda n: torch.zeros(n, dtype=torch.int32)), (lambda *n: torch.zeros(*n))
    return dict(h=torch.zeros(N, D, dtype=BF), w_lm=torch.zeros(V, D, dtype=BF), actions=i32(N), weights=f32(N),
                advantages=f32(N), logp_old=f32(N), logp_ref=f32(N), clip_lo=0.2, clip_hi=0.2, beta=0.1,
                dh=torch.zeros(N, D, dtype=BF), dw_lm=f32(V, D))


@pytest.fixture
def launches(monkeypatch):
    """The launches of a call on host tensors, with the device that was current at each."""
    seen = []
    here = ["cuda:0"]

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, here[0] = here[0], str(self.dev)

        def __exit__(self, *_):
            here[0] = self.before

    cuda = types.SimpleNamespace(current_device=lambda: 0, device=Device)
    monkeypatch.setattr(model, "_device", lambda name, t: t.device, raising=False)
    monkeypatch.setattr(model.torch, "cuda", cuda)
    for name in ("gptb_gemm_bf16", "gptb_policy_loss", "gptb_token_logprobs"):
        monkeypatch.setattr(model, name, lambda *a, name=name, **k: seen.append((name, here[0])))
    monkeypatch.setattr(model, "gptb_policy_loss_workspace_bytes", lambda rows: 256)
    return seen


def test_every_launch_is_on_the_tensors_device(launches):
    model.lm_head_policy(**good(), rows_per_chunk=4)
    g = good()
    model.lm_head_logprobs(g["h"], g["w_lm"], g["actions"], rows_per_chunk=4)
    assert len(launches) == 3 * 4 + 3 * 2 and {dev for _, dev in launches} == {"cpu"}


def test_host_tensors_are_refused():
    g = good()
    with pytest.raises(ValueError, match="device memory"):
        model.lm_head_policy(**g)
    with pytest.raises(ValueError, match="device memory"):
        model.lm_head_logprobs(g["h"], g["w_lm"], g["actions"])


BAD = [dict(h=torch.zeros(N, D)), dict(h=torch.zeros(N * D, dtype=BF)), dict(h=torch.zeros(D, N, dtype=BF).t()),
       dict(h=torch.zeros(N, D + 4, dtype=BF)[:, 4:]), dict(h=torch.zeros(N, D - 4, dtype=BF)),
       dict(h=torch.zeros(N + 1, D, dtype=BF)),
       dict(w_lm=torch.zeros(V, D)), dict(w_lm=torch.zeros(V, D + 8, dtype=BF)), dict(w_lm=torch.zeros(V + 1, D, dtype=BF)),
       dict(w_lm=torch.zeros(D, V, dtype=BF).t()), dict(w_lm=torch.zeros(V, D, dtype=BF, device="meta")),
       dict(dh=torch.zeros(N, D)), dict(dh=torch.zeros(N - 1, D, dtype=BF)), dict(dh=torch.zeros(N, D + 4, dtype=BF)[:, 4:]),
       dict(dw_lm=torch.zeros(V, D, dtype=BF)), dict(dw_lm=torch.zeros(V - 8, D)), dict(dw_lm=torch.zeros(V, D + 2)[:, 2:]),
       dict(dw_lm=torch.zeros(D, V).t()),
       dict(actions=torch.zeros(N, dtype=torch.int64)), dict(actions=torch.zeros(N - 1, dtype=torch.int32)),
       dict(weights=torch.zeros(N, dtype=torch.float64)), dict(weights=torch.zeros(2 * N)[::2]), dict(advantages=torch.zeros(N, dtype=BF)),
       dict(logp_old=torch.zeros(N + 1)), dict(logp_ref=torch.zeros(N, device="meta")), dict(logp_ref=None),
       dict(clip_lo=-0.1), dict(clip_hi=float("nan")), dict(beta=float("inf")),
       dict(rows_per_chunk=0), dict(rows_per_chunk=-8)]


@pytest.mark.parametrize("bad", BAD, ids=lambda b: next(iter(b)))
def test_policy_refusals(launches, bad):
    with pytest.raises(ValueError):
        model.lm_head_policy(**(good() | bad))
    assert not launches
    if next(iter(bad)) in ("h", "w_lm", "actions", "rows_per_chunk"):
        g = {k: v for k, v in (good() | bad).items() if k in ("h", "w_lm", "rows_per_chunk")}
        with pytest.raises(ValueError):
            model.lm_head_logprobs(**g, tokens=(good() | bad)["actions"])
        assert not launches


def test_ranges_of_wider_arrays_are_taken(launches):
    """Row strides beyond the width, as the operators take them; no rows at all."""
    g = good()
    g |= dict(h=torch.zeros(N, D + 8, dtype=BF)[:, :D], w_lm=torch.zeros(V, D + 8, dtype=BF)[:, 8:],
              dh=torch.zeros(N, 2 * D, dtype=BF)[:, D:], dw_lm=torch.zeros(V, D + 4)[:, :D], logp_ref=None, beta=0.0)
    model.lm_head_policy(**g)
    assert len(launches) == 4
    none = {k: (v[:0] if torch.is_tensor(v) and v.shape[0] == N else v) for k, v in good().items()}
    stats, logp = model.lm_head_policy(**none)
    assert len(launches) == 4 and logp.numel() == 0 and not stats.any()
