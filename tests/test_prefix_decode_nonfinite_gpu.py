"""NaN and infinities in what a decode step reads over a shared prompt: with a
window some samples of a prompt see a row that others do not, and only those that
see it are reached.  The others are held to the bounds of the oracle."""
import numpy as np
import pytest
import torch

from oracle import rollout as orl
from rollout_inputs import prefix_case
from test_packed_gpu import within

pytestmark = pytest.mark.gpu

H, HK = 4, 2


def call(gb, d, window):
    B = d["q"].shape[0]
    o, lse = torch.full_like(d["q"], 7.0), torch.full((B, H), 7.0, device="cuda")
    ws = torch.full((gb.gptb_prefix_decode_workspace_bytes(B, H, HK),), 255, dtype=torch.uint8, device="cuda")
    gb.gptb_prefix_decode_attention(d["q"], d["kp"], d["vp"], d["cp"], d["cg"], d["k"], d["v"], d["lens"], o, lse, H, HK, window, ws)
    assert gb.gptb_device_error() == 0
    return o.double().cpu().numpy(), lse.double().cpu().numpy()


@pytest.mark.parametrize("window", [-1, 60, 130, 500])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf"), 3e38])
@pytest.mark.parametrize("what", ["vp", "kp", "vp column", "q", "v"])
def test_only_the_samples_that_see_a_row_are_reached(cuda_lib, what, value, window):
    # two prompts whose samples are between 1 and 300 tokens in; the second begins inside a tile of the first
    plens, lens, T = [700, 333], [1, 300, 7, 40, 120, 2, 55, 200, 90, 3], 300
    d = prefix_case(plens, [6, 3], lens, T, H, HK, seed=30, extra=1)
    f = lambda x: np.nan_to_num(x.double().cpu().numpy())  # noqa: E731
    group = [0] * 6 + [1] * 3 + [2]
    plen, p0 = [700, 333, 0], [0, 700, 1033]
    spots = [(0, 640), (0, 699), (0, 570), (1, 290), (1, 332)]  # (prompt, row)
    for at in [[s] for s in spots] + [spots]:
        bad = {n: t.clone() for n, t in d.items()}
        clean = {n: t.clone() for n, t in d.items()}
        hit = np.zeros((len(lens), H, 128), bool)
        hit_lse = np.zeros((len(lens), H), bool)
        for g, j in at:
            for x, y in ((bad, value), (clean, 0.0)):
                if what == "q":
                    x["q"][g + 3] = y
                elif what == "v":
                    x["v"][g * 6 + 1, 0] = y
                elif what == "vp column":
                    x["vp"][p0[g] + j, 128 + 9] = y
                else:
                    x[what][p0[g] + j] = y
            for b, n in enumerate(lens):
                t = plen[group[b]] + n - 1
                if what == "q":
                    sees, heads, cols = b == g + 3, slice(None), slice(None)
                elif what == "v":
                    sees, heads, cols = b == g * 6 + 1, slice(None), slice(None)  # (its first own row, in or out of the window)
                else:
                    sees = group[b] == g and (t - j <= window or window < 0)
                    heads, cols = (slice(2, 4), slice(9, 10)) if what == "vp column" else (slice(None), slice(None))
                if sees:
                    hit[b, heads, cols] = True
                    if what in ("q", "kp"):
                        hit_lse[b, heads] = True
        o, lse = call(cuda_lib, bad, window)
        want, wlse, err = orl.prefix_decode(f(clean["q"]), f(clean["kp"]).reshape(-1, HK, 128), f(clean["vp"]).reshape(-1, HK, 128),
                                            clean["cp"].tolist(), clean["cg"].tolist(), f(clean["k"]), f(clean["v"]), lens, window)
        within(np.where(hit, want, o), want, err)
        empty = np.isneginf(wlse)
        assert np.array_equal(np.isneginf(np.where(hit_lse, wlse, lse)), empty)
        assert np.abs(np.where(hit_lse | empty, 0.0, lse) - np.where(hit_lse | empty, 0.0, wlse)).max() <= 1e-4
        if np.isnan(value) and what != "v":
            assert not np.isfinite(o[hit]).any()
        if np.isfinite(value) and what[0] == "v":
            assert np.isfinite(o).all()
