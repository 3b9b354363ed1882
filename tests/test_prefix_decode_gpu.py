"""The shared-prefix decode step through the C ABI against the fp64 oracle: each
element of o within the bound that rounding P and the result to bf16 can cause
(oracle/rollout.py; 2 % and 1e-5 of the largest value for the fp32 arithmetic),
lse within 1e-4.  Cache rows behind a sequence's length hold NaN."""
import numpy as np
import pytest
import torch

from oracle import rollout as orl
from rollout_inputs import heads, prefix_case
from test_packed_gpu import within

pytestmark = pytest.mark.gpu


def call(gb, d, H, Hk, window, ws=None):
    B = d["q"].shape[0]
    o = torch.full_like(d["q"], 7.0)
    lse = torch.full((B, H), 7.0, device="cuda")
    if ws is None:
        ws = torch.full((gb.gptb_prefix_decode_workspace_bytes(B, H, Hk),), 255, dtype=torch.uint8, device="cuda")
    gb.gptb_prefix_decode_attention(d["q"], d["kp"], d["vp"], d["cp"], d["cg"], d["k"], d["v"], d["lens"], o, lse, H, Hk,
                                    window, ws)
    return o, lse


def check(gb, d, H, Hk, window):
    o, lse = call(gb, d, H, Hk, window)
    assert gb.gptb_device_error() == 0
    f = lambda t: np.nan_to_num(t.double().cpu().numpy())  # noqa: E731
    ro, rl, err = orl.prefix_decode(f(d["q"]), f(d["kp"]).reshape(-1, Hk, 128), f(d["vp"]).reshape(-1, Hk, 128),
                                    d["cp"].tolist(), d["cg"].tolist(), f(d["k"]), f(d["v"]), d["lens"].tolist(), window)
    within(o.double().cpu().numpy(), ro, err)
    seen = np.isfinite(rl)
    lse = lse.double().cpu().numpy()
    assert np.array_equal(np.isfinite(lse), seen) and np.all(lse[~seen] == -np.inf)
    assert np.abs(lse[seen] - rl[seen]).max(initial=0.0) <= 1e-4
    return o


@pytest.mark.parametrize("window", [-1, 0, 30, 150, 10 ** 6])
@pytest.mark.parametrize("plens,sizes,lens,T", [
    ([1], [1], [1], 1),
    ([40], [3], [1, 5, 9], 9),
    ([300], [4], [1, 130, 128, 200], 200),
    ([128, 257, 1], [2, 5, 1], [1, 2, 60, 64, 3, 100, 40, 7], 100),
    ([0, 90], [2, 2], [3, 4, 5, 6], 8),
], ids=["one", "short", "one prompt", "three prompts", "an empty prompt"])
def test_prefix_decode(cuda_lib, plens, sizes, lens, T, window):
    check(cuda_lib, prefix_case(plens, sizes, lens, T, 4, 2), 4, 2, window)


@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 6), (10, 5), (13, 13), (9, 3), (8, 1)])
def test_prefix_decode_head_layouts(cuda_lib, H, Hk):
    lens = [1 + (37 * i) % 90 for i in range(11)]
    check(cuda_lib, prefix_case([333, 150], [7, 4], lens, 90, H, Hk, seed=1), H, Hk, -1)


@pytest.mark.parametrize("H,Hk,n", [(1, 1, 300), (3, 1, 100), (16, 2, 40), (128, 1, 3), (100, 1, 2)])
def test_more_samples_than_one_query_tile_holds(cuda_lib, H, Hk, n):
    lens = [1 + (13 * i) % 20 for i in range(n)]
    check(cuda_lib, prefix_case([200], [n], lens, 20, H, Hk, seed=2), H, Hk, -1)


def test_sequences_without_keys_without_group_and_with_bad_lengths(cuda_lib):
    gb = cuda_lib
    d = prefix_case([50, 0], [3, 2], [0, 4, 9, 0, 2, 0, 3, -1], 8, 4, 2, seed=3, extra=3)
    d["lens"][2] = 9  # longer than the cache
    o = check(gb, d, 4, 2, -1)
    for b in (2, 3, 5, 7):
        assert torch.all(o[b] == 0)
    check(gb, d, 4, 2, 3)


def test_no_prefix_is_the_plain_decode_step(cuda_lib):
    gb = cuda_lib
    d = prefix_case([], [], [5, 130, 256, 1], 256, 6, 3, seed=4, extra=4)
    d["kp"] = d["vp"] = torch.empty(0, 3 * 128, dtype=torch.bfloat16, device="cuda")
    check(gb, d, 6, 3, -1)


def test_prefix_rows_of_a_wider_array_and_of_other_groups(cuda_lib):
    """k and v as column ranges of a packed qkv array; another group's prompt holds NaN."""
    gb = cuda_lib
    H, Hk = 4, 2
    d = prefix_case([70, 30, 100], [1, 1, 2], [3, 4, 5, 6], 8, H, Hk, seed=5)
    wide = torch.full((200, (H + 2 * Hk) * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, H * 128:(H + Hk) * 128] = d["kp"]
    wide[:, (H + Hk) * 128:] = d["vp"]
    d["kp"], d["vp"] = wide[:, H * 128:(H + Hk) * 128], wide[:, (H + Hk) * 128:]
    whole, _ = call(gb, d, H, Hk, -1)
    check(gb, d, H, Hk, -1)
    wide[70:100] = float("nan")
    o, _ = call(gb, d, H, Hk, -1)
    keep = [0, 2, 3]
    assert torch.equal(o[keep], whole[keep]) and torch.all(torch.isnan(o[1]))


def test_prefix_decode_large_batch_same_bits_every_time(cuda_lib):
    gb = cuda_lib
    g = np.random.default_rng(6)
    lens = g.integers(1, 400, 90).tolist()
    d = prefix_case([900, 2000, 40], [30, 50, 10], lens, 400, 4, 2, seed=6)
    first = check(gb, d, 4, 2, -1)
    for _ in range(100):
        assert torch.equal(call(gb, d, 4, 2, -1)[0], first)


def test_prefix_decode_captured_step_follows_lengths(cuda_lib):
    """A captured step replayed while the sequences grow, with its workspace used by another graph in between."""
    gb = cuda_lib
    d = prefix_case([150, 60], [2, 3], [40] * 5, 40, 4, 2, seed=7)
    ws = torch.empty(gb.gptb_prefix_decode_workspace_bytes(5, 4, 2), dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    torch.cuda.synchronize()
    for w in (-1, 20):
        call(gb, d, 4, 2, w, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(gb, d, 4, 2, w, ws))
        graphs.append(graph)
    for lens in ([1, 2, 3, 4, 5], [40, 1, 0, 17, 33]):
        d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for w, (o, lse) in zip((-1, 20), outs):
            eo, el = call(gb, d, 4, 2, w)
            assert torch.equal(o, eo) and torch.equal(lse, el)


def test_bad_prefix_offsets_are_reported(cuda_lib):
    gb = cuda_lib
    for name, bad in (("cp", [0, 80, 40]), ("cp", [0, 50, 9999]), ("cp", [5, 50, 100]), ("cg", [0, 3, 1]),
                      ("cg", [0, 2, 99]), ("cg", [-7, 2, 4]), ("cg", [0, 2 ** 31 - 1, 4]), ("cp", [0, -2 ** 31, 100])):
        d = prefix_case([60, 40], [2, 2], [3, 4, 5, 6], 8, 4, 2, seed=8)
        d[name].copy_(torch.tensor(bad, dtype=torch.int32))
        call(gb, d, 4, 2, -1)
        assert gb.gptb_device_error() == gb.ERR_BAD_INPUT, (name, bad)
        assert gb.gptb_device_error() == 0
