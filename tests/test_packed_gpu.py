"""Packed attention (forward, backward) through the C ABI against the fp64
oracle.  Every element of o, dq, dk, dv is held to the bound that rounding P and
dS to bf16, o before D and the result can cause (oracle/rollout.py), with 2 % and
1e-5 of the largest value for the fp32 arithmetic in between; lse to 1e-4 (128
products of up to 11.4 in sum, each step of the sum off by at most 2^-24 of it:
at most 9e-5)."""
import numpy as np
import pytest
import torch

from oracle import rollout as orl
from rollout_inputs import heads, packed, qkv_views

pytestmark = pytest.mark.gpu

LENS = {
    "one token": [1],
    "short": [3, 1, 60, 2, 5],
    "a tile": [128],
    "a tile and one": [129],
    "tile edges": [127, 1, 128, 64, 65, 63],
    "empty ones": [0, 5, 0, 0, 300, 0],
    "ragged": [700, 13, 257, 40],
    "ends between the tiles of a pair": [640, 300, 212, 500],
    "many": [1 + i % 7 for i in range(150)],
}


def within(got, want, err):
    slack = 1.02 * err + 1e-5 * max(1e-30, float(np.abs(want).max(initial=0.0)))
    off = np.abs(got - want) - slack
    assert np.all(np.isfinite(got))
    assert off.size == 0 or off.max() <= 0, (float(np.abs(got - want).max()), float((np.abs(got - want) / slack).max()))


def run(gb, lens, H, Hk, window, backward=True, pad=0, seed=0):
    qkv, dout, cu = packed(lens, H, Hk, seed, pad)
    q, k, v = qkv_views(qkv, H, Hk)
    n = q.shape[0]
    o = torch.full((n, H * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, n), 7.0, device="cuda")
    gb.gptb_packed_attention(q, k, v, cu, o, lse, H, Hk, window)
    got = {"o": o, "lse": lse}
    if backward:
        dqkv = torch.full_like(qkv, 7.0)
        dq, dk, dv = qkv_views(dqkv, H, Hk)
        ws = torch.full((gb.gptb_packed_attention_workspace_bytes(n, H),), 255, dtype=torch.uint8, device="cuda")
        gb.gptb_packed_attention_backward(q, k, v, o, dout, lse, cu, dq, dk, dv, H, Hk, window, ws)
        got |= {"dq": dq, "dk": dk, "dv": dv}
    assert gb.gptb_device_error() == 0
    m = int(sum(lens))
    want = orl.packed_attention(heads(q[:m], H), heads(k[:m], Hk), heads(v[:m], Hk), cu.cpu().numpy(), window,
                                heads(dout[:m], H) if backward else None)
    return got, want, m


def check(got, want, m, H, Hk):
    for n in got:
        if n == "lse":
            assert np.abs(got[n].double().cpu().numpy()[:, :m] - want[n]).max(initial=0.0) <= 1e-4
            assert torch.all(got[n][:, m:] == 7.0)
        else:
            within(heads(got[n][:m], Hk if n in ("dk", "dv") else H), want[n], want["err"][n])
            assert torch.all(got[n][m:] == 7.0), n  # rows behind the last sequence are left as they were


@pytest.mark.parametrize("name", sorted(LENS))
@pytest.mark.parametrize("window", [-1, 0, 37])
def test_packed_attention(cuda_lib, name, window):
    got, want, m = run(cuda_lib, LENS[name], 4, 2, window)
    check(got, want, m, 4, 2)


@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 6), (10, 5), (8, 1)])
def test_packed_head_layouts(cuda_lib, H, Hk):
    got, want, m = run(cuda_lib, [200, 31, 90], H, Hk, -1)
    check(got, want, m, H, Hk)


@pytest.mark.parametrize("pad", [1, 40, 300])
@pytest.mark.parametrize("lens", [[5], [100, 20], [256], [130, 126]])
def test_rows_behind_the_last_sequence_hold_nan_and_stay(cuda_lib, lens, pad):
    got, want, m = run(cuda_lib, lens, 2, 1, -1, pad=pad)
    check(got, want, m, 2, 1)


@pytest.mark.parametrize("lens", [[700, 13, 257, 40, 1400], [60] * 40])
def test_packed_more_chains_than_multiprocessors(cuda_lib, lens):
    """19 tiles of 6 kv heads: each chain of backward steps by one CTA (a cluster shares each where there are fewer)."""
    got, want, m = run(cuda_lib, lens, 6, 6, -1)
    check(got, want, m, 6, 6)


@pytest.mark.parametrize("H,Hk,n", [(8, 8, 1), (8, 2, 500), (1, 1, 900), (16, 1, 130)])
def test_packed_chains_shared_by_clusters(cuda_lib, H, Hk, n):
    """Clusters of 8, 4 and 8 CTAs, some of them without a step; two calls give the same dk and dv bits."""
    a, want, m = run(cuda_lib, [n, 3], H, Hk, -1, seed=n)
    check(a, want, m, H, Hk)
    b, _, _ = run(cuda_lib, [n, 3], H, Hk, -1, seed=n)
    assert torch.equal(a["dk"], b["dk"]) and torch.equal(a["dv"], b["dv"])


def test_packed_long_sequence_with_window(cuda_lib):
    got, want, m = run(cuda_lib, [1500, 900], 2, 2, 300)
    check(got, want, m, 2, 2)


@pytest.mark.parametrize("seed", range(6))
def test_packed_random_lengths(cuda_lib, seed):
    r = np.random.default_rng(seed)
    lens = np.exp(r.uniform(0, np.log(900), r.integers(3, 12))).astype(int).tolist()
    got, want, m = run(cuda_lib, lens, 2, 1, [-1, -1, 200][seed % 3], seed=seed, pad=seed % 2 * 31)
    check(got, want, m, 2, 1)


def test_packed_nothing_to_do(cuda_lib):
    for lens, pad in (([], 0), ([], 9), ([0, 0], 9), ([0], 0)):
        got, want, m = run(cuda_lib, lens, 2, 1, -1, pad=pad)
        check(got, want, m, 2, 1)


def test_packed_rows_do_not_depend_on_their_neighbours(cuda_lib):
    """A sequence gives the same rows alone and among others at the same place in its tiles (forward, dk and dv)."""
    gb = cuda_lib
    qkv, dout, cu = packed([256, 200, 300], 2, 1, seed=5)
    alone = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    outs = []
    for x, d, c, at in ((qkv, dout, cu, 256), (qkv[256:456], dout[256:456], alone, 0)):
        q, k, v = qkv_views(x, 2, 1)
        o, lse = torch.empty(len(x), 256, dtype=torch.bfloat16, device="cuda"), torch.empty(2, len(x), device="cuda")
        gb.gptb_packed_attention(q, k, v, c, o, lse, 2, 1)
        dqkv = torch.empty(len(x), 512, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(gb.gptb_packed_attention_workspace_bytes(len(x), 2), dtype=torch.uint8, device="cuda")
        gb.gptb_packed_attention_backward(q, k, v, o, d, lse, c, *qkv_views(dqkv, 2, 1), 2, 1, -1, ws)
        outs.append((o[at:at + 200], lse[:, at:at + 200], dqkv[at:at + 200, 256:]))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_packed_forward_same_bits_every_time(cuda_lib):
    """Two CTAs on every multiprocessor and long rows: a product that overtook the one before it would show."""
    gb = cuda_lib
    for lens, H, Hk, window, times in (([6000, 37, 1500], 12, 12, -1, 40), ([300, 900, 45] * 8, 10, 5, 700, 60)):
        qkv, _, cu = packed(lens, H, Hk, seed=11)
        q, k, v = qkv_views(qkv, H, Hk)
        outs = [torch.empty(len(q), H * 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        lse = torch.empty(H, len(q), device="cuda")
        gb.gptb_packed_attention(q, k, v, cu, outs[0], lse, H, Hk, window)
        for _ in range(times):
            gb.gptb_packed_attention(q, k, v, cu, outs[1], lse, H, Hk, window)
            assert torch.equal(*outs)


def test_packed_captured_call_follows_its_lengths(cuda_lib):
    """A captured forward and backward, replayed with other lengths in the same offsets array, on a stream of its own."""
    gb = cuda_lib
    H, Hk, n = 4, 2, 500
    qkv, dout, _ = packed([n], H, Hk, seed=8)
    q, k, v = qkv_views(qkv, H, Hk)
    cu = torch.tensor([0, 100, 500, 500], dtype=torch.int32, device="cuda")
    o, lse = torch.empty(n, H * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H, n, device="cuda")
    dqkv = torch.empty_like(qkv)
    ws = torch.empty(gb.gptb_packed_attention_workspace_bytes(n, H), dtype=torch.uint8, device="cuda")

    def step():
        gb.gptb_packed_attention(q, k, v, cu, o, lse, H, Hk)
        gb.gptb_packed_attention_backward(q, k, v, o, dout, lse, cu, *qkv_views(dqkv, H, Hk), H, Hk, -1, ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for new in ([0, 100, 500, 500], [0, 0, 129, 500], [0, 7, 8, 300]):
        cu.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        m = new[-1]
        want = orl.packed_attention(heads(q[:m], H), heads(k[:m], Hk), heads(v[:m], Hk), new, -1, heads(dout[:m], H))
        got = dict(zip(("dq", "dk", "dv"), qkv_views(dqkv, H, Hk)), o=o)
        for name, t in got.items():
            within(heads(t[:m], Hk if name in ("dk", "dv") else H), want[name], want["err"][name])


def test_bad_offsets_are_reported(cuda_lib):
    gb = cuda_lib
    qkv, dout, _ = packed([300], 2, 1)
    q, k, v = qkv_views(qkv, 2, 1)
    ws = torch.empty(gb.gptb_packed_attention_workspace_bytes(300, 2), dtype=torch.uint8, device="cuda")
    for bad in ([0, 200, 100, 300], [0, 400], [3, 300], [0, -5, 300], [0, 2 ** 31 - 1, 300], [0, 300, -2 ** 31]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        o, lse = torch.empty(300, 256, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 300, device="cuda")
        gb.gptb_packed_attention(q, k, v, cu, o, lse, 2, 1)
        assert gb.gptb_device_error() == gb.ERR_BAD_INPUT, bad
        gb.gptb_packed_attention_backward(q, k, v, o, dout, lse, cu, *qkv_views(torch.empty_like(qkv), 2, 1), 2, 1, -1, ws)
        assert gb.gptb_device_error() == gb.ERR_BAD_INPUT, bad
