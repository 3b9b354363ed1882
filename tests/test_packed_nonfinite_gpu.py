"""NaN and infinities inside the sequences of a packed batch: a row's reach those
that see it, and no others, in the same sequence or another, whatever tiles they
share.  Rows that no such value may reach are held to the bounds of
test_packed_gpu.py against the oracle of the same batch with zeros in its place."""
import numpy as np
import pytest
import torch

from oracle import rollout as orl
from rollout_inputs import heads, packed, qkv_views
from test_packed_gpu import within

pytestmark = pytest.mark.gpu

H, HK = 4, 2
BATCHES = {
    "short ones in a tile": [40, 3, 30, 5, 50],
    "over many tiles": [150, 700, 1, 333, 64],
    "ends on tiles": [128, 64, 256, 128],
}
SPOTS = [  # (array, sequence, place in it as a share, a kv head or all, a column or all, value)
    ("v", 1, 0.5, 1, 7, float("nan")), ("v", 1, 0.0, None, None, float("inf")), ("v", 2, 1.0, 0, None, float("-inf")),
    ("v", 0, 1.0, None, 100, float("nan")), ("v", 3, 0.3, None, None, 3e38),
    ("k", 1, 0.5, 0, 3, float("inf")), ("k", 0, 1.0, None, None, float("nan")), ("k", 3, 0.0, None, 127, float("-inf")),
    ("q", 1, 0.5, 1, 64, float("nan")), ("q", 2, 0.0, None, None, float("inf")),
    ("qkv", 1, None, None, None, float("nan")), ("qkv", 3, None, None, None, float("nan")),
]


def sees(cu, window):
    """[rows, rows]: row t sees row j."""
    seq = np.searchsorted(cu, np.arange(cu[-1]), side="right") - 1
    t, j = np.arange(cu[-1])[:, None], np.arange(cu[-1])[None]
    return (seq[:, None] == seq[None]) & (j <= t) & ((t - j <= window) | (window < 0))


def spoil(qkv, cu, spot):
    """qkv with the value in it, with zeros in its place, and {array: [(rows, kv head, columns)]} of where it is."""
    name, s, share, head, col, x = spot
    a, b = int(cu[s]), int(cu[s + 1])
    rows = np.arange(a, b) if share is None else np.array([a + round((b - 1 - a) * share)])
    cols = slice(None) if col is None else slice(col, col + 1)
    bad, clean = qkv.clone(), qkv.clone()
    for n in name:
        for kv in range(HK) if head is None else [head]:
            for t, y in ((bad, x), (clean, 0.0)):
                view = qkv_views(t, H, HK)["qkv".index(n)]
                view = view.view(len(t), -1, 128) if view.is_contiguous() else view.unflatten(1, (-1, 128))
                which = slice(kv * (H // HK), (kv + 1) * (H // HK)) if n == "q" else slice(kv, kv + 1)
                view[torch.tensor(rows).cuda()[:, None], torch.arange(view.shape[1])[which].cuda()[None], cols] = y
    return bad, clean, rows, (range(HK) if head is None else [head]), cols


def case(lens, window, spot, pad=0):
    qkv, dout, cu = packed(lens, H, HK, seed=3, pad=pad)
    cu_h = cu.cpu().numpy()
    bad, clean, rows, kvs, cols = spoil(qkv, cu_h, spot)
    vis = sees(cu_h, window)
    return bad, clean, dout, cu, cu_h, rows, kvs, cols, vis


@pytest.mark.parametrize("spot", SPOTS, ids=lambda s: f"{s[0]}{s[1]}-{s[2]}-{s[5]}")
@pytest.mark.parametrize("window", [-1, 0, 50])
@pytest.mark.parametrize("batch", sorted(BATCHES))
def test_forward(cuda_lib, batch, window, spot):
    gb = cuda_lib
    for pad in (0, 21):
        bad, clean, _, cu, cu_h, rows, kvs, cols, vis = case(BATCHES[batch], window, spot, pad)
        m, n = int(cu_h[-1]), len(bad)
        o, lse = torch.full((n, H * 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((H, n), 7.0, device="cuda")
        gb.gptb_packed_attention(*qkv_views(bad, H, HK)[:3], cu, o, lse, H, HK, window)
        assert gb.gptb_device_error() == 0
        q, k, v = (heads(t[:m], h) for t, h in zip(qkv_views(clean, H, HK), (H, HK, HK)))
        want = orl.packed_attention(q, k, v, cu_h, window)
        # the outputs that the value reaches: whole heads of the rows that see a key or are a query, columns of those
        # that see a value row
        hit, hit_lse = np.zeros((m, H, 128), bool), np.zeros((H, m), bool)
        for kv in kvs:
            for h in range(kv * (H // HK), (kv + 1) * (H // HK)):
                if "v" in spot[0]:
                    hit[vis[:, rows].any(1), h, cols] = True
                for name in set(spot[0]) - {"v"}:
                    reach = np.isin(np.arange(m), rows) if name == "q" else vis[:, rows].any(1)
                    hit[reach, h] = True
                    hit_lse[h, reach] = True
        got, got_lse = heads(o[:m], H), lse.double().cpu().numpy()[:, :m]
        if np.isfinite(spot[5]):  # (3e38: the sums of visible rows stay below the type's largest, and no bound holds for them)
            assert np.all(np.isfinite(got))
        elif spot[0] != "k":  # (an infinite score of -inf is a masked one)
            assert not np.isfinite(got[hit]).any() and not np.isfinite(got_lse[hit_lse]).any()
        within(np.where(hit, want["o"], got), want["o"], want["err"]["o"])
        assert np.abs(np.where(hit_lse, want["lse"], got_lse) - want["lse"]).max() <= 1e-4
        assert torch.all(o[m:] == 7.0) and torch.all(lse[:, m:] == 7.0)


def test_a_long_sequence_after_a_spoilt_one(cuda_lib):
    """None of its rows is reached, however many tiles they look back over: within the bounds, and where a query tile
    looks back over more than 2048 keys the same bits as after a sound one."""
    gb = cuda_lib
    qkv, _, cu = packed([37, 6000, 20], H, HK, seed=4)
    outs = []
    for x in (0.5, float("nan")):
        y = qkv.clone()
        y[:37] = x
        o, lse = torch.empty(len(y), H * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H, len(y), device="cuda")
        gb.gptb_packed_attention(*qkv_views(y, H, HK), cu, o, lse, H, HK)
        outs.append((o, lse))
    (o, lse), (o_nan, lse_nan) = outs
    assert torch.equal(lse[:, 37:], lse_nan[:, 37:]) and torch.equal(o[2048:], o_nan[2048:])
    q, k, v = (heads(t[37:2048], h) for t, h in zip(qkv_views(qkv, H, HK), (H, HK, HK)))
    want = orl.packed_attention(q, k, v, np.array([0, 2011]), -1)
    for got in (o, o_nan):
        within(heads(got[37:2048], H), want["o"], want["err"]["o"])


D_SPOTS = [("d", 1, 0.5, 1, 7, float("nan")), ("d", 2, 0.0, None, None, float("inf")),
           ("d", 3, 1.0, 0, 90, float("-inf")), ("d", 0, None, None, None, float("nan"))]
CASES = [(batch, window, spot) for batch in sorted(BATCHES) for window in (-1, 0, 50) for spot in SPOTS + D_SPOTS]
# (2 to 10 key tiles of 2 kv heads: clusters of 8 and 4 CTAs; 40 of them: no clusters)
BATCHES["no clusters"] = [150, 700, 1, 4200, 64]
CASES += [("no clusters", 50, spot) for spot in (SPOTS + D_SPOTS)[1::3]]


@pytest.mark.parametrize("batch,window,spot", CASES, ids=lambda s: s if not isinstance(s, tuple) else f"{s[0]}{s[1]}-{s[2]}-{s[5]}")
def test_backward(cuda_lib, batch, window, spot):
    """A query is spoilt that sees a spoilt row, or whose own q or dout is; its dq, and dk and dv of the keys that it
    sees, may be anything, every other gradient is that of the batch with zeros there."""
    gb = cuda_lib
    lens = BATCHES[batch]
    for pad in (0, 21):
        qkv, dout, cu = packed(lens, H, HK, seed=3, pad=pad)
        cu_h = cu.cpu().numpy()
        m, n = int(cu_h[-1]), len(qkv)
        name, s, share, head, col, x = spot
        d_bad, d_clean = dout.clone(), dout.clone()
        if name == "d":
            a, b = int(cu_h[s]), int(cu_h[s + 1])
            rows = np.arange(a, b) if share is None else np.array([a + round((b - 1 - a) * share)])
            kvs, bad, clean = range(HK) if head is None else [head], qkv, qkv
            cols = slice(None) if col is None else slice(col, col + 1)
            for kv in kvs:
                for t, y in ((d_bad, x), (d_clean, 0.0)):
                    for h in range(kv * (H // HK), (kv + 1) * (H // HK)):
                        t.view(n, H, 128)[torch.tensor(rows).cuda(), h, cols] = y
        else:
            bad, clean, rows, kvs, cols = spoil(qkv, cu_h, spot)
        vis = sees(cu_h, window)
        q, k, v = qkv_views(bad, H, HK)
        o, lse = torch.empty(n, H * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H, n, device="cuda")
        gb.gptb_packed_attention(q, k, v, cu, o, lse, H, HK, window)
        dqkv = torch.full_like(bad, 7.0)
        ws = torch.full((gb.gptb_packed_attention_workspace_bytes(n, H),), 255, dtype=torch.uint8, device="cuda")
        gb.gptb_packed_attention_backward(q, k, v, o, d_bad, lse, cu, *qkv_views(dqkv, H, HK), H, HK, window, ws)
        assert gb.gptb_device_error() == 0
        want = orl.packed_attention(*(heads(t[:m], h) for t, h in zip(qkv_views(clean, H, HK), (H, HK, HK))), cu_h, window,
                                    heads(d_clean[:m], H))
        bad_q = np.zeros((m, H), bool)
        for kv in kvs:
            own = name in ("q", "d")
            bad_q[rows if own else vis[:, rows].any(1), kv * (H // HK):(kv + 1) * (H // HK)] = True
        bad_kv = np.stack([vis[bad_q[:, kv * (H // HK):(kv + 1) * (H // HK)].any(1)].any(0) for kv in range(HK)], 1)
        for what, t, hit in zip(("dq", "dk", "dv"), qkv_views(dqkv, H, HK), (bad_q, bad_kv, bad_kv)):
            got = heads(t[:m], hit.shape[1])
            within(np.where(hit[:, :, None], want[what], got), want[what], want["err"][what])
            if np.isnan(x) and name in ("qkv", "q", "d"):
                assert not np.isfinite(got[hit]).any()
            assert torch.all(t[m:] == 7.0)


@pytest.mark.parametrize("rows", [[1500], [3000, 3100], list(range(1200, 4000, 300))])
@pytest.mark.parametrize("window", [-1, 1900])
def test_rows_far_behind_a_spoilt_one(cuda_lib, rows, window):
    """V rows of one kv head spoilt in the midst of long sequences: rows before them and of other sequences, also those
    that share tiles with them, are not reached, rows that see one are."""
    gb = cuda_lib
    lens = [1900, 2300, 40]
    qkv, _, cu = packed(lens, H, HK, seed=6)
    q, k, v = qkv_views(qkv, H, HK)
    cu_h = cu.cpu().numpy()
    want = orl.packed_attention(*(heads(t, h) for t, h in zip((q, k, v), (H, HK, HK))), cu_h, window)
    for r in rows:
        v[r, 128:] = float("nan")
    o, lse = torch.empty(len(qkv), H * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H, len(qkv), device="cuda")
    gb.gptb_packed_attention(q, k, v, cu, o, lse, H, HK, window)
    assert gb.gptb_device_error() == 0
    hit = np.zeros((len(qkv), H), bool)
    hit[:, 2:] = sees(cu_h, window)[:, rows].any(1)[:, None]
    got = heads(o, H)
    assert not np.isfinite(got[hit]).any()
    within(np.where(hit[:, :, None], want["o"], got), want["o"], want["err"]["o"])
    assert np.abs(lse.double().cpu().numpy() - want["lse"]).max() <= 1e-4
