"""The rollout operators together, as a policy update uses them: prompts read
whole by packed attention, answers sampled token by token over the shared
prompts, the answers' log-probabilities, the policy loss through the lm_head,
and the packed backward on prompts and answers.  Each stage is held to the fp64
oracle of what the stages before gave it."""
import numpy as np
import pytest
import torch

from gpt_transformer_block_b200 import model
from oracle import rollout as orl
from rollout_inputs import heads, normed, offsets
from test_packed_gpu import within

pytestmark = pytest.mark.gpu

H, HK, D = 4, 2, 512
W = (H + 2 * HK) * 128


def project(x, w):
    """A stand-in for the block's QKV projection with its QK normalisation: bf16 rows [N, (H + 2 HK) * 128]."""
    y = (x.float() @ w.float().t()).view(-1, H + 2 * HK, 128)
    n = H + HK
    y[:, :n] = y[:, :n] * torch.rsqrt(y[:, :n].square().mean(-1, keepdim=True) + 1e-6)
    return y.view(-1, W).bfloat16()


@pytest.mark.parametrize("window", [-1, 70])
def test_prefill_decode_and_policy_update(cuda_lib, window):
    gb = cuda_lib
    g = torch.Generator().manual_seed(3)
    plens, sizes, steps = [37, 130, 64], [3, 1, 4], 5
    V, B = 1000, sum(sizes)
    wte = torch.randn(V, D, generator=g).bfloat16().cuda()
    w_qkv = (torch.randn(W, D, generator=g) * 0.05).bfloat16().cuda()
    w_lm = (torch.randn(V, D, generator=g) * 0.2).bfloat16().cuda()
    prompts = torch.randint(0, V, (sum(plens),), generator=g).cuda()
    cp, cg = torch.tensor(offsets(plens)).cuda(), torch.tensor(offsets(sizes)).cuda()

    # the prompts, whole
    qkv = project(wte[prompts], w_qkv)
    cols = lambda t: (t[:, :H * 128], t[:, H * 128:(H + HK) * 128], t[:, (H + HK) * 128:])  # noqa: E731
    q, k, v = cols(qkv)
    o, lse = torch.empty(len(q), H * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H, len(q), device="cuda")
    gb.gptb_packed_attention(q, k, v, cp, o, lse, H, HK, window)
    want = orl.packed_attention(heads(q, H), heads(k, HK), heads(v, HK), cp.cpu().numpy(), window)
    within(heads(o, H), want["o"], want["err"]["o"])

    # the samples, token by token: k and v of the prompts stay where the projection put them
    T = 8
    kc = torch.full((B, T, HK, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    group = np.repeat(np.arange(len(sizes)), sizes)
    h_last = o[torch.tensor(np.array(offsets(plens))[1:][group] - 1).cuda()]  # the state that samples the first token
    ws = torch.empty(gb.gptb_prefix_decode_workspace_bytes(B, H, HK), dtype=torch.uint8, device="cuda")
    tokens, states, logps = [], [], []
    for t in range(steps):
        z = h_last.float() @ w_lm.float().t()
        pick = torch.multinomial(torch.softmax(z, -1).cpu(), 1, generator=g)[:, 0].to(torch.int32).cuda()
        logps.append(model.lm_head_logprobs(h_last.contiguous(), w_lm, pick))
        tokens.append(pick)
        states.append(h_last)
        nq, nk, nv = cols(project(wte[pick.long()], w_qkv))
        kc[:, t], vc[:, t] = nk.view(B, HK, 128), nv.view(B, HK, 128)
        lens = torch.full((B,), t + 1, dtype=torch.int32, device="cuda")
        od, ld = torch.empty(B, H, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(B, H, device="cuda")
        gb.gptb_prefix_decode_attention(nq.contiguous(), k, v, cp, cg, kc, vc, lens, od, ld, H, HK, window, ws)
        f = lambda x: np.nan_to_num(x.double().cpu().numpy())  # noqa: E731
        ro, rl, err = orl.prefix_decode(f(nq).reshape(B, H, 128), heads(k, HK), heads(v, HK), cp.tolist(), cg.tolist(), f(kc),
                                        f(vc), lens.tolist(), window)
        within(od.double().cpu().numpy(), ro, err)
        h_last = od.view(B, H * 128)

    # prompt and answer of every sample as one packed sequence: the decode steps' outputs are its last rows
    answers = torch.stack(tokens, 1).long()  # [B, steps]
    seqs = [torch.cat([prompts[cp[i]:cp[i + 1]], a]) for i, a in zip(group, answers)]
    cu = torch.tensor(offsets([len(s) for s in seqs])).cuda()
    x = project(wte[torch.cat(seqs)], w_qkv)
    q, k, v = cols(x)
    n = len(x)
    o, lse = torch.empty(n, H * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(H, n, device="cuda")
    gb.gptb_packed_attention(q, k, v, cu, o, lse, H, HK, window)
    rows = torch.cat([torch.arange(int(e) - steps, int(e)) for e in cu[1:]]).cuda()
    want = orl.packed_attention(heads(q, H), heads(k, HK), heads(v, HK), cu.cpu().numpy(), window)
    # (two results within err of the exact one are within 2 err of each other)
    last = rows.view(B, steps)[:, -1]
    got, other = o[last].double().cpu().numpy().reshape(B, H, 128), h_last.double().cpu().numpy().reshape(B, H, 128)
    at = last.cpu().numpy()
    assert np.all(np.abs(got - other) <= 2.04 * want["err"]["o"][at] + 2e-5 * np.abs(want["o"]).max())

    # the policy update on the sampled tokens: the row before a token predicts it, prompt rows carry no weight
    acts, wts = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, device="cuda")
    acts[rows - 1], wts[rows - 1] = answers.reshape(-1).int(), 1.0 / (B * steps)
    adv, old, ref = (torch.zeros(n, device="cuda") for _ in range(3))
    adv[rows - 1] = torch.randn(B, generator=g).repeat_interleave(steps).cuda()
    old[rows - 1] = torch.stack(logps, 1).reshape(-1)
    ref[rows - 1] = old[rows - 1] + 0.3 * torch.randn(B * steps, generator=g).cuda()
    dh, dw = torch.empty(n, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(V, D, device="cuda")
    stats, logp = model.lm_head_policy(o, w_lm, acts, wts, adv, old, ref, 0.2, 0.2, 0.05, dh, dw, rows_per_chunk=300)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    z = f((f_ := o.float() @ w_lm.float().t()).bfloat16())
    loss, kl, clipped, lp, dz, coef, gap = orl.policy_loss(z, acts.cpu().numpy(), f(wts), f(adv), f(old), f(ref), 0.2, 0.2, 0.05)
    # a logit that lies next to a rounding border of bf16 may round either way: 2^-7 of the largest, through the softmax
    off = 2.0 ** -7 * np.abs(f(f_)).max()
    live = f(wts) > 0
    assert np.abs(f(logp) - lp)[live].max() <= 2 * off and torch.all(logp[torch.tensor(~live)] == 0)
    mag = (f(wts) * (np.exp(lp - f(old)) * np.abs(f(adv)) + 0.05 * (1 + np.exp(f(ref) - lp))))[live].sum()
    assert gap[live].min() > 0 and abs(float(stats[0]) - loss) <= 4 * off * mag + 1e-6
    bound = lambda a, b: 4 * off * np.abs(a) @ np.abs(b) + 2.0 ** -7 * np.abs(a) @ np.abs(b)  # noqa: E731
    big = np.abs(dz) + np.abs(coef)[:, None] * off
    assert np.all(np.abs(f(dh) - dz @ f(w_lm)) <= bound(big, f(w_lm)) + 1e-9)
    assert np.all(np.abs(f(dw) - dz.T @ f(o)) <= bound(big.T, f(o)) + 1e-9)
    assert np.all(f(dh)[~live] == 0)

    # and its gradient back through the attention of all sequences
    dqkv = torch.empty_like(x)
    bws = torch.empty(gb.gptb_packed_attention_workspace_bytes(n, H), dtype=torch.uint8, device="cuda")
    gb.gptb_packed_attention_backward(q, k, v, o, dh, lse, cu, *cols(dqkv), H, HK, window, bws)
    want = orl.packed_attention(heads(q, H), heads(k, HK), heads(v, HK), cu.cpu().numpy(), window, heads(dh, H))
    for name, t, m in zip(("dq", "dk", "dv"), cols(dqkv), (H, HK, HK)):
        within(heads(t, m), want[name], want["err"][name])
    assert gb.gptb_device_error() == 0


def test_lm_head_policy_chunks_add_up(cuda_lib):
    """One chunk and several give the same loss, log-probabilities and gradients (dw up to the order of its sums)."""
    g = torch.Generator().manual_seed(5)
    N, V = 700, 640
    h = torch.randn(N, D, generator=g).bfloat16().cuda()
    w = (torch.randn(V, D, generator=g) * 0.1).bfloat16().cuda()
    a = torch.randint(0, V, (N,), generator=g, dtype=torch.int32).cuda()
    old = model.lm_head_logprobs(h, w, a, rows_per_chunk=256)
    assert torch.equal(old, model.lm_head_logprobs(h, w, a))
    wt, adv = torch.full((N,), 1.0 / N, device="cuda"), torch.randn(N, generator=g).cuda()
    out = []
    for chunk in (8192, 256):
        dh, dw = torch.empty_like(h), torch.zeros(V, D, device="cuda")
        out.append((*model.lm_head_policy(h, w, a, wt, adv, old, None, 0.2, 0.2, 0.0, dh, dw, rows_per_chunk=chunk), dh, dw))
    one, many = out
    assert torch.equal(one[1], many[1]) and torch.equal(one[2], many[2])
    assert abs(float(one[0][0]) + float((wt * adv).sum())) <= 1e-5  # on-policy: -sum w A
    assert (one[0] - many[0]).abs().max() <= 1e-6
    # three partial sums in place of one: fp32 sums of N products each
    assert (one[3] - many[3]).abs().max() <= N * 2.0 ** -23 * float(one[3].abs().max())


def test_an_operator_on_a_stream_of_its_own(cuda_lib):
    """stream=: the call waits for that stream's work, not the current one's."""
    gb = cuda_lib
    g = torch.Generator().manual_seed(6)
    x = normed(g, 200, 4, 128).view(200, 512).cuda()
    cu = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    o, lse = torch.empty(200, 256, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 200, device="cuda")
    want = torch.empty_like(o)
    gb.gptb_packed_attention(x[:, :256], x[:, 256:384], x[:, 384:], cu, want, lse, 2, 1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    late = torch.zeros_like(x)
    with torch.cuda.stream(s):
        late.copy_(x)
    gb.gptb_packed_attention(late[:, :256], late[:, 256:384], late[:, 384:], cu, o, lse, 2, 1, stream=s)
    s.synchronize()
    assert torch.equal(o, want)


def test_two_calls_at_once(cuda_lib):
    """Calls of each operator on two streams at the same time, with outputs and workspaces of their own."""
    gb = cuda_lib
    g = torch.Generator().manual_seed(7)
    n, V = 900, 4001
    x = normed(g, n, H + 2 * HK, 128).view(n, W).cuda()
    dout = torch.randn(n, H * 128, generator=g).bfloat16().cuda()
    cu = torch.tensor([0, 300, 310, 900], dtype=torch.int32, device="cuda")
    cg = torch.tensor([0, 2, 5, 6], dtype=torch.int32, device="cuda")
    kc, vc = (normed(g, 6, 40, HK, 128).cuda() for _ in range(2))
    lens = torch.tensor([1, 40, 7, 0, 33, 12], dtype=torch.int32, device="cuda")
    z = torch.randn(n, V, generator=g).cuda()
    a = torch.randint(0, V, (n,), generator=g, dtype=torch.int32).cuda()
    row = [torch.randn(n, generator=g).cuda() for _ in range(4)]
    q, k, v = x[:, :H * 128], x[:, H * 128:(H + HK) * 128], x[:, (H + HK) * 128:]

    def buffers():
        e = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        bf, u8 = torch.bfloat16, torch.uint8
        return {"o": e(n, H * 128, dt=bf), "lse": e(H, n), "dk": e(n, HK * 128, dt=bf), "dv": e(n, HK * 128, dt=bf),
                "dq": e(n, H * 128, dt=bf), "ws": e(gb.gptb_packed_attention_workspace_bytes(n, H), dt=u8),
                "od": e(6, H, 128, dt=bf), "ld": e(6, H), "wd": e(gb.gptb_prefix_decode_workspace_bytes(6, H, HK), dt=u8),
                "dz": e(n, V), "logp": e(n), "stats": e(3), "wp": e(gb.gptb_policy_loss_workspace_bytes(n), dt=u8)}

    def enqueue(b, s):
        gb.gptb_packed_attention(q, k, v, cu, b["o"], b["lse"], H, HK, -1, s)
        gb.gptb_packed_attention_backward(q, k, v, b["o"], dout, b["lse"], cu, b["dq"], b["dk"], b["dv"], H, HK, -1, b["ws"], s)
        gb.gptb_prefix_decode_attention(b["o"][:6], k, v, cu, cg, kc, vc, lens, b["od"], b["ld"], H, HK, -1, b["wd"], s)
        gb.gptb_policy_loss(z, a, row[0], row[1], row[2], row[3], 0.2, 0.2, 0.1, b["dz"], b["logp"], b["stats"], b["wp"], s)

    want = buffers()
    enqueue(want, None)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [buffers() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for b, s in zip(got, streams):
            enqueue(b, s)
    torch.cuda.synchronize()
    for b in got:
        for name in ("o", "lse", "dk", "dv", "od", "ld", "dz", "logp", "stats"):
            assert torch.equal(b[name], want[name]), name
        # dq: fp32 sums in another order may round to the neighbouring bf16
        assert (b["dq"].float() - want["dq"].float()).abs().max() <= 2.0 ** -7 * want["dq"].float().abs().max()
    assert gb.gptb_device_error() == 0
