"""Arguments of the rollout operators that do not fit what the kernels read,
refused on the host without a GPU."""
import pytest
import torch

from test_rollout_refusals import _fwd, gb  # noqa: F401  (gb: the fixture)


def test_int_and_float_arrays_off_their_elements_boundary(gb):
    """Refused on the host: a kernel would read them at a misaligned address."""
    lib = gb.load()
    for at in (65, 66, 67):
        assert _fwd(lib, cu=at) == gb.ERR_INVALID_ARG and _fwd(lib, lse=(1 << 21) + at) == gb.ERR_INVALID_ARG
        bwd = dict(q=4096, ldq=256, k=8192, ldk=128, v=12288, ldv=128, o=1 << 20, ldo=256, dout=1 << 21, lddo=256, lse=1 << 22,
                   cu=64, dq=1 << 23, lddq=256, dk=1 << 24, lddk=128, dv=1 << 25, lddv=128, total=10, n_seq=2, H=2, Hkv=1,
                   window=-1, ws=1 << 26, bytes=1 << 30)
        for n in ("cu", "lse"):
            assert lib.gptb_packed_attention_backward(*(bwd | {n: at}).values(), None) == gb.ERR_INVALID_ARG, n
        dec = dict(q=4096, kp=8192, vp=12288, ld=256, cp=64, total=100, cg=128, n=2, k=1 << 20, v=1 << 21, lens=192, T=16,
                   o=1 << 22, lse=None, B=4, H=4, Hkv=2, window=-1, ws=1 << 23, bytes=1 << 30)
        for n in ("cp", "cg", "lens", "lse"):
            assert lib.gptb_prefix_decode_attention(*(dec | {n: at}).values(), None) == gb.ERR_INVALID_ARG, n
        pol = dict(z=4096, ld=100, dtype=gb.BF16, rows=10, V=100, a=64, w=128, A=192, old=256, ref=320, lo=0.2, hi=0.2,
                   beta=0.1, dz=1 << 20, ldd=100, logp=384, stats=448, ws=1 << 21, bytes=1 << 30)
        for n in ("a", "w", "A", "old", "ref", "logp", "stats"):
            assert lib.gptb_policy_loss(*(pol | {n: at}).values(), None) == gb.ERR_INVALID_ARG, n
        for a, lp in ((at, 128), (64, at)):
            assert lib.gptb_token_logprobs(4096, 100, gb.BF16, 10, 100, a, lp, None) == gb.ERR_INVALID_ARG


@pytest.fixture
def sent(gb, monkeypatch):  # noqa: F811
    """What the binding hands to the C entry points, on host tensors without memory."""
    got = []
    monkeypatch.setattr(gb, "_device", lambda name, t: t.device)
    monkeypatch.setattr(gb, "_enqueue", lambda dev, fn, args, stream, what: got.append((what, args)))
    return got


def test_numbers_beyond_32_bits(gb, sent):  # noqa: F811
    """A window of any size is one; sizes that a C int does not hold are refused, not cut to what it holds."""
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    e = lambda *s, dt=bf: torch.empty(*s, dtype=dt, device="meta")  # noqa: E731
    q, k, cu, lse, ws = e(10, 256), e(10, 128), e(3, dt=i32), e(2, 10, dt=f32), e(1 << 20, dt=torch.uint8)
    for w, c in ((5, 5), (-1, -1), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 63, 2 ** 31 - 1),
                 (-2 ** 32, -2)):
        gb.gptb_packed_attention(q, k, k, cu, q, lse, 2, 1, w)
        gb.gptb_packed_attention_backward(q, k, k, q, q, lse, cu, q, k, k, 2, 1, w, ws)
        gb.gptb_prefix_decode_attention(e(4, 2, 128), k, k, cu, cu, e(4, 16, 1, 128), e(4, 16, 1, 128), e(4, dt=i32), e(4, 2, 128),
                                        None, 2, 1, w, ws)
        fwd, bwd, dec = (a for _, a in sent[-3:])
        assert fwd[-1] == c and bwd[-3] == c and dec[-3] == c, w
    n, per_row = 2 ** 32 + 8, lambda m, dt=f32: e(m, dt=dt)  # noqa: E731
    for rows, V in ((n, 1), (1, n)):
        z, a, r = e(rows, V), per_row(rows, i32), per_row(rows)
        with pytest.raises(ValueError, match="2\\*\\*31"):
            gb.gptb_token_logprobs(z, a, r)
        with pytest.raises(ValueError, match="2\\*\\*31"):
            gb.gptb_policy_loss(z, a, r, r, r, r, 0.2, 0.2, 0.1, None, r, e(3, dt=f32), ws)
    with pytest.raises(ValueError, match="2\\*\\*31"):
        gb.gptb_packed_attention(e(n, 256), e(n, 128), e(n, 128), cu, e(n, 256), e(2, n, dt=f32), 2, 1)
