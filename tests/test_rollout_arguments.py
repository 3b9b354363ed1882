"""Arguments of the rollout operators that do not fit what the kernels read,
refused on the host without a GPU."""
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
