"""Calls of the rollout operators that the host refuses, without a GPU: the C
entry points by their codes, the binding by ValueError before the library is
reached."""
import ctypes

import pytest
import torch

BF = torch.bfloat16


@pytest.fixture(scope="module")
def gb():
    from gpt_transformer_block_b200 import build
    build.build()
    import gpt_transformer_block_b200 as gb
    gb.load()
    return gb


def _fwd(lib, **kw):
    a = dict(q=4096, ldq=256, k=8192, ldk=128, v=12288, ldv=128, cu=64, o=1 << 20, ldo=256, lse=1 << 21, total=10, n_seq=2,
             H=2, Hkv=1, window=-1)
    a |= kw
    return lib.gptb_packed_attention(*a.values(), None)


BAD_SHAPES = [dict(total=-1), dict(n_seq=-1), dict(H=0), dict(Hkv=0), dict(H=3, Hkv=2), dict(window=-2), dict(total=2 ** 30 + 1),
              dict(cu=None)]


def test_packed_attention_refusals(gb):
    lib = gb.load()
    for bad in BAD_SHAPES + [dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(lse=None), dict(q=4097),
                             dict(o=(1 << 20) + 8), dict(ldq=248), dict(ldq=260), dict(ldk=120), dict(ldo=128), dict(ldv=-128)]:
        assert _fwd(lib, **bad) == gb.ERR_INVALID_ARG, bad
    assert _fwd(lib, total=0) == gb.OK and _fwd(lib, n_seq=0) == gb.OK  # nothing to do


def test_packed_backward_refusals(gb):
    lib = gb.load()
    need = gb.gptb_packed_attention_workspace_bytes(10, 2)
    assert need >= 10 * 2 * 128 * 4 + 10 * 2 * 4
    assert gb.gptb_packed_attention_workspace_bytes(-1, 2) == 0 and gb.gptb_packed_attention_workspace_bytes(10, 0) == 0
    base = dict(q=4096, ldq=256, k=8192, ldk=128, v=12288, ldv=128, o=1 << 20, ldo=256, dout=1 << 21, lddo=256, lse=1 << 22,
                cu=64, dq=1 << 23, lddq=256, dk=1 << 24, lddk=128, dv=1 << 25, lddv=128, total=10, n_seq=2, H=2, Hkv=1,
                window=-1, ws=1 << 26, bytes=need)
    call = lambda **kw: lib.gptb_packed_attention_backward(*(base | kw).values(), None)  # noqa: E731
    for bad in BAD_SHAPES + [{n: None} for n in ("q", "k", "v", "o", "dout", "lse", "dq", "dk", "dv", "ws")] + [
            {n: 132} for n in ("lddq", "lddk", "lddv", "lddo")] + [dict(ws=8)]:
        assert call(**bad) == gb.ERR_INVALID_ARG, bad
    assert call(bytes=need - 1) == gb.ERR_WORKSPACE
    assert call(n_seq=0) == gb.OK


def test_prefix_decode_refusals(gb):
    lib = gb.load()
    need = gb.gptb_prefix_decode_workspace_bytes(4, 4, 2)
    assert need > 0
    for bad in ((-1, 4, 2), (4, 0, 2), (4, 4, 0), (4, 5, 2), (4, 129, 1)):
        assert gb.gptb_prefix_decode_workspace_bytes(*bad) == 0
    base = dict(q=4096, kp=8192, vp=12288, ld=256, cp=64, total=100, cg=128, n=2, k=1 << 20, v=1 << 21, lens=192, T=16,
                o=1 << 22, lse=None, B=4, H=4, Hkv=2, window=-1, ws=1 << 23, bytes=need)
    call = lambda **kw: lib.gptb_prefix_decode_attention(*(base | kw).values(), None)  # noqa: E731
    for bad in [{n: None} for n in ("q", "k", "v", "lens", "o", "kp", "vp", "cp", "cg", "ws")] + [
            {n: 4104} for n in ("q", "k", "v", "o", "kp", "ws")] + [
            dict(B=-1), dict(H=0), dict(Hkv=3), dict(T=0), dict(total=-1), dict(n=-1), dict(window=-2), dict(ld=128), dict(ld=260)]:
        assert call(**bad) == gb.ERR_INVALID_ARG, bad
    assert call(H=258, Hkv=2) == gb.ERR_UNSUPPORTED
    assert call(B=1 << 20, T=1 << 20) == gb.ERR_UNSUPPORTED
    assert call(bytes=need - 1) == gb.ERR_WORKSPACE
    assert call(B=0) == gb.OK


def test_policy_loss_refusals(gb):
    lib = gb.load()
    need = gb.gptb_policy_loss_workspace_bytes(10)
    assert need > 0 and gb.gptb_policy_loss_workspace_bytes(-1) == 0
    base = dict(z=4096, ld=100, dtype=gb.BF16, rows=10, V=100, a=64, w=128, A=192, old=256, ref=320, lo=0.2, hi=0.2, beta=0.1,
                dz=1 << 20, ldd=100, logp=384, stats=448, ws=1 << 21, bytes=need)
    call = lambda **kw: lib.gptb_policy_loss(*(base | kw).values(), None)  # noqa: E731
    nan = float("nan")
    for bad in [{n: None} for n in ("z", "a", "w", "A", "old", "ref", "logp", "stats", "ws")] + [
            dict(rows=-1), dict(V=0), dict(ld=99), dict(ldd=99), dict(z=4097), dict(dz=(1 << 20) + 1), dict(lo=-0.1), dict(lo=1.5),
            dict(hi=-0.1), dict(lo=nan), dict(hi=nan), dict(beta=nan), dict(beta=float("inf")), dict(ws=8),
            dict(dz=4096, ldd=104), dict(dtype=gb.F32, z=4098)]:
        assert call(**bad) == gb.ERR_INVALID_ARG, bad
    assert call(dtype=gb.FP8_E4M3) == gb.ERR_UNSUPPORTED
    assert call(bytes=need - 1) == gb.ERR_WORKSPACE
    lp = lambda **kw: lib.gptb_token_logprobs(*(dict(z=4096, ld=100, dtype=gb.BF16, rows=10, V=100, a=64, lp=128) | kw).values(), None)  # noqa: E731
    for bad in (dict(z=None), dict(a=None), dict(lp=None), dict(rows=-1), dict(V=0), dict(ld=99)):
        assert lp(**bad) == gb.ERR_INVALID_ARG, bad
    assert lp(dtype=9) == gb.ERR_UNSUPPORTED and lp(rows=0) == gb.OK


def test_the_binding_refuses_host_tensors_types_and_shapes(gb):
    q, k = torch.zeros(10, 256, dtype=BF), torch.zeros(10, 128, dtype=BF)
    cu, lse = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 10)
    with pytest.raises(ValueError, match="device memory"):
        gb.gptb_packed_attention(q, k, k, cu, q, lse, 2, 1)
    # the checks of one argument, on the device that the others are on
    cpu = q.device
    assert gb._rows("q", q, 256, BF, cpu, 10) == (q.data_ptr(), 256)
    assert gb._rows("q", q[:, 128:], 128, BF, cpu, 10) == (q.data_ptr() + 256, 256)
    assert gb._rows("q", q[3:4, 128:], 128, BF, cpu, 1)[1] >= 128
    for bad, why in ((q.float(), "float32"), (q[:, :200], "shape"), (q[:9], "shape"), (q[0], "shape"),
                     (torch.zeros(256, 10, dtype=BF).t(), "contiguous"), (q.to("meta"), "on meta")):
        with pytest.raises(ValueError, match=why):
            gb._rows("q", bad, 256, BF, cpu, 10)
    assert gb._flat("cu", cu, torch.int32, cpu, 2) == cu.data_ptr()
    for bad, why in ((cu.long(), "int64"), (cu[:1], "shape"), (torch.zeros(4, dtype=torch.int32)[::2], "shape"),
                     (cu.to("meta"), "on meta")):
        with pytest.raises(ValueError, match=why):
            gb._flat("cu", bad, torch.int32, cpu, 2)
    with pytest.raises(ValueError, match="workspace"):
        gb._workspace(torch.zeros(8, device="meta"), cpu)
    z = torch.zeros(4, 8, dtype=torch.float16)
    with pytest.raises(ValueError, match="float16"):
        gb.gptb_token_logprobs(z, cu, lse)
    with pytest.raises(ValueError, match="device memory"):
        gb.gptb_token_logprobs(z.float(), cu, lse)
