"""Host-side checks of the token mixers' and token log probabilities' entry
points (no GPU work): bad arguments come back as the documented status codes
before the device is touched."""
import ctypes
import os

import pytest


def _lib():
    from bit_trellis_quantized_gb300 import native

    if not os.path.exists(native.LIB_PATH):
        from bit_trellis_quantized_gb300 import build

        build.build()
    return native, native.lib()


G = 0x10000


def test_paged_attention_validation():
    native, L = _lib()
    need = L.escha_paged_attention_workspace(2, 16, 2, 256, 1000)
    base = dict(q=G, k=G, v=2 * G, dt=native.ESCHA_F16, table=G, lens=G, B=2, Hq=16, Hkv=2, d=256, page=64, n=10, mp=16,
                ml=1000, scale=0.1, kn=None, vn=None, out=G, lse=None, ws=G, wsb=need, s=None)

    def call(**kw):
        return L.escha_paged_attention(*{**base, **kw}.values())

    E = native
    for code, kw in ((E.ESCHA_E_ARG, dict(q=None)), (E.ESCHA_E_ARG, dict(table=None)), (E.ESCHA_E_ARG, dict(out=None)),
                     (E.ESCHA_E_ARG, dict(dt=E.ESCHA_F32)), (E.ESCHA_E_ARG, dict(B=0)), (E.ESCHA_E_ARG, dict(ml=0)),
                     (E.ESCHA_E_ARG, dict(page=0)), (E.ESCHA_E_ARG, dict(n=0)), (E.ESCHA_E_ARG, dict(mp=0)),
                     (E.ESCHA_E_ARG, dict(kn=G)), (E.ESCHA_E_ARG, dict(vn=G)), (E.ESCHA_E_ARG, dict(v=G)),
                     (E.ESCHA_E_ARG, dict(scale=float("inf"))), (E.ESCHA_E_ARG, dict(scale=float("nan"))),
                     (E.ESCHA_E_SHAPE, dict(d=96)), (E.ESCHA_E_SHAPE, dict(Hq=15)), (E.ESCHA_E_SHAPE, dict(Hq=130)),
                     (E.ESCHA_E_SHAPE, dict(B=65536)), (E.ESCHA_E_SHAPE, dict(Hq=2048, Hkv=2048)),
                     (E.ESCHA_E_SHAPE, dict(n=1 << 24, page=64)), (E.ESCHA_E_SHAPE, dict(ml=(1 << 30) + 1)),
                     (E.ESCHA_E_ALIGN, dict(q=G + 8)), (E.ESCHA_E_ALIGN, dict(lens=G + 4)),
                     (E.ESCHA_E_ALIGN, dict(lse=G + 4)), (E.ESCHA_E_ALIGN, dict(kn=G, vn=G + 2))):
        assert call(**kw) == code, kw
    need = L.escha_paged_attention_workspace(2, 16, 2, 256, 100000)
    assert need > 0
    assert call(ml=100000, wsb=need, ws=None) == E.ESCHA_E_ARG
    assert call(ml=100000, wsb=need - 1) == E.ESCHA_E_WORKSPACE
    assert call(ml=100000, wsb=need, ws=G + 8) == E.ESCHA_E_ALIGN
    assert b"paged_attention" in L.escha_last_error()
    assert L.escha_paged_attention_workspace(2, 16, 2, 100, 1000) == 0


def test_delta_rule_validation():
    native, L = _lib()
    need = L.escha_delta_rule_workspace(2, 300, 2, 4, 128, 64, 200)
    base = dict(q=G, k=G, v=G, dt=native.ESCHA_BF16, g=G, beta=G, state=G, at=G, n=2, T=300, Hk=2, Hv=4, dk=128, dv=64,
                ml=200, scale=0.1, eps=1e-6, out=G, ws=G, wsb=need, s=None)

    def call(**kw):
        return L.escha_delta_rule(*{**base, **kw}.values())

    E = native
    for code, kw in ((E.ESCHA_E_ARG, dict(k=None)), (E.ESCHA_E_ARG, dict(state=None)), (E.ESCHA_E_ARG, dict(at=None)),
                     (E.ESCHA_E_ARG, dict(dt=E.ESCHA_F32)), (E.ESCHA_E_ARG, dict(n=0)), (E.ESCHA_E_ARG, dict(T=0)),
                     (E.ESCHA_E_ARG, dict(Hk=0)), (E.ESCHA_E_ARG, dict(ml=0)), (E.ESCHA_E_ARG, dict(scale=float("nan"))),
                     (E.ESCHA_E_ARG, dict(eps=float("inf"))), (E.ESCHA_E_SHAPE, dict(Hv=3)),
                     (E.ESCHA_E_SHAPE, dict(dk=96)), (E.ESCHA_E_SHAPE, dict(dv=48)), (E.ESCHA_E_SHAPE, dict(dv=288)),
                     (E.ESCHA_E_SHAPE, dict(n=65536)), (E.ESCHA_E_SHAPE, dict(Hk=1, Hv=65536)),
                     (E.ESCHA_E_ALIGN, dict(v=G + 2)), (E.ESCHA_E_ALIGN, dict(g=G + 4)),
                     (E.ESCHA_E_ALIGN, dict(state=G + 8))):
        assert call(**kw) == code, kw
    if need:
        assert call(ws=None) == E.ESCHA_E_ARG
        assert call(wsb=need - 1) == E.ESCHA_E_WORKSPACE
    assert L.escha_delta_rule_workspace(0, 300, 2, 4, 128, 64, 200) == 0


def test_token_logprobs_validation():
    native, L = _lib()
    need = L.escha_token_logprobs_workspace(1, 500000)
    assert need > 0 and L.escha_token_logprobs_workspace(1, 100) == 0
    base = dict(x=G, dt=native.ESCHA_F32, M=1, V=500000, ld=500000, ids=G, n=1, top=5, lp=G, ent=G, lse=G, ti=G, tl=G,
                ws=G, wsb=need, s=None)

    def call(**kw):
        return L.escha_token_logprobs(*{**base, **kw}.values())

    E = native
    for code, kw in ((E.ESCHA_E_ARG, dict(x=None)), (E.ESCHA_E_ARG, dict(dt=4)), (E.ESCHA_E_ARG, dict(M=0)),
                     (E.ESCHA_E_ARG, dict(V=0)), (E.ESCHA_E_SHAPE, dict(V=(1 << 30) + 1)),
                     (E.ESCHA_E_SHAPE, dict(ld=499999)), (E.ESCHA_E_ARG, dict(n=-1)), (E.ESCHA_E_ARG, dict(n=1025)),
                     (E.ESCHA_E_ARG, dict(top=33)), (E.ESCHA_E_ARG, dict(top=-1)), (E.ESCHA_E_ARG, dict(V=4, top=5)),
                     (E.ESCHA_E_ARG, dict(ids=None)), (E.ESCHA_E_ARG, dict(lp=None)), (E.ESCHA_E_ARG, dict(ti=None)),
                     (E.ESCHA_E_ARG, dict(n=0, top=0, ent=None, lse=None)), (E.ESCHA_E_ALIGN, dict(x=G + 4)),
                     (E.ESCHA_E_ALIGN, dict(ids=G + 4)), (E.ESCHA_E_ARG, dict(ws=None)),
                     (E.ESCHA_E_WORKSPACE, dict(wsb=need - 1))):
        assert call(**kw) == code, kw


def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    native, _ = _lib()
    x = torch.zeros((2, 4, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        native.paged_attention(x, x[None], x[None].clone(), torch.zeros((2, 1), dtype=torch.int32),
                               torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        native.delta_rule(x, x, x, x[..., 0].float(), x[..., 0].float(), torch.zeros((1, 4, 64, 64)),
                          torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        native.token_logprobs(torch.zeros((2, 9)))


def test_wrappers_refuse_a_stream_of_another_device():
    torch = pytest.importorskip("torch")
    native, _ = _lib()

    class Stream:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="cuda:1"):
        native._On(0, Stream())


def test_wrappers_refuse_sizes_past_the_abis_integers():
    torch = pytest.importorskip("torch")
    native, _ = _lib()

    class Tensor:  # as much of one as comes before the check
        is_cuda = True

        def __init__(self, *shape):
            self.shape, self.dim = torch.Size(shape), lambda: len(shape)

    for M, V in ((2 ** 32 + 1, 1), (1, 2 ** 31)):
        with pytest.raises(ValueError, match="2\\^31"):
            native.token_logprobs(Tensor(M, V))


def test_delta_rule_workspace_by_type():
    """fp16 keys and queries are read where they are: no place for copies of them is asked for."""
    native, L = _lib()
    sizes = (3, 32000, 16, 32, 128, 128, 32000)
    either = L.escha_delta_rule_workspace(*sizes)
    assert L.escha_delta_rule_workspace_dtype(native.ESCHA_BF16, *sizes) == either
    need = L.escha_delta_rule_workspace_dtype(native.ESCHA_F16, *sizes)
    assert 0 < need == either - 2 * 32000 * 16 * 128 * 2
    assert L.escha_delta_rule(G, G, G, native.ESCHA_F16, G, G, G, G, *sizes, 0.1, 1e-6, G, G, need - 1, None) == native.ESCHA_E_WORKSPACE
    assert L.escha_delta_rule(G, G, G, native.ESCHA_BF16, G, G, G, G, *sizes, 0.1, 1e-6, G, G, need, None) == native.ESCHA_E_WORKSPACE
    assert L.escha_delta_rule_workspace_dtype(native.ESCHA_F32, *sizes) == 0
    assert L.escha_delta_rule_workspace_dtype(native.ESCHA_F16, 0, *sizes[1:]) == 0
