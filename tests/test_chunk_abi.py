"""Host-side checks (no GPU work) of the entry points of the append, the
attention of a chunk and the adjusted logits, and of the rotations' frequencies."""
import math
import os

import numpy as np
import pytest


def _lib():
    from bit_trellis_quantized_gb300 import native

    if not os.path.exists(native.LIB_PATH):
        from bit_trellis_quantized_gb300 import build

        build.build()
    return native, native.lib()


G = 0x10000


def test_rotary_append_validation():
    native, L = _lib()
    E = native
    base = dict(q=G, k=G, v=G, sdt=E.ESCHA_F32, ql=4096, kl=512, vl=512, turns=G, rot=64, inter=0, factor=1.0, pos=None, qo=2 * G,
                kp=3 * G, vp=4 * G, dt=E.ESCHA_F16, table=G, at=G, lens=G, n=2, T=9, Hq=16, Hkv=2, d=256, page=64, np=10, mp=4, s=None)

    def call(**kw):
        return L.escha_rotary_append(*{**base, **kw}.values())

    for code, kw in ((E.ESCHA_E_ARG, dict(k=None)), (E.ESCHA_E_ARG, dict(vp=None)), (E.ESCHA_E_ARG, dict(at=None)),
                     (E.ESCHA_E_ARG, dict(q=None)), (E.ESCHA_E_ARG, dict(qo=None)), (E.ESCHA_E_ARG, dict(dt=E.ESCHA_F32)),
                     (E.ESCHA_E_ARG, dict(sdt=E.ESCHA_BF16)), (E.ESCHA_E_ARG, dict(turns=None)), (E.ESCHA_E_ARG, dict(inter=2)),
                     (E.ESCHA_E_ARG, dict(factor=float("nan"))), (E.ESCHA_E_ARG, dict(T=0)), (E.ESCHA_E_ARG, dict(n=0)),
                     (E.ESCHA_E_ARG, dict(page=0)), (E.ESCHA_E_ARG, dict(vp=3 * G)), (E.ESCHA_E_ARG, dict(qo=G)),
                     (E.ESCHA_E_SHAPE, dict(rot=24)), (E.ESCHA_E_SHAPE, dict(rot=272)), (E.ESCHA_E_SHAPE, dict(rot=-16)),
                     (E.ESCHA_E_SHAPE, dict(ql=4095)), (E.ESCHA_E_SHAPE, dict(kl=508)), (E.ESCHA_E_SHAPE, dict(vl=0)),
                     (E.ESCHA_E_SHAPE, dict(d=96)), (E.ESCHA_E_SHAPE, dict(Hq=15)), (E.ESCHA_E_SHAPE, dict(n=65536)),
                     (E.ESCHA_E_SHAPE, dict(np=1 << 25)), (E.ESCHA_E_ALIGN, dict(kl=514)), (E.ESCHA_E_ALIGN, dict(k=G + 8)),
                     (E.ESCHA_E_ALIGN, dict(pos=G + 4)), (E.ESCHA_E_ALIGN, dict(turns=G + 8))):
        assert call(**kw) == code, kw
    # in place: of one type and dense
    assert call(qo=G, sdt=E.ESCHA_F16, ql=4104) == E.ESCHA_E_ARG
    assert b"rotary_append" in L.escha_last_error()


def test_chunk_attention_validation():
    native, L = _lib()
    E = native
    need = L.escha_chunk_attention_workspace(2, 100, 16, 2, 256, 1000)
    base = dict(q=G, k=G, v=2 * G, dt=E.ESCHA_F16, table=G, at=G, lens=G, n=2, T=100, Hq=16, Hkv=2, d=256, page=64, np=10, mp=16,
                ml=1000, scale=0.1, out=G, lse=None, ws=G, wsb=need, s=None)

    def call(**kw):
        return L.escha_chunk_attention(*{**base, **kw}.values())

    for code, kw in ((E.ESCHA_E_ARG, dict(q=None)), (E.ESCHA_E_ARG, dict(at=None)), (E.ESCHA_E_ARG, dict(out=None)),
                     (E.ESCHA_E_ARG, dict(dt=E.ESCHA_F32)), (E.ESCHA_E_ARG, dict(n=0)), (E.ESCHA_E_ARG, dict(T=0)),
                     (E.ESCHA_E_ARG, dict(ml=0)), (E.ESCHA_E_ARG, dict(page=0)), (E.ESCHA_E_ARG, dict(mp=0)),
                     (E.ESCHA_E_ARG, dict(scale=float("inf"))), (E.ESCHA_E_SHAPE, dict(d=96)), (E.ESCHA_E_SHAPE, dict(Hq=15)),
                     (E.ESCHA_E_SHAPE, dict(n=65536)), (E.ESCHA_E_SHAPE, dict(T=1 << 30)), (E.ESCHA_E_SHAPE, dict(np=1 << 25)),
                     (E.ESCHA_E_SHAPE, dict(ml=(1 << 30) + 1)), (E.ESCHA_E_ALIGN, dict(q=G + 8)), (E.ESCHA_E_ALIGN, dict(lse=G + 4))):
        assert call(**kw) == code, kw
    assert L.escha_chunk_attention_workspace(2, 0, 16, 2, 256, 1000) == 0
    need = L.escha_chunk_attention_workspace(1, 4, 16, 2, 256, 131072)
    if need:
        assert call(n=1, T=4, ml=131072, wsb=need, ws=None) == E.ESCHA_E_ARG
        assert call(n=1, T=4, ml=131072, wsb=need - 1) == E.ESCHA_E_WORKSPACE
        assert call(n=1, T=4, ml=131072, wsb=need, ws=G + 8) == E.ESCHA_E_ALIGN


def test_adjust_logits_validation():
    native, L = _lib()
    E = native
    base = dict(x=G, out=2 * G, dt=E.ESCHA_F32, M=3, V=1000, ld=1000, ol=1000, ids=G, at=G, n=9, prompt=None, rep=G, freq=None,
                pres=None, bi=G, b=G, ba=G, nb=4, allowed=G, nm=3, rows=None, s=None)

    def call(**kw):
        return L.escha_adjust_logits(*{**base, **kw}.values())

    for code, kw in ((E.ESCHA_E_ARG, dict(x=None)), (E.ESCHA_E_ARG, dict(out=None)), (E.ESCHA_E_ARG, dict(dt=4)),
                     (E.ESCHA_E_ARG, dict(M=0)), (E.ESCHA_E_ARG, dict(V=0)), (E.ESCHA_E_SHAPE, dict(ld=999)),
                     (E.ESCHA_E_SHAPE, dict(ol=999)), (E.ESCHA_E_ARG, dict(out=G, ol=1001)), (E.ESCHA_E_ARG, dict(n=-1)),
                     (E.ESCHA_E_ARG, dict(n=1 << 30)), (E.ESCHA_E_ARG, dict(at=None)), (E.ESCHA_E_ARG, dict(ids=None)),
                     (E.ESCHA_E_ARG, dict(b=None)), (E.ESCHA_E_ARG, dict(ba=None)), (E.ESCHA_E_ARG, dict(nb=-1)),
                     (E.ESCHA_E_ARG, dict(nm=2)), (E.ESCHA_E_ARG, dict(nm=0)), (E.ESCHA_E_ARG, dict(allowed=None)),
                     (E.ESCHA_E_ARG, dict(allowed=None, nm=0, rows=G)), (E.ESCHA_E_SHAPE, dict(V=(1 << 30) + 1)),
                     (E.ESCHA_E_SHAPE, dict(M=1 << 30, V=1 << 20, ld=1 << 20, ol=1 << 20, nm=1 << 30)),
                     (E.ESCHA_E_ALIGN, dict(x=G + 4)), (E.ESCHA_E_ALIGN, dict(rep=G + 4)), (E.ESCHA_E_ALIGN, dict(rows=G + 4))):
        assert call(**kw) == code, kw


def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    native, _ = _lib()
    x = torch.zeros((2, 4, 64), dtype=torch.float16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        native.rotary_append(x, x, x, x[None], x[None].clone(), i(1, 1), i(2), i(1))
    with pytest.raises(ValueError):
        native.chunk_attention(x, x[None], x[None].clone(), i(1, 1), i(2), i(1))
    with pytest.raises(ValueError):
        native.adjust_logits(torch.zeros((2, 9)))


def _angle(native_rotary, i, p):
    """The angle of position p in 2^64ths of a turn, as the kernel forms it, in radians within (-pi, pi]."""
    part = (p * int(native_rotary.turns[i])) % 2 ** 64
    return (part - 2 ** 64 if part >= 2 ** 63 else part) / 2 ** 63 * math.pi


@pytest.mark.parametrize("p", [0, 1, 131071, 2 ** 31 - 1, -5])
def test_turns_are_the_frequencies(p):
    native, _ = _lib()
    r = native.Rotary(64, base=1e6, device="cpu")
    assert np.allclose(r.frequencies, 1e6 ** (-np.arange(32) / 32), rtol=1e-15)
    for i in range(32):
        want, got = p * r.frequencies[i], _angle(r, i, p)
        # 2^-53 of the frequency and 2^-65 of a turn, p times each, and 64-bit cosines of angles of 2^31
        tol = 2.0 ** -51 * max(1.0, abs(want)) + abs(p) * 2.0 ** -62
        assert abs(math.cos(got) - math.cos(want)) <= tol and abs(math.sin(got) - math.sin(want)) <= tol
    assert r.factor == 1.0 and not r.interleaved


def test_scalings():
    native, _ = _lib()
    plain = native.Rotary(128, base=1e4, device="cpu").frequencies
    assert np.allclose(native.Rotary(128, scaling={"type": "linear", "factor": 8}, device="cpu").frequencies, plain / 8)
    ntk = native.Rotary(128, scaling={"type": "ntk", "factor": 8}, device="cpu").frequencies
    assert ntk[0] == plain[0] and abs(ntk[-1] * 8 / plain[-1] - 1) < 1e-12 and np.all(np.diff(ntk / plain) < 0)
    r = native.Rotary(128, scaling={"type": "yarn", "factor": 4, "original": 4096}, device="cpu")
    turns = 4096 * plain / (2 * math.pi)
    assert np.array_equal(r.frequencies[turns > 40], plain[turns > 40])
    assert np.allclose(r.frequencies[turns < 0.8], plain[turns < 0.8] / 4, rtol=1e-15)
    assert np.all(np.diff(r.frequencies) < 0) and abs(r.factor - (0.1 * math.log(4) + 1)) < 1e-15
    assert native.Rotary(128, scaling={"type": "yarn", "factor": 4, "original": 4096, "attention": 1.5}, device="cpu").factor == 1.5
    given = native.Rotary(32, frequencies=[0.5] * 16, device="cpu")
    assert set(given.turns.tolist()) == {round(0.5 / (2 * math.pi) * 2 ** 64)}
    # a frequency of more than a turn a position, and one below 0
    fast = native.Rotary(16, frequencies=[7.0, -1.0] + [0.0] * 6, device="cpu")
    assert abs(math.cos(_angle(fast, 0, 3)) - math.cos(21)) < 1e-14 and abs(math.sin(_angle(fast, 1, 2)) - math.sin(-2)) < 1e-14
    for kw in (dict(rot=24), dict(rot=0), dict(rot=32, base=1.0), dict(rot=32, scaling={"type": "else"}),
               dict(rot=32, scaling={"type": "linear", "factor": 0}), dict(rot=32, scaling={"type": "linear", "factor": 2, "more": 1}),
               dict(rot=32, frequencies=[1.0] * 15), dict(rot=32, frequencies=[math.nan] * 16),
               dict(rot=32, frequencies=[1.0] * 16, scaling={"type": "linear", "factor": 2})):
        with pytest.raises(ValueError):
            native.Rotary(**kw, device="cpu")


def test_chunk_order_is_0_or_1():
    native, L = _lib()
    assert L.escha_debug_set_chunk_order(2) == native.ESCHA_E_ARG and L.escha_debug_set_chunk_order(-1) == native.ESCHA_E_ARG
    assert L.escha_debug_set_chunk_order(1) == 0 and L.escha_debug_set_chunk_order(0) == 0


def test_chunk_wait_is_bounded():
    native, L = _lib()
    assert L.escha_debug_set_chunk_wait(-1) == native.ESCHA_E_ARG and L.escha_debug_set_chunk_wait((1 << 19) + 1) == native.ESCHA_E_ARG
    assert L.escha_debug_set_chunk_wait(0) == 0 and L.escha_debug_set_chunk_wait(1 << 19) == 0


def test_yarn_without_its_lengths_is_refused():
    native, _ = _lib()
    good = {"type": "yarn", "factor": 4, "original": 4096}
    native.Rotary(64, scaling=good, device="cpu")
    for bad in ({"type": "yarn", "factor": 4}, {**good, "original": 0}, {**good, "original": -1}, {**good, "beta_fast": 0},
                {**good, "beta_slow": -1.0}, {**good, "original": math.nan}):
        with pytest.raises(ValueError):
            native.Rotary(64, scaling=bad, device="cpu")
