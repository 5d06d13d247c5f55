"""GPU checks of escha_delta_rule against its recurrence in 64 bits."""
import numpy as np
import pytest

import mixer_refs as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _native():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_trellis_quantized_gb300 import native

    return native


def make(seed, lens, Hk, Hv, dk, dv, dtype, before=0, behind=0, like=0.0):
    """Inputs; `like`: how alike the keys of a head are (0: independent)."""
    rng = np.random.default_rng(seed)
    T = before + sum(lens) + behind
    k = rng.standard_normal((T, Hk, dk)) + like * rng.standard_normal((1, Hk, dk))
    rate = np.exp(rng.standard_normal(Hv) * 1.5 - 2.5)
    c = dict(q=torch.from_numpy(rng.standard_normal((T, Hk, dk))).to(DT[dtype]), k=torch.from_numpy(k).to(DT[dtype]),
             v=torch.from_numpy(rng.standard_normal((T, Hv, dv))).to(DT[dtype]),
             g=torch.from_numpy(-rate * np.log1p(np.exp(rng.standard_normal((T, Hv))))).float(),
             beta=torch.from_numpy(1 / (1 + np.exp(-rng.standard_normal((T, Hv))))).float(),
             state=torch.from_numpy(rng.standard_normal((len(lens), Hv, dk, dv)) * 0.2).float(),
             at=torch.from_numpy(before + np.cumsum([0] + list(lens))).int())
    return {k: v.cuda() for k, v in c.items()}


def f64(t):
    return t.double().cpu().numpy()


def run_and_check(native, c, dtype, scale=None, eps=1e-6, max_len=None, out=None):
    """The state's error against its size: each token adds roundings of sums of
    dk products held to 2^-22 of their terms or better, alike in size and of
    either sign, and what a token adds fades as the state does; a factor of 4
    for the tail: 2^-20 sqrt(dk) sqrt(tokens, 64 at most). An output adds half
    a step of its type."""
    scale = c["k"].shape[2] ** -0.5 if scale is None else scale
    want, want_state = ref.delta_rule(f64(c["q"]), f64(c["k"]), f64(c["v"]), f64(c["g"]), f64(c["beta"]),
                                      f64(c["state"]), c["at"].cpu().numpy(), scale, eps)
    state = c["state"].clone()
    marked = torch.full_like(c["v"], 77.0) if out is None else out
    got = native.delta_rule(c["q"], c["k"], c["v"], c["g"], c["beta"], state, c["at"], scale=scale, norm_eps=eps,
                            max_len=max_len, out=marked)
    torch.cuda.synchronize()
    T, (n, Hv, dk, dv) = c["q"].shape[0], c["state"].shape
    tol = 2.0 ** -20 * np.sqrt(dk * min(T + 1, 64))
    got, new = f64(got), f64(state)
    for s in range(n):
        for h in range(Hv):
            size = max(np.linalg.norm(want_state[s, h]), np.linalg.norm(f64(c["state"])[s, h]) * 1e-3)
            assert np.linalg.norm(new[s, h] - want_state[s, h]) <= tol * size, (s, h)
    none = np.isnan(want)
    assert np.all(got[none] == 77.0)
    size = np.max(np.abs(np.where(none, 0, want)), axis=(0, 2), keepdims=True)
    bound = ref.HALF[dtype] * np.abs(want) + tol * size + (2.0 ** -25 if dtype == "f16" else 0)
    assert np.all(np.abs(got - want)[~none] <= np.broadcast_to(bound, want.shape)[~none])
    return got, state


SHAPES = [
    ("f16", [1], 1, 1, 64, 32), ("bf16", [1, 0, 1, 1], 2, 4, 128, 128), ("f16", [3, 1, 0, 9], 2, 2, 128, 64),
    ("bf16", [64], 1, 3, 64, 96), ("f16", [63, 65, 0, 129, 1], 2, 4, 128, 128), ("bf16", [200], 1, 2, 128, 256),
    ("f16", [17, 130, 33], 3, 3, 64, 128), ("bf16", [0, 0, 5], 2, 2, 64, 160), ("f16", [300], 2, 4, 128, 32),
    ("bf16", [2, 127, 128, 0, 191, 192, 193], 1, 2, 128, 64),
    # many sequences; heads for one round of 64 columns a CTA, or two of 32
    ("f16", [70, 33, 0, 64, 31] * 8, 2, 4, 64, 64), ("bf16", [100, 1, 40] * 14, 1, 2, 128, 128),
    ("f16", [70, 33, 0, 64, 31] * 6, 2, 4, 64, 64), ("bf16", [100, 1, 40] * 12, 1, 2, 128, 128),
    ("bf16", [33 + i % 9 for i in range(70)], 1, 2, 64, 64), ("f16", [97] * 5, 3, 15, 128, 128),
]


@pytest.mark.parametrize("dtype,lens,Hk,Hv,dk,dv", SHAPES)
@pytest.mark.parametrize("max_len", [1, 1000])
def test_matches_the_recurrence(dtype, lens, Hk, Hv, dk, dv, max_len):
    native = _native()
    c = make(21, lens, Hk, Hv, dk, dv, dtype)
    out, state = run_and_check(native, c, dtype, max_len=max_len)
    again, state2 = run_and_check(native, c, dtype, max_len=max_len)
    assert np.array_equal(out, again) and torch.equal(state, state2)


@pytest.mark.parametrize("max_len", [1, 1000])
@pytest.mark.parametrize("dk", [64, 128])
def test_rows_of_no_sequence_and_bad_bounds(max_len, dk):
    native = _native()
    c = make(22, [70, 0, 20], 1, 2, dk, 64, "bf16", before=5, behind=30)
    run_and_check(native, c, "bf16", max_len=max_len)
    c["at"] = torch.tensor([-9, 60, 60, 1 << 30], dtype=torch.int32, device="cuda")  # clamped
    run_and_check(native, c, "bf16", max_len=max_len)


@pytest.mark.parametrize("max_len", [1, 1000])
def test_strong_and_weak_decay(max_len):
    """Decays that clear the state, none at all, and both next to each other."""
    native = _native()
    c = make(23, [150, 90], 2, 4, 128, 64, "f16")
    c["g"][:, 0] = 0.0
    c["g"][:, 1] = -30.0
    c["g"][40:200:37, 2] = -float("inf")
    c["g"][10:200:3, 3] = -90.0
    c["beta"][:, 0] = 1.0
    c["beta"][5:9, 1] = 0.0
    run_and_check(native, c, "f16", max_len=max_len)


@pytest.mark.parametrize("max_len", [1, 1000])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_keys_alike(max_len, dtype):
    """Keys of a head nearly the same: the corrections of a chunk hang on each
    other strongly (the coupling matrix is near its largest)."""
    native = _native()
    c = make(24, [140], 1, 2, 64, 64, dtype, like=6.0)
    run_and_check(native, c, dtype, max_len=max_len)


def check_columns(c, state):
    """Every column of the state to the bound of run_and_check of its own size:
    columns do not meet and scale with their values. (All tokens count, as a
    state that grows keeps what each was off.)"""
    _, want_state = ref.delta_rule(*(f64(c[x]) for x in ("q", "k", "v", "g", "beta", "state")), c["at"].cpu().numpy(),
                                      c["k"].shape[2] ** -0.5, 1e-6)
    T, dk = c["k"].shape[0], c["k"].shape[2]
    tol = 2.0 ** -20 * np.sqrt(dk * (T + 1))
    off, size = np.linalg.norm(f64(state) - want_state, axis=2), np.linalg.norm(want_state, axis=2)
    assert np.all(off <= tol * size)


@pytest.mark.parametrize("max_len", [1, 1000])
@pytest.mark.parametrize("dk", [64, 128])
def test_columns_of_very_different_sizes(max_len, dk):
    """Values of 2^-40 to 2^80 by column, over states of their size, and over
    others 2^-60 to 2^10 times that."""
    native = _native()
    c = make(31, [100, 45], 1, 2, dk, 64, "bf16")
    sizes = torch.exp2(torch.linspace(-40, 80, 64, device="cuda"))
    c["v"] = (c["v"].float() * sizes).bfloat16()
    c["state"][0] *= sizes
    c["state"][1] *= sizes * torch.exp2(torch.linspace(-60, 10, 64, device="cuda")[torch.randperm(64, device="cuda")])
    state = c["state"].clone()
    native.delta_rule(*(c[x] for x in ("q", "k", "v", "g", "beta")), state, c["at"], max_len=max_len)
    check_columns(c, state)


@pytest.mark.parametrize("max_len", [1, 1000])
def test_sizes_that_jump_and_states_that_grow(max_len):
    """Values that go up from chunk to chunk, 2^-50 to 2^100 at once too; decays
    of 0 in one head; positive g, which lets the state grow, in another."""
    native = _native()
    c = make(32, [32 * 6], 1, 3, 64, 32, "bf16")
    for i, e in enumerate((-50, -50, 90, 92, 100, 100)):
        c["v"][32 * i:32 * i + 32] = (c["v"][32 * i:32 * i + 32].float() * 2.0 ** e).bfloat16()
    c["state"] *= 2.0 ** -50
    c["g"][32 * 4:, 0] = -float("inf")
    c["g"][32 * 5, 1] = -float("inf")
    c["g"][:, 2] = 0.1
    state = c["state"].clone()
    native.delta_rule(*(c[x] for x in ("q", "k", "v", "g", "beta")), state, c["at"], max_len=max_len)
    check_columns(c, state)


@pytest.mark.parametrize("max_len", [1, 1000])
def test_a_nan_stays_in_its_column_and_sequence(max_len):
    native = _native()
    c = make(33, [50, 70, 40], 1, 2, 64, 64, "f16")
    args = [c[x] for x in ("q", "k", "v", "g", "beta")]
    clean = c["state"].clone()
    want = native.delta_rule(*args, clean, c["at"], max_len=max_len)
    c["v"][90, 1, 17] = float("nan")
    c["state"][0, 0, 5, 3] = float("inf")
    c["v"][130, 0, 40] = float("inf")
    state = c["state"].clone()
    got = native.delta_rule(*args, state, c["at"], max_len=max_len)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[50:120, 1, 17] = hit[:50, 0, 3] = hit[120:, 0, 40] = True
    assert torch.equal(got[~hit], want[~hit])
    assert not bool(got[90:120, 1, 17].isfinite().any()) and not bool(state[1, 1, :, 17].isfinite().all())
    same = torch.ones_like(state, dtype=torch.bool)
    same[1, 1, :, 17] = same[0, 0, :, 3] = same[2, 0, :, 40] = False
    assert torch.equal(state[same], clean[same])


@pytest.mark.parametrize("max_len", [1, 1000])
def test_keys_taken_as_they_are(max_len):
    native = _native()
    c = make(25, [100, 3], 2, 2, 64, 32, "bf16")
    c["k"] = (c["k"].float() / c["k"].float().norm(dim=-1, keepdim=True)).bfloat16()
    run_and_check(native, c, "bf16", scale=1.0, eps=None, max_len=max_len)
    run_and_check(native, c, "bf16", scale=0.3, eps=0.0, max_len=max_len)
    c["k"][7] = 0  # a key of nothing changes nothing
    run_and_check(native, c, "bf16", eps=1e-6, max_len=max_len)


def test_both_routes_over_a_long_prompt_then_steps():
    """A prompt in chunks, then token by token: the state carries over."""
    native = _native()
    c = make(26, [520], 2, 4, 128, 128, "bf16")
    whole = c["state"].clone()
    want = native.delta_rule(c["q"], c["k"], c["v"], c["g"], c["beta"], whole, c["at"], max_len=1)
    state = c["state"].clone()
    parts = []
    for a, b in ((0, 511), (511, 512), (512, 518), (518, 520)):
        at = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        parts.append(native.delta_rule(*(c[x][a:b].contiguous() for x in ("q", "k", "v", "g", "beta")), state, at))
    got = torch.cat(parts)
    # the two routes differ by what each may be off: see run_and_check
    tol = 2 * 2.0 ** -20 * np.sqrt(128 * 64)
    assert float((state - whole).norm() / whole.norm()) <= tol
    bound = 2 * ref.HALF["bf16"] * want.double().abs() + tol * want.double().abs().max()
    assert bool(((got.double() - want.double()).abs() <= bound).all())


@pytest.mark.parametrize("max_len", [1, 1000])
def test_streams_and_a_captured_call(max_len):
    native = _native()
    c = make(27, [80, 1, 0, 150], 2, 4, 64, 64, "f16")
    args = [c[x] for x in ("q", "k", "v", "g", "beta")]
    state = c["state"].clone()
    want = native.delta_rule(*args, state, c["at"], max_len=max_len)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    states = [c["state"].clone() for _ in side]
    torch.cuda.synchronize()
    outs = [native.delta_rule(*args, st, c["at"], max_len=max_len, stream=s) for s, st in zip(side, states)]
    torch.cuda.synchronize()
    for o, st in zip(outs, states):
        assert torch.equal(o, want) and torch.equal(st, state)
    st, out = c["state"].clone(), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        native.delta_rule(*args, st, c["at"], max_len=max_len, out=out)
    for _ in range(2):
        st.copy_(c["state"])
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(st, state)


def test_states_behind_32_bit_offsets():
    native = _native()
    n, Hv, dk, dv = 1030, 32, 128, 1024 // 8
    state = torch.zeros((n * 8 + 3, Hv, dk, dv), device="cuda")  # 4.3e9 values
    assert state.numel() > 1 << 32
    n = state.shape[0]
    c = make(28, [5, 70], 4, Hv, dk, dv, "f16")
    state[0], state[-1] = c["state"][0], c["state"][1]
    at = torch.full((n + 1,), 5, dtype=torch.int32, device="cuda")
    at[0], at[-1] = 0, 75
    for max_len in (1, 1000):
        want_state = c["state"].clone()
        args = [c[x] for x in ("q", "k", "v", "g", "beta")]
        want = native.delta_rule(*args, want_state, c["at"], max_len=max_len)
        state[0], state[-1] = c["state"][0], c["state"][1]
        got = native.delta_rule(*args, state, at, max_len=max_len)
        tol = 2 * 2.0 ** -20 * np.sqrt(128 * 64)
        for x, y in ((state[0], want_state[0]), (state[-1], want_state[1])):
            assert float((x - y).norm() / y.norm()) <= tol
        assert float((got.double() - want.double()).abs().max()) <= 2 * ref.HALF["f16"] * float(want.abs().max()) + tol
        assert not bool(state[1:-1].any())


def test_refusals():
    native = _native()
    c = make(29, [8], 2, 4, 64, 64, "f16")
    good = {x: c[x] for x in ("q", "k", "v", "g", "beta", "state", "at")}

    def bad(exc, **kw):
        with pytest.raises(exc):
            native.delta_rule(**{**good, **kw})

    bad(TypeError, q=c["q"].float())
    bad(TypeError, v=c["v"].bfloat16())
    bad(TypeError, state=c["state"].half())
    bad(TypeError, at=c["at"].long())
    bad(ValueError, k=c["k"][:4])
    bad(ValueError, g=c["g"].t())
    bad(ValueError, at=c["at"][:1])
    bad(ValueError, beta=c["beta"].cpu())
    bad(ValueError, norm_eps=-1.0)
    bad(native.EschaError, max_len=0)
    bad(native.EschaError, scale=float("inf"))
    d = make(30, [8], 2, 4, 64, 48, "f16")
    bad(native.EschaError, v=d["v"], state=d["state"])


@pytest.mark.parametrize("dtype,T,before,Hk,Hv,dk,dv", [("f16", 6500, 0, 2, 2, 64, 64), ("bf16", 9001, 41, 1, 2, 128, 96),
                                                        ("bf16", 6400, 31, 2, 4, 64, 32)])
def test_one_long_sequence(dtype, T, before, Hk, Hv, dk, dv):
    """Thousands of tokens, the first not on a chunk's boundary; calls one behind
    another on one workspace, and replayed, give the same bits."""
    native = _native()
    c = make(34, [T], Hk, Hv, dk, dv, dtype, before=before, behind=7)
    got, state = run_and_check(native, c, dtype, max_len=T)
    args = [c[x] for x in ("q", "k", "v", "g", "beta")]
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    st, out = c["state"].clone(), torch.full_like(c["v"], 77.0)
    # calls one behind another share a workspace
    for _ in range(3):
        st.copy_(c["state"])
        native.delta_rule(*args, st, c["at"], max_len=T, out=out, ws=ws)
        native.delta_rule(*args, c["state"].clone(), c["at"], max_len=T, ws=ws)
    assert torch.equal(st, state) and np.array_equal(f64(out), got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        native.delta_rule(*args, st, c["at"], max_len=T, out=out, ws=ws)
    for _ in range(2):
        st.copy_(c["state"])
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(st, state) and np.array_equal(f64(out), got)


@pytest.mark.parametrize("lens,chunks", [([1] * 255 + [2000], True), ([0] * 255 + [2000], True), ([1] * 63 + [500], True),
                                         ([700], True), ([12, 1], True), ([1] * 100, False), ([0, 1] * 40, False),
                                         ([3] * 50, False), ([9], False)])
def test_without_max_len_a_long_sequence_among_short_ones_goes_in_chunks(lens, chunks):
    """Only chunks need a workspace. The rows are right either way."""
    native = _native()
    c = make(35, lens, 1, 2, 64, 32, "f16")
    run_and_check(native, c, "f16")
    call = dict(state=c["state"].clone(), ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    args = {x: c[x] for x in ("q", "k", "v", "g", "beta", "at")}
    if chunks:
        with pytest.raises(native.EschaError, match="workspace"):
            native.delta_rule(**args, **call)
    else:
        native.delta_rule(**args, **call)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_workspace_of_the_types_own_size(dtype):
    native = _native()
    c = make(36, [100, 333, 1], 2, 4, 128, 64, dtype)
    need = native.lib().escha_delta_rule_workspace_dtype(native._dtype_tag(c["q"]), 3, 434, 2, 4, 128, 64, 333)
    whole = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    args = [c[x] for x in ("q", "k", "v", "g", "beta")]
    want, got = c["state"].clone(), c["state"].clone()
    out = native.delta_rule(*args, want, c["at"], max_len=333)
    run_and_check(native, c, dtype, max_len=333)
    assert torch.equal(native.delta_rule(*args, got, c["at"], max_len=333, ws=whole[:need]), out) and torch.equal(got, want)
    assert bool((whole[need:] == 0xA5).all())


@pytest.mark.parametrize("max_len", [1, 1000])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("what", ["q", "k", "g", "beta"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_nan_or_infinity_stays_in_its_heads_and_sequence(max_len, dtype, what, bad):
    """Of q and k: in the value heads of its key head, of g and beta in its own;
    nothing else changes by a bit, but outputs of its chunk ahead of it."""
    native = _native()
    c = make(37, [50, 70, 40], 2, 4, 64, 64, dtype)
    names = ("q", "k", "v", "g", "beta")
    clean = c["state"].clone()
    want = native.delta_rule(*(c[x] for x in names), clean, c["at"], max_len=max_len)
    t = 90  # of the second sequence, 40 tokens into it
    if what in ("q", "k"):
        c[what][t, 1, 9], heads = bad, slice(2, 4)
    else:
        c[what][t, 1], heads = bad, slice(1, 2)
    state = c["state"].clone()
    got = native.delta_rule(*(c[x] for x in names), state, c["at"], max_len=max_len)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[t - (31 if max_len > 1 else 0):120, heads] = True
    assert torch.equal(got[~hit], want[~hit])
    assert not bool(got[t, heads].isfinite().any())
    same = torch.ones_like(state, dtype=torch.bool)
    same[1, heads] = what == "q"
    assert torch.equal(state[same], clean[same])
    if what != "q":
        assert not bool(state[1, heads].isfinite().any())
        assert not bool(got[t:120, heads].isfinite().any())
