"""GPU checks of escha_paged_attention against its formula in 64 bits."""
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


def make(seed, lens, Hq, Hkv, d, page, dtype, spare=3, poison=True):
    """A cache whose unused slots hold NaN and infinities, and a step's inputs."""
    rng = np.random.default_rng(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    n_pages, width = sum(need) + spare, max(max(need), 1)
    order = rng.permutation(n_pages)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    c = dict(q=rng.standard_normal((len(lens), Hq, d)) * 2, k_new=rng.standard_normal((len(lens), Hkv, d)),
             v_new=rng.standard_normal((len(lens), Hkv, d)), k=rng.standard_normal((n_pages, Hkv, page, d)),
             v=rng.standard_normal((n_pages, Hkv, page, d)))
    if poison:
        live = np.zeros((n_pages, page), bool)
        for b, n in enumerate(lens):
            for j in range(max(n, 0)):
                live[table[b, j // page], j % page] = True
        c["k"][~live.repeat(Hkv, 0).reshape(n_pages, Hkv, page)] = np.nan
        c["v"][~live.repeat(Hkv, 0).reshape(n_pages, Hkv, page)] = np.inf
    c = {k: torch.from_numpy(v).to(DT[dtype]).cuda() for k, v in c.items()}
    c["table"], c["lens"] = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    return c


def f64(t):
    return t.double().cpu().numpy()


def check(c, out, lse, scale, dtype, cap=None):
    """Bound of a value: half a step of the type, and through the scores, each
    a sum of d products in f32 (at most (d + 4) 2^-24 sum |q||k| off, before
    and behind the maximum), through the weights (split in two 16-bit parts:
    2^-15 of each together with the exponential's error) and the sums."""
    q = f64(c["q"])
    want, want_lse, mass, reach = ref.attention(q, f64(c["k"]), f64(c["v"]), c["table"].cpu().numpy(),
                                                c["lens"].cpu().numpy(), scale, cap)
    x_err = (q.shape[2] + 4) * 2.0 ** -24 * reach
    tol = ref.HALF[dtype] * np.abs(want) + (2 * x_err[..., None] + 2.0 ** -15) * mass
    if dtype == "f16":
        tol = tol + 2.0 ** -25  # half the smallest step near 0
    assert np.all(np.abs(f64(out) - want) <= tol)
    got = f64(lse)
    none = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got), none)
    tol = x_err + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(none, 0, want_lse))
    assert np.all(np.abs(got[~none] - want_lse[~none]) <= tol[~none])


SHAPES = [
    ("f16", [1], 2, 2, 64, 16), ("bf16", [1, 0, 2], 4, 1, 128, 1), ("f16", [15, 16, 17], 8, 1, 256, 16),
    ("bf16", [63, 64, 65, 0, 129], 16, 2, 256, 64), ("f16", [300, 5, 0, 0, 77], 5, 1, 128, 17),
    ("bf16", [1000], 16, 2, 256, 64), ("f16", [700, 699], 3, 3, 64, 48), ("bf16", [40, 513], 22, 2, 64, 32),
    ("f16", [257, 31], 64, 1, 64, 128), ("bf16", [33, 2000, 1], 24, 1, 128, 256), ("f16", [4097], 6, 2, 128, 1024),
    ("bf16", [500] * 9 + [0] * 3, 16, 4, 64, 16),
    # units cut over all CTAs
    ("bf16", [9000, 0, 5], 24, 1, 128, 32), ("f16", [5000, 130], 64, 2, 64, 48), ("f16", [4500, 4500, 1], 10, 2, 256, 64),
    # clusters of 4, 2 and 1, longest first and not
    ("bf16", [3000, 17, 2900] + [64 * (i % 5) + i for i in range(57)], 8, 4, 128, 64),
    ("bf16", [(i * 37) % 300 for i in range(59)] + [1500], 12, 4, 128, 32),
    ("f16", [700] + [i * 11 for i in range(59)], 4, 4, 128, 16),
    ("f16", [900] + [(i * 53) % 200 for i in range(99)], 16, 8, 64, 64), ("bf16", [(i * 29) % 131 for i in range(70)], 16, 16, 64, 16),
    ("f16", [40, 1300] * 16, 32, 4, 256, 64),
]


@pytest.mark.parametrize("dtype,lens,Hq,Hkv,d,page", SHAPES)
@pytest.mark.parametrize("new", [False, True])
def test_matches_the_formula(dtype, lens, Hq, Hkv, d, page, new):
    native = _native()
    c = make(11, lens, Hq, Hkv, d, page, dtype)
    kw, before = {}, (c["k"].clone(), c["v"].clone())
    if new:
        kw = dict(k_new=c["k_new"], v_new=c["v_new"])
        for b, n in enumerate(lens):
            if n:  # what the cache holds at the new position must not matter
                pg = int(c["table"][b, (n - 1) // page])
                c["k"][pg, :, (n - 1) % page] = float("nan")
                c["v"][pg, :, (n - 1) % page] = float("nan")
    out, lse = native.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], scale=0.11, **kw)
    torch.cuda.synchronize()
    if new:
        for b, n in enumerate(lens):
            if n:
                pg = int(c["table"][b, (n - 1) // page])
                before[0][pg, :, (n - 1) % page] = c["k_new"][b]
                before[1][pg, :, (n - 1) % page] = c["v_new"][b]
    # the pools hold what they held, and the new token
    for got, want in zip((c["k"], c["v"]), before):
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    check(c, out, lse, 0.11, dtype)
    again, lse2 = native.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], scale=0.11, **kw)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,d", [("f16", 64), ("bf16", 128), ("f16", 256)])
def test_dropped_and_bad_pages_hold_no_keys(dtype, d):
    native = _native()
    c = make(12, [100, 64, 40, 16], 4, 2, d, 16, dtype)
    t = c["table"]
    t[0, 2], t[0, 5] = -1, 1 << 30  # a dropped page, an entry past the pool
    t[1, :] = -5  # nothing left
    t[2, 2] = c["k"].shape[0]  # the page of the new position is none
    before = c["k"].clone()
    out, lse = native.paged_attention(c["q"], c["k"], c["v"], t, c["lens"], k_new=c["k_new"], v_new=c["v_new"])
    torch.cuda.synchronize()
    check(c, out, lse, d ** -0.5, dtype)
    assert torch.all(out[1] == 0) and torch.all(torch.isneginf(lse[1]))
    before[int(t[0, 6]), :, 3] = c["k_new"][0]
    before[int(t[3, 0]), :, 15] = c["k_new"][3]
    assert torch.equal(c["k"].view(torch.int16), before.view(torch.int16))


def test_lengths_past_the_table_or_the_bound_are_cut():
    native = _native()
    c = make(13, [48, 48, 48], 4, 2, 64, 16, "f16", poison=False)
    c["lens"] = torch.tensor([1 << 30, -7, 40], dtype=torch.int32, device="cuda")
    out, lse = native.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"])
    check(c, out, lse, 64 ** -0.5, "f16")
    out, lse = native.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], max_len=33)
    check(c, out, lse, 64 ** -0.5, "f16", cap=33)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_far_apart_scores(dtype):
    """One key far above the rest, far below them, and all alike."""
    native = _native()
    c = make(14, [200, 200, 200], 2, 1, 128, 32, dtype, poison=False)
    c["q"][:] = 0
    c["q"][0, :, 0], c["q"][1, :, 0] = 200.0, -200.0
    c["k"][:, :, :, 0] = 0.5
    c["k"][int(c["table"][0, 4]), 0, 7, 0] = 8.0
    c["k"][int(c["table"][1, 2]), 0, 1, 0] = 8.0
    out, lse = native.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], scale=1.0)
    check(c, out, lse, 1.0, dtype)
    assert torch.equal(out[0, 0], c["v"][int(c["table"][0, 4]), 0, 7])


@pytest.mark.parametrize("dtype,d", [("f16", 64), ("bf16", 128), ("f16", 256)])
def test_many_keys_of_next_to_no_weight(dtype, d):
    """One key of value 0 that takes almost all weight; 40000 others, each at
    2^-25.4 of it, make up the output: their weights are as good as any."""
    native = _native()
    c = make(17, [40000], 4, 2, d, 64, dtype, poison=False)
    c["q"][:] = 0
    c["q"][:, :, 1] = 1.1  # (of both types: 1.1 rounded)
    c["k"][:, :, :, 1] = 0
    pg = int(c["table"][0, 100])
    c["k"][pg, :, 3] = 0
    c["k"][pg, :, 3, 1] = 16.0
    c["v"][:] = c["v"].abs()
    c["v"][pg, :, 3] = 0
    out, lse = native.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], scale=1.0)
    assert float(out.abs().min()) > 5e-4
    check(c, out, lse, 1.0, dtype)


def test_one_long_sequence_among_short_ones():
    native = _native()
    c = make(15, [20000, 3, 0, 777], 16, 2, 256, 64, "bf16")
    out, lse = native.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], k_new=c["k_new"], v_new=c["v_new"])
    check(c, out, lse, 1 / 16, "bf16")


def test_pages_behind_32_bit_offsets():
    native = _native()
    Hkv, page, d = 8, 64, 256
    n_pages = (1 << 32) // (Hkv * page * d) + 9  # the last pages start past 2^32 values
    k = torch.empty((n_pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    used = [n_pages - 1, 0, n_pages - 5, n_pages // 2 + 1]
    gen = torch.Generator(device="cuda").manual_seed(3)
    for p in used:
        k[p] = torch.randn(k.shape[1:], generator=gen, device="cuda").bfloat16()
        v[p] = torch.randn(k.shape[1:], generator=gen, device="cuda").bfloat16()
    small = dict(q=torch.randn((1, 16, d), generator=gen, device="cuda").bfloat16(), k=k[used].clone(), v=v[used].clone(),
                 table=torch.arange(4, dtype=torch.int32, device="cuda")[None],
                 lens=torch.tensor([250], dtype=torch.int32, device="cuda"))
    new = torch.randn((2, 1, Hkv, d), generator=gen, device="cuda").bfloat16()
    out, lse = native.paged_attention(small["q"], k, v, torch.tensor([used], dtype=torch.int32, device="cuda"),
                                      small["lens"], k_new=new[0], v_new=new[1])
    small["k"][3, :, 250 - 193] = new[0, 0]
    small["v"][3, :, 250 - 193] = new[1, 0]
    check(small, out, lse, 1 / 16, "bf16")
    assert torch.equal(k[used], small["k"]) and torch.equal(v[used], small["v"])


def test_streams_and_a_captured_step():
    native = _native()
    c = make(16, [90, 400, 0, 33], 8, 2, 128, 16, "f16", poison=False)
    args = (c["q"], c["k"], c["v"], c["table"], c["lens"])
    want, want_lse = native.paged_attention(*args)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    got = [native.paged_attention(*args, stream=s) for s in side for _ in range(4)]
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want) and torch.equal(l, want_lse)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        native.paged_attention(*args, out=out, lse=lse)
    c["lens"].copy_(torch.tensor([1, 399, 20, 0], dtype=torch.int32))  # lengths are read by the replay
    c["table"][2, :2] = c["table"][1, :2]
    graph.replay()
    torch.cuda.synchronize()
    check(c, out, lse, 128 ** -0.5, "f16")


def test_refusals():
    native = _native()
    c = make(17, [40], 4, 2, 64, 16, "f16")
    good = dict(q=c["q"], k_pool=c["k"], v_pool=c["v"], table=c["table"], lens=c["lens"])

    def bad(exc, **kw):
        with pytest.raises(exc):
            native.paged_attention(**{**good, **kw})

    bad(TypeError, q=c["q"].float())
    bad(TypeError, k_pool=c["k"].bfloat16())
    bad(TypeError, lens=c["lens"].long())
    bad(ValueError, lens=c["lens"].repeat(2))
    bad(ValueError, q=c["q"].transpose(1, 2))
    bad(ValueError, table=c["table"].cpu())
    bad(ValueError, k_new=c["k_new"])
    bad(ValueError, k_new=c["k_new"], v_new=c["v_new"][:, :1])
    bad(native.EschaError, v_pool=c["k"])
    bad(native.EschaError, scale=float("nan"))
    bad(native.EschaError, q=c["q"][:, :3].contiguous())
    bad(native.EschaError, max_len=0)
    bad(ValueError, ws=torch.empty(16, device="cuda"))
    wide = torch.zeros((1, 200), dtype=torch.int32, device="cuda")  # long enough to need a workspace
    one = make(19, [40], 4, 2, 64, 32, "f16")
    with pytest.raises(native.EschaError, match="workspace"):
        native.paged_attention(one["q"], one["k"], one["v"], wide, one["lens"], ws=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype,lens,cap,Hq,Hkv,d,page", [
    ("f16", [48, 33, 1 << 30, 32, 0], 33, 4, 2, 64, 16), ("bf16", [400, 200, 201] * 30, 200, 16, 4, 128, 32),
    ("f16", [700, 699, 650], 699, 16, 2, 256, 64), ("bf16", [5000, 4501, 4500], 4500, 24, 1, 128, 32),
    ("f16", [9000], 8999, 16, 1, 64, 48)])
def test_no_new_token_behind_the_bound(dtype, lens, cap, Hq, Hkv, d, page):
    """A length past max_len, or past what its row of the table holds, has no
    place for the new token: it is not stored over a key that is there, and not
    attended."""
    native = _native()
    for by_table in (False, True):
        c = make(18, [min(n, 10000) for n in lens], Hq, Hkv, d, page, dtype, poison=False)
        c["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        bound = cap // page * page if by_table else cap
        kw = {} if by_table else dict(max_len=cap)
        if by_table:
            c["table"] = c["table"][:, :cap // page].contiguous()
        want = c["k"].clone(), c["v"].clone()
        for b, n in enumerate(lens):
            if 0 < n <= bound:
                pg = int(c["table"][b, (n - 1) // page])
                want[0][pg, :, (n - 1) % page], want[1][pg, :, (n - 1) % page] = c["k_new"][b], c["v_new"][b]
        out, lse = native.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], k_new=c["k_new"], v_new=c["v_new"], **kw)
        torch.cuda.synchronize()
        assert torch.equal(c["k"], want[0]) and torch.equal(c["v"], want[1])
        check(c, out, lse, d ** -0.5, dtype, cap=bound)


@pytest.mark.parametrize("dtype,lens,Hq,Hkv,d", [("f16", [300, 200, 77], 16, 4, 64), ("bf16", [5000, 4700, 9], 6, 2, 128),
                                                 ("f16", [700, 650, 31], 24, 2, 256)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_nan_or_infinity_stays_with_those_who_read_it(dtype, lens, Hq, Hkv, d, bad):
    native = _native()
    group = Hq // Hkv
    for what in ("q", "k", "v"):
        c = make(20, lens, Hq, Hkv, d, 16, dtype)
        args = [c[x] for x in ("q", "k", "v", "table", "lens")]
        want, want_lse = native.paged_attention(*args)
        hit = torch.zeros_like(want, dtype=torch.bool)
        if what == "q":
            c["q"][1, 3, 5], hit[1, 3] = bad, True
        else:
            c[what][int(c["table"][1, 7]), 1, 3, 5] = bad  # position 115 of the second sequence, key head 1
            hit[1, group:2 * group, slice(None) if what == "k" else 5] = True
        out, lse = native.paged_attention(*args)
        assert torch.equal(out[~hit], want[~hit])
        rows = hit.any(-1) if what != "v" else torch.zeros_like(lse, dtype=torch.bool)
        assert torch.equal(lse[~rows], want_lse[~rows])
        if bad != bad:
            assert bool(out[hit].isnan().all()) and bool(lse[rows].isnan().all())
        elif what == "v":
            assert not bool(out[hit].isfinite().any())
