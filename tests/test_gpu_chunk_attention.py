"""GPU checks of escha_chunk_attention against its formula in 64 bits."""
import time

import numpy as np
import pytest

import chunk_refs as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _native():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_trellis_quantized_gb300 import native

    return native


def make(seed, new, old, Hq, Hkv, d, page, dtype, pad=0, poison=True, spare=3):
    """A cache with the new tokens in it, whose unused slots hold NaN and infinities."""
    rng = np.random.default_rng(seed)
    lens = [a + b for a, b in zip(new, old)]
    need = [-(-max(n, 0) // page) for n in lens]
    n_pages, width = sum(need) + spare, max(max(need), 1)
    table, order, p = np.full((len(lens), width), -1, np.int32), rng.permutation(n_pages), 0
    for b, c in enumerate(need):
        table[b, :c], p = order[p:p + c], p + c
    T = sum(new) + pad
    q = torch.from_numpy(rng.standard_normal((T, Hq, d)) * 2).to(DT[dtype])
    q[T - pad:] = float("nan")
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = {x: torch.randn((n_pages, Hkv, page, d), generator=gen, device="cuda").to(DT[dtype]) for x in "kv"}
    if poison:
        live = torch.zeros((n_pages, 1, page, 1), dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(max(n, 0)):
                live[table[b, j // page], 0, j % page] = True
        c["k"] = torch.where(live.cuda(), c["k"], float("nan"))
        c["v"] = torch.where(live.cuda(), c["v"], float("inf"))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(c, q=q.cuda(), table=torch.from_numpy(table).cuda(), at=i32(np.cumsum([0] + new).tolist()), lens=i32(lens))


def args(c):
    return c["q"], c["k"], c["v"], c["table"], c["at"], c["lens"]


def f64(t):
    return t.double().cpu().numpy()


def check(c, out, lse, scale, dtype, cap=None, odd=False):
    """Bound of a value: the weights enter the second product rounded to the
    type (half a step of each: HALF of the absolute weighted values; fp16 ones
    below 2^-25 of the largest by 2^-36 of it at most), half a step of the
    output's, and through the scores, each a sum of d products in f32 ((d + 4)
    2^-24 sum |q||k| off), 2^-15 of each with the exponential and the sums. lse
    comes from unrounded weights."""
    h = HALF[dtype]
    want, want_lse, mass, reach, most = ref.chunk_attention(f64(c["q"]), f64(c["k"]), f64(c["v"]), c["table"].cpu().numpy(),
                                                            c["at"].cpu().numpy(), c["lens"].cpu().numpy(), scale, cap)
    on = ~np.isnan(want_lse) if not odd else slice(None)
    x_err = (c["q"].shape[2] + 4) * 2.0 ** -24 * reach
    tol = h * np.abs(want) + (h * (1 + h) + 2 * x_err[..., None] + 2.0 ** -15) * mass
    if dtype == "f16":
        tol = tol + 2.0 ** -25 + 2.0 ** -36 * most[..., None]
    assert np.all(np.abs(f64(out) - want)[on] <= tol[on])
    got, none = f64(lse), np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got[on]), none[on])
    tol = x_err + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(none, 0, want_lse))
    on = ~np.isnan(want_lse) & ~none
    assert np.all(np.abs(got - want_lse)[on] <= tol[on])


SHAPES = [
    # dtype, new, old, Hq, Hkv, d, page, pad
    ("f16", [1], [0], 2, 2, 64, 16, 0), ("bf16", [1, 0, 2], [0, 0, 0], 4, 1, 128, 1, 3),
    ("f16", [4], [696], 16, 2, 256, 64, 0), ("bf16", [15, 16, 17], [0, 1, 300], 8, 1, 256, 16, 0),
    ("bf16", [63, 64, 65, 0, 129], [1, 0, 63, 0, 100], 16, 2, 256, 64, 2), ("f16", [300, 5, 0, 77], [0, 9, 3, 0], 5, 1, 128, 17, 1),
    ("f16", [129, 130], [500, 127], 3, 3, 64, 48, 0), ("bf16", [40, 70], [600, 3], 22, 2, 64, 32, 0),
    ("f16", [31, 2], [257, 31], 64, 1, 64, 128, 0), ("bf16", [33, 1, 1], [900, 2000, 0], 24, 1, 128, 256, 0),
    ("bf16", [2] * 40, [(i * 37) % 300 for i in range(40)], 16, 4, 64, 16, 7), ("f16", [600], [0], 6, 2, 128, 1024, 0),
    ("f16", [513], [511], 8, 4, 256, 32, 0), ("bf16", [700], [100], 4, 1, 128, 64, 0), ("f16", [257], [255], 1, 1, 64, 16, 0),
    ("bf16", [1] * 200, [(i * 53) % 700 for i in range(200)], 8, 2, 128, 16, 0),
    ("f16", [8], [9000], 16, 2, 256, 64, 0), ("bf16", [3, 1], [6000, 5000], 20, 4, 128, 16, 0), ("f16", [5], [8191], 8, 1, 64, 32, 0),
    ("bf16", [257, 1, 64], [4000, 4100, 1], 11, 1, 256, 128, 0),
]


@pytest.mark.parametrize("dtype,new,old,Hq,Hkv,d,page,pad", SHAPES)
def test_matches_the_formula(dtype, new, old, Hq, Hkv, d, page, pad):
    native = _native()
    c = make(31, new, old, Hq, Hkv, d, page, dtype, pad)
    T = sum(new)
    out, lse = torch.full_like(c["q"], 7.0), torch.full(c["q"].shape[:2], 7.0, device="cuda")
    native.chunk_attention(*args(c), scale=0.11, out=out, lse=lse)
    torch.cuda.synchronize()
    assert bool((out[T:] == 7).all()) and bool((lse[T:] == 7).all())
    check(c, out, lse, 0.11, dtype)
    again, lse2 = native.chunk_attention(*args(c), scale=0.11, max_len=max(max(c["lens"].tolist()), 1))
    assert again.shape == out.shape
    check(c, again, lse2, 0.11, dtype)
    third, lse3 = native.chunk_attention(*args(c), scale=0.11)
    assert torch.equal(out[:T], third[:T]) and torch.equal(lse[:T], lse3[:T])


@pytest.mark.parametrize("dtype,d", [("f16", 64), ("bf16", 128), ("f16", 256)])
def test_dropped_and_bad_pages_hold_no_keys(dtype, d):
    native = _native()
    c = make(32, [30, 64, 20, 1, 200], [70, 0, 20, 15, 3], 4, 2, d, 16, dtype)
    t = c["table"]
    t[0, 2], t[0, 5] = -1, 1 << 30  # a dropped page, an entry past the pool
    t[1, :] = -5  # nothing left
    t[2, 2] = c["k"].shape[0]  # the last tokens' own page is none
    t[4, 0] = -1  # the first tokens have no key at all
    out, lse = native.chunk_attention(*args(c))
    torch.cuda.synchronize()
    check(c, out, lse, d ** -0.5, dtype)
    assert torch.all(out[30:94] == 0) and torch.all(torch.isneginf(lse[30:94]))
    assert torch.all(out[115:128] == 0) and torch.all(torch.isneginf(lse[115:128]))


@pytest.mark.parametrize("dtype,d", [("f16", 64), ("bf16", 256)])
def test_lengths_past_the_table_or_the_bound_and_below_the_tokens(dtype, d):
    native = _native()
    c = make(33, [20, 20, 20, 3], [28, 28, 28, 200], 4, 2, d, 16, dtype, poison=False)
    c["table"] = c["table"][:, :4].contiguous()
    c["lens"] = torch.tensor([1 << 30, -7, 5, 203], dtype=torch.int32, device="cuda")
    c["table"][0, 3] = c["table"][1, 3] = 0
    out, lse = native.chunk_attention(*args(c))
    check(c, out, lse, d ** -0.5, dtype)
    assert torch.all(out[20:55] == 0) and torch.all(torch.isneginf(lse[20:55]))
    out, lse = native.chunk_attention(*args(c), max_len=33)
    check(c, out, lse, d ** -0.5, dtype, cap=33)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_far_apart_scores(dtype, d):
    """One key far above the rest, early or late; rising scores, each tile's far above the last one's; all alike."""
    native = _native()
    c = make(34, [150, 150, 150, 150], [250] * 4, 2, 1, d, 32, dtype, poison=False)
    c["q"][:] = 0
    c["q"][:, :, 0] = 1.0
    c["q"][450:] = 0
    c["k"][:, :, :, 0] = 0.5
    c["k"][int(c["table"][0, 2]), 0, 7, 0] = 64.0
    c["k"][int(c["table"][1, 7]), 0, 20, 0] = 64.0
    for j in range(400):
        c["k"][int(c["table"][2, j // 32]), 0, j % 32, 0] = j * 0.25
    out, lse = native.chunk_attention(*args(c), scale=1.0)
    check(c, out, lse, 1.0, dtype)
    assert torch.equal(out[0, 0], c["v"][int(c["table"][0, 2]), 0, 7])


@pytest.mark.parametrize("dtype,d", [("f16", 64), ("bf16", 128), ("f16", 256)])
def test_many_keys_of_next_to_no_weight(dtype, d):
    """One key of value 0 that takes almost all weight; 20000 others, each at
    2^-25 of it or so, make up the output."""
    native = _native()
    c = make(35, [3], [20000], 4, 2, d, 64, dtype, poison=False)
    c["q"][:] = 0
    c["q"][:, :, 1] = 1.1
    c["k"][:, :, :, 1] = 0
    pg = int(c["table"][0, 100])
    c["k"][pg, :, 3] = 0
    c["k"][pg, :, 3, 1] = 15.0
    c["v"][:] = c["v"].abs()
    c["v"][pg, :, 3] = 0
    out, lse = native.chunk_attention(*args(c), scale=1.0)
    assert float(out.abs().min()) > 2e-4
    check(c, out, lse, 1.0, dtype)


@pytest.mark.parametrize("dtype,new,old,Hq,Hkv,d", [("f16", [200], [100], 16, 4, 64), ("bf16", [150], [3], 6, 2, 128),
                                                    ("f16", [90, 40], [0, 300], 24, 2, 256), ("bf16", [5], [7000], 16, 2, 256)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("page", [16, 17])
def test_nan_and_infinity_stay_with_the_tokens_that_see_them(dtype, new, old, Hq, Hkv, d, page, bad):
    """A key or value behind a token is masked, whatever it holds; the others'
    outputs keep their bits."""
    native = _native()
    group = Hq // Hkv
    for what in ("q", "k", "v"):
        c = make(36, new, old, Hq, Hkv, d, page, dtype)
        want, want_lse = (x.clone() for x in native.chunk_attention(*args(c)))
        hit = torch.zeros_like(want, dtype=torch.bool)
        last = new[0] - 3
        if what == "q":
            c["q"][last, 3, 5], hit[last, 3] = bad, True
        else:
            p = old[0] + last  # a new token's own key or value
            c[what][int(c["table"][0, p // page]), 1, p % page, 5] = bad
            hit[last:new[0], group:2 * group, slice(None) if what == "k" else 5] = True
        out, lse = native.chunk_attention(*args(c))
        assert torch.equal(out[~hit], want[~hit])
        rows = hit.any(-1) if what != "v" else torch.zeros_like(lse, dtype=torch.bool)
        assert torch.equal(lse[~rows], want_lse[~rows])
        if bad != bad:
            assert bool(out[hit].isnan().all()) and bool(lse[rows].isnan().all())
        elif what == "v":
            assert not bool(out[hit].isfinite().any())


def test_pages_behind_32_bit_offsets():
    native = _native()
    Hkv, page, d = 8, 64, 256
    n_pages = (1 << 32) // (Hkv * page * d) + 9
    k = torch.empty((n_pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    used = [n_pages - 1, 0, n_pages - 5, n_pages // 2 + 1]
    gen = torch.Generator(device="cuda").manual_seed(3)
    for p in used:
        k[p] = torch.randn(k.shape[1:], generator=gen, device="cuda").bfloat16()
        v[p] = torch.randn(k.shape[1:], generator=gen, device="cuda").bfloat16()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    c = dict(q=torch.randn((30, 16, d), generator=gen, device="cuda").bfloat16(), k=k, v=v, table=i32([used]),
             at=i32([0, 30]), lens=i32([250]))
    out, lse = native.chunk_attention(*args(c))
    c.update(k=k[used].clone(), v=v[used].clone(), table=i32([[0, 1, 2, 3]]))
    check(c, out, lse, 1 / 16, "bf16")


@pytest.mark.parametrize("dtype,d,Hq,Hkv", [("f16", 256, 16, 2), ("bf16", 128, 20, 4), ("f16", 64, 3, 3)])
def test_chunks_of_a_prompt_and_single_tokens_agree(dtype, d, Hq, Hkv):
    """A prompt at once, in parts, and its last token as a decode step's: all within the bound of the formula."""
    native = _native()
    c = make(37, [400], [0], Hq, Hkv, d, 16, dtype)
    out, lse = native.chunk_attention(*args(c))
    check(c, out, lse, d ** -0.5, dtype)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for a, b in ((0, 7), (7, 200), (200, 399), (399, 400)):
        part = dict(c, q=c["q"][a:b].contiguous(), at=i32([0, b - a]), lens=i32([b]))
        o, l = native.chunk_attention(*args(part))
        check(part, o, l, d ** -0.5, dtype)
    o, l = native.paged_attention(c["q"][399:].contiguous(), c["k"], c["v"], c["table"], c["lens"])
    assert float((o.float() - out[399:].float()).abs().max()) <= 4 * HALF[dtype] * float(c["v"].float().nan_to_num(0, 0, 0).abs().max())
    assert float((l - lse[399:]).abs().max()) <= 2.0 ** -17


def test_streams_and_a_captured_step():
    native = _native()
    c = make(38, [3, 40, 0, 1], [90, 400, 0, 33], 8, 2, 128, 16, "f16", poison=False)
    want, want_lse = native.chunk_attention(*args(c))
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    got = [native.chunk_attention(*args(c), stream=s) for s in side for _ in range(4)]
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want) and torch.equal(l, want_lse)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        native.chunk_attention(*args(c), out=out, lse=lse)
    c["lens"].copy_(torch.tensor([80, 430, 7, 3], dtype=torch.int32))  # lengths and bounds are read by the replay
    c["at"].copy_(torch.tensor([0, 10, 37, 41, 44], dtype=torch.int32))
    c["table"][2, :1] = c["table"][1, 0]
    graph.replay()
    torch.cuda.synchronize()
    check(c, out, lse, 128 ** -0.5, "f16")


def test_nothing_behind_the_bound_counts():
    """max_len inside a page: what lies behind it, in pages that are there, holds NaN and infinities."""
    native = _native()
    for dtype, d, page in (("f16", 64, 16), ("bf16", 128, 64), ("f16", 256, 128), ("bf16", 256, 17)):
        for cap in (33, 100, 129, 200):
            c = make(40, [20, 90, 1], [190, 130, 209], 4, 2, d, page, dtype)
            for b in range(3):
                for j in range(cap, 260):
                    if j // page < c["table"].shape[1] and int(c["table"][b, j // page]) >= 0:
                        c["k"][int(c["table"][b, j // page]), :, j % page] = float("nan")
                        c["v"][int(c["table"][b, j // page]), :, j % page] = float("inf")
            out, lse = native.chunk_attention(*args(c), max_len=cap)
            check(c, out, lse, d ** -0.5, dtype, cap=cap)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-3, 3.0])
@pytest.mark.parametrize("dtype,d,Hq", [("f16", 64, 7), ("bf16", 128, 9), ("f16", 256, 13)])
def test_scales_of_any_sign_and_odd_groups(dtype, d, Hq, scale):
    native = _native()
    c = make(41, [70, 3], [200, 0], Hq, 1, d, 16, dtype)
    out, lse = native.chunk_attention(*args(c), scale=scale)
    check(c, out, lse, scale, dtype)


def test_sequences_that_share_pages():
    """A prefix of one sequence in the tables of others, and one page in every place of a table."""
    native = _native()
    c = make(42, [5, 40, 12], [150, 160, 180], 8, 2, 128, 16, "bf16", poison=False)
    c["table"][1, :9] = c["table"][0, :9]
    c["table"][2, :] = c["table"][0, 0]
    out, lse = native.chunk_attention(*args(c))
    check(c, out, lse, 128 ** -0.5, "bf16")


@pytest.mark.parametrize("dtype,new,old,Hq,Hkv,d,page", [
    ("f16", [2500], [500], 16, 4, 256, 64), ("bf16", [1800, 3, 700], [100, 5000, 0], 12, 4, 128, 16),
    ("f16", [3100, 40], [0, 2000], 8, 8, 64, 32), ("bf16", [300], [20000], 16, 2, 256, 64)])
def test_many_units(dtype, new, old, Hq, Hkv, d, page):
    """More units than CTAs, handed on and cut, against products in 64 bits on the GPU (bound as in check)."""
    native = _native()
    c = make(43, new, old, Hq, Hkv, d, page, dtype, poison=False)
    out, lse = native.chunk_attention(*args(c))
    again, lse2 = native.chunk_attention(*args(c))
    first, h, group = 0, HALF[dtype], Hq // Hkv
    for b, (n, o) in enumerate(zip(new, old)):
        pages = c["table"][b, :-(-(n + o) // page)].long()
        for i in range(Hkv):
            k, v = (c[x][pages, i].reshape(-1, d)[:n + o].double() for x in "kv")
            for a in range(0, n, 512):
                e = min(n, a + 512)
                q = c["q"][first + a:first + e, i * group:(i + 1) * group].double()
                x = torch.einsum("thd,kd->thk", q, k) * d ** -0.5
                seen = torch.ones(e - a, n + o, dtype=torch.bool, device="cuda").tril(o + a)[:, None]
                x = torch.where(seen, x, -torch.inf)
                p = torch.softmax(x, 2)
                want, mass = torch.einsum("thk,kd->thd", p, v), torch.einsum("thk,kd->thd", p, v.abs())
                reach = torch.where(seen, torch.einsum("thd,kd->thk", q.abs(), k.abs()), 0).amax(2) * d ** -0.5
                x_err = (d + 4) * 2.0 ** -24 * reach
                tol = h * want.abs() + (h * (1 + h) + 2 * x_err[..., None] + 2.0 ** -15) * mass
                if dtype == "f16":
                    tol = tol + 2.0 ** -25 + 2.0 ** -36 * (n + o) * float(v.abs().max())
                rows = slice(first + a, first + e), slice(i * group, (i + 1) * group)
                assert bool(((out[rows].double() - want).abs() <= tol).all())
                want = torch.logsumexp(x, 2)
                assert bool(((lse[rows].double() - want).abs() <= x_err + 2.0 ** -20 + 2.0 ** -22 * want.abs()).all())
        first += n
    assert torch.equal(lse, lse2) and torch.equal(out, again)


def test_outputs_at_any_16_bytes():
    native = _native()
    c = make(44, [33], [50], 6, 2, 64, 16, "f16")
    want, want_lse = native.chunk_attention(*args(c))
    for off in (8, 16, 24):
        buf = torch.full((33 * 6 * 64 + 64,), 7.0, dtype=torch.float16, device="cuda")
        out = buf[off:off + 33 * 6 * 64].view(33, 6, 64)
        native.chunk_attention(*args(c), out=out)
        assert torch.equal(out, want) and bool((buf[:off] == 7).all()) and bool((buf[off + 33 * 6 * 64:] == 7).all())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_bounds_that_descend_stay_in_the_buffers(d):
    """Not allowed, and without meaning: but the call ends, what lies around the buffers stays, and the next call is right."""
    native = _native()
    c = make(45, [30, 30, 30, 30], [300, 0, 5000, 9], 4, 2, d, 16, "bf16", poison=False)
    want, want_lse = native.chunk_attention(*args(c))
    for at in ([0, 120, 0, 120, 5], [120, 90, 60, 30, 0], [-5, 1 << 30, -1 << 30, 7, 1 << 30], [0, 0, 0, 0, 0]):
        buf = torch.full((120 * 4 * d + 2048,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[1024:1024 + 120 * 4 * d].view(120, 4, d)
        bad = dict(c, at=torch.tensor(at, dtype=torch.int32, device="cuda"))
        native.chunk_attention(*args(bad), out=out)
        torch.cuda.synchronize()
        assert bool((buf[:1024] == 7).all()) and bool((buf[-1024:] == 7).all())
    out, lse = native.chunk_attention(*args(c))
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_two_captured_graphs_with_their_own_workspaces():
    native = _native()
    cs = [make(46 + i, [4, 1], [5000, 300], 16, 2, 256, 64, "f16", poison=False) for i in range(2)]
    want = [native.chunk_attention(*args(c)) for c in cs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(native.chunk_attention(*args(c)))
        graphs.append(g)
    side = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_refusals():
    native = _native()
    c = make(39, [10], [30], 4, 2, 64, 16, "f16")
    good = dict(q=c["q"], k_pool=c["k"], v_pool=c["v"], table=c["table"], at=c["at"], lens=c["lens"])

    def bad(exc, **kw):
        with pytest.raises(exc):
            native.chunk_attention(**{**good, **kw})

    bad(TypeError, k_pool=c["k"].bfloat16())
    bad(TypeError, lens=c["lens"].long())
    bad(TypeError, at=c["at"].float())
    bad(ValueError, lens=c["lens"].repeat(2))
    bad(ValueError, at=c["at"].repeat(2))
    bad(ValueError, q=c["q"].transpose(1, 2))
    bad(ValueError, table=c["table"].cpu())
    bad(ValueError, out=c["q"][:5].clone())
    bad(native.EschaError, scale=float("nan"))
    bad(native.EschaError, q=c["q"][:, :3].contiguous())
    bad(native.EschaError, max_len=0)
    bad(ValueError, ws=torch.empty(16, device="cuda"))
    one = make(39, [4], [20000], 16, 2, 64, 16, "f16", poison=False)  # few tokens over many keys: parts in a workspace
    with pytest.raises(native.EschaError, match="workspace"):
        native.chunk_attention(*args(one), ws=torch.empty(256, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype,Hq,Hkv,d", [("f16", 8, 2, 64), ("bf16", 6, 3, 128), ("f16", 16, 2, 256)])
@pytest.mark.parametrize("page", [16, 17])
@pytest.mark.parametrize("cut", [False, True])
def test_short_sequences_keep_their_values_that_are_not_finite(dtype, Hq, Hkv, d, page, cut):
    """CTAs that take one short unit after another: a NaN or an infinity among a sequence's last values shows in every column that has
    one, of every token that attends it, and nowhere else. ``cut``: few enough sequences under a bound that cuts all units into ranges."""
    native = _native()
    rng = np.random.default_rng(50)
    if cut:
        Hkv, Hq = 8, 8 * (Hq // Hkv)
    n, max_len = (110, 1 << 18) if cut else (300, 128)
    new = rng.integers(1, 6, n).tolist()
    c = make(51, new, rng.integers(0, 123, n).tolist(), Hq, Hkv, d, page, dtype)
    c["table"] = torch.nn.functional.pad(c["table"], (0, max_len // page), value=0)
    need = native.lib().escha_chunk_attention_workspace(n, sum(new), Hq, Hkv, d, max_len)
    assert (need > 0) == cut
    table, lens = c["table"].cpu().numpy(), c["lens"].tolist()
    for s in range(n):
        for _ in range(rng.integers(0, 4)):  # values of new tokens: seen by them and those behind them
            j, (a, b) = lens[s] - 1 - rng.integers(0, new[s]), sorted(rng.integers(0, d + 1, 2))
            c["v"][int(table[s, j // page]), rng.integers(0, Hkv), j % page, a:b] = (float("nan"), float("inf"), float("-inf"))[rng.integers(0, 3)]
    nan, plus, minus = (np.zeros((sum(new), Hq, d), bool) for _ in range(3))
    seq, pos = ref.places(np.cumsum([0] + new), lens, sum(new))
    v = f64(c["v"])
    for t in range(sum(new)):  # what each token attends, from the cache as it is
        pages = table[seq[t], :pos[t] // page + 1]
        rows = np.concatenate(v[pages], 1)[:, :pos[t] + 1]
        for what, has in ((nan, np.isnan(rows)), (plus, np.isposinf(rows)), (minus, np.isneginf(rows))):
            what[t] = np.repeat(has.any(1), Hq // Hkv, 0)
    nan |= plus & minus
    for _ in range(3):
        out, lse = native.chunk_attention(*args(c), max_len=max_len)
        got = f64(out)
        assert np.array_equal(np.isnan(got), nan)
        assert np.array_equal(got == np.inf, plus & ~nan) and np.array_equal(got == -np.inf, minus & ~nan)
    clean = dict(c, v=torch.where(c["v"].isfinite(), c["v"], 0))
    want, want_lse = native.chunk_attention(*args(clean), max_len=max_len)
    odd = torch.from_numpy(nan | plus | minus).cuda()
    assert torch.equal(out[~odd], want[~odd]) and torch.equal(lse, want_lse)
    check(clean, want, want_lse, d ** -0.5, dtype)


@pytest.mark.parametrize("dtype,n,longest,Hq,Hkv,d,page", [("f16", 300, 6, 8, 2, 64, 16), ("bf16", 400, 3, 4, 4, 128, 17), ("f16", 200, 60, 16, 2, 256, 64)])
def test_units_are_taken_over_in_any_order(dtype, n, longest, Hq, Hkv, d, page):
    """Whole units of many sequences, handed out from the first or from the last one on: every row is written, with the same bits."""
    native = _native()
    rng = np.random.default_rng(52)
    new = rng.integers(0, longest + 1, n)
    new[rng.integers(0, n, n // 10)] = 0
    new[40:90] = 0  # more than 32 in a row that have none
    c = make(53, new.tolist(), rng.integers(0, 200, n).tolist(), Hq, Hkv, d, page, dtype, pad=2)
    assert native.lib().escha_chunk_attention_workspace(n, int(new.sum()) + 2, Hq, Hkv, d, 512) == 0  # (whole units)
    got = []
    for backwards in (False, True):
        native.set_chunk_order(backwards)
        try:
            out, lse = torch.full_like(c["q"], 7.0), torch.full(c["q"].shape[:2], 7.0, device="cuda")
            native.chunk_attention(*args(c), max_len=512, out=out, lse=lse)
            torch.cuda.synchronize()
        finally:
            native.set_chunk_order()
        assert bool((out[-2:] == 7).all()) and bool((lse[-2:] == 7).all())
        got.append((out, lse))
    check(c, *got[0], d ** -0.5, dtype)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("d,old", [(64, 200), (128, 200), (256, 200), (256, 9000)])
def test_large_values_behind_a_slowly_rising_maximum(d, old):
    """bf16 values near the type's largest, where the scores' maximum rises by 5.8 powers of two from a tile to a later one: the weights
    of what is summed stay at 1 or below, so the sums of two such values with weights 1 and e^-4 stay finite (1.02 * 2e38)."""
    native = _native()
    c = make(55, [6, 40], [old, 150], 4, 2, d, 16, "bf16", poison=False)
    c["q"][:] = 0
    c["q"][:, :, 0] = 1
    c["k"][..., 0] = -100
    for s in range(2):
        for j, x in ((3, 0.0), (140, 4.0)):
            pg = int(c["table"][s, j // 16])
            c["k"][pg, :, j % 16, 0], c["v"][pg, :, j % 16] = x, 2e38
    out, lse = native.chunk_attention(*args(c), scale=1.0)
    assert bool(out.isfinite().all())
    check(c, out, lse, 1.0, "bf16")


GIVE_UP = [("f16", [3] * 200, [(i * 37) % 400 for i in range(200)], 8, 2, 64, 1024), ("bf16", [4, 30], [9000, 700], 16, 2, 256, None),
           ("bf16", [700, 2, 40], [100, 3000, 0], 12, 4, 128, None), ("f16", [900], [300], 16, 2, 256, 1200)]


@pytest.mark.parametrize("dtype,new,old,Hq,Hkv,d,max_len", GIVE_UP)
@pytest.mark.parametrize("page", [16, 17])
def test_a_call_whose_waits_give_up_ends(dtype, new, old, Hq, Hkv, d, max_len, page):
    """Waits between the warps that run out after a few polls: the call ends, and the next one is right."""
    native = _native()
    c = make(54, new, old, Hq, Hkv, d, page, dtype, poison=False)
    want, want_lse = native.chunk_attention(*args(c), max_len=max_len)
    torch.cuda.synchronize()
    for polls in (0, 1, 3, 10, 40):
        native.set_chunk_wait(polls)
        try:
            began = time.time()
            native.chunk_attention(*args(c), max_len=max_len)
            torch.cuda.synchronize()
            assert time.time() - began < 5
        finally:
            native.set_chunk_wait()
        out, lse = native.chunk_attention(*args(c), max_len=max_len)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("dtype,new,old,Hq,Hkv,d,max_len", GIVE_UP)
@pytest.mark.parametrize("page", [16, 17])
@pytest.mark.parametrize("backwards", [False, True])
def test_rows_are_right_or_nan_after_waits_that_gave_up(dtype, new, old, Hq, Hkv, d, max_len, page, backwards):
    """Whatever was left undone is NaN, in whole heads and in lse, not what the buffers or the workspace held."""
    native = _native()
    c = make(56, new, old, Hq, Hkv, d, page, dtype, poison=False)
    want, want_lse = native.chunk_attention(*args(c), max_len=max_len)
    n, T, cap = len(new), sum(new), max_len or c["table"].shape[1] * page
    ws = torch.empty(max(native.lib().escha_chunk_attention_workspace(n, T, Hq, Hkv, d, cap), 16), dtype=torch.uint8, device="cuda")
    other = dict(c, q=torch.randn_like(c["q"]))
    for polls in (0, 1, 2, 5, 20, 100):
        native.chunk_attention(*args(other), max_len=max_len, ws=ws)  # parts of another call in the workspace
        out, lse = torch.full_like(want, 7.0), torch.full_like(want_lse, 7.0)
        native.set_chunk_wait(polls)
        native.set_chunk_order(backwards)
        try:
            native.chunk_attention(*args(c), max_len=max_len, ws=ws, out=out, lse=lse)
            torch.cuda.synchronize()
        finally:
            native.set_chunk_wait()
            native.set_chunk_order()
        nan = lse.isnan()
        assert bool(((out == want).all(-1) | nan).all()) and bool(((lse == want_lse) | nan).all())
        assert bool(out[nan].isnan().all())
        if polls == 0:
            assert bool(nan.any())
    out, lse = native.chunk_attention(*args(c), max_len=max_len)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
