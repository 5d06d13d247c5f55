"""GPU checks of escha_token_logprobs against its formula in 64 bits."""
import numpy as np
import pytest

import mixer_refs as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _native():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_trellis_quantized_gb300 import native

    return native


def run_and_check(native, x, ids, top):
    """Of ln s: every term's exponential is within 2^-20 (the exponent's
    rounding, |x - m| 2^-23 where the term still counts, and the function's),
    sums add 2^-20 more. Of a log probability or lse: that and the f32 roundings
    of its parts. Of the entropy: ln s, and t / s with terms (x - m) p."""
    r = native.token_logprobs(x, None if ids is None else torch.from_numpy(ids.astype(np.int32)).cuda(), top)
    torch.cuda.synchronize()
    x64 = x.double().cpu().numpy()
    want = ref.logprobs(x64, np.zeros((len(x64), 0), int) if ids is None else ids, top)
    got = {k: None if v is None else v.double().cpu().numpy() for k, v in r.items()}
    assert np.array_equal(got["top_ids"], want["top_ids"])

    def near(a, b, abs_tol):
        assert a.shape == b.shape
        odd = ~np.isfinite(b)
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(a[odd & ~np.isnan(b)], b[odd & ~np.isnan(b)])
        assert np.all(np.abs(a - b)[~odd] <= (abs_tol + 2.0 ** -22 * np.abs(np.where(odd, 0, b)))[~odd])

    near(got["lse"], want["lse"], 2.0 ** -19)
    if ids is not None:
        near(got["logprobs"], want["logprobs"], 2.0 ** -19)
    near(got["top_logprobs"], want["top_logprobs"], 2.0 ** -19)
    near(got["entropy"], want["entropy"], 2.0 ** -17)
    return r


SIZES = [(1, 1, 1), (2, 2, 0), (3, 5, 5), (5, 17, 3), (1, 31, 31), (4, 33, 32), (7, 1000, 20), (2, 4096, 1),
         (3, 4099, 7), (1, 8191, 32), (700, 257, 4), (1, 40000, 20), (3, 152064, 8), (650, 6007, 2)]


@pytest.mark.parametrize("M,V,top", SIZES)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_matches_the_formula(M, V, top, dtype):
    native = _native()
    rng = np.random.default_rng(31)
    x = torch.from_numpy(rng.standard_normal((M, V)) * 3).to(DT[dtype]).cuda()
    ids = rng.integers(0, V, (M, 3))
    a = run_and_check(native, x, ids, top)
    b = run_and_check(native, x, ids, top)
    for k in a:
        assert torch.equal(a[k], b[k])


@pytest.mark.parametrize("dtype,M,V", [("f16", 2, 161024), ("bf16", 4, 165185), ("f16", 5, 135991), ("f32", 2, 156288)])
def test_last_row_in_more_parts_than_an_even_share(dtype, M, V):
    """Ranges of 8 and 9 units (16 and 17): the last row lies in the smaller
    ones, up to 5 parts more than CTAs / M + 2; its largest values are in its
    last parts."""
    native = _native()
    rng = np.random.default_rng(38)
    x = rng.standard_normal((M, V)) * 3
    x[:, V - 3000::97] += 20
    run_and_check(native, torch.from_numpy(x).to(DT[dtype]).cuda(), rng.integers(0, V, (M, 2)), 32)


@pytest.mark.parametrize("dtype,M,V", [("f32", 1, 500000), ("bf16", 2, 900001), ("f32", 5, 393693), ("bf16", 28, 30001),
                                       ("f16", 29, 30003), ("f32", 68, 10007), ("bf16", 69, 10005), ("f16", 100, 31000),
                                       ("f16", 153, 31001), ("f32", 306, 6000)])
def test_every_way_rows_are_dealt_out(dtype, M, V):
    """Cut over all CTAs, in clusters of 8, 4 and 2, one a CTA; rows on every
    alignment, their largest values at both ends and in the middle."""
    native = _native()
    rng = np.random.default_rng(39)
    x = rng.standard_normal((M, V + 1)) * 3
    for at in (0, 3, V // 2, V - 2, V - 1):
        x[:, at] += 12 + rng.standard_normal(M)
    x = torch.from_numpy(x).to(DT[dtype]).cuda()[:, :V]
    ids = rng.integers(0, V, (M, 2))
    a, b = run_and_check(native, x, ids, 32), run_and_check(native, x, ids, 32)
    for k in a:
        assert torch.equal(a[k], b[k])
    run_and_check(native, x, None, 0)


def test_many_long_rows():
    native = _native()
    gen = torch.Generator(device="cuda").manual_seed(40)
    M, V = 306, 100500
    x = torch.randn((M, V), generator=gen, device="cuda") * 3
    r = native.token_logprobs(x, torch.zeros(M, dtype=torch.int32, device="cuda"), 5)
    lp = torch.log_softmax(x.double(), 1)
    assert float((r["logprobs"] - lp[:, 0]).abs().max()) <= 2.0 ** -18
    assert float((r["entropy"] + (lp.exp() * lp).sum(1)).abs().max()) <= 2.0 ** -16
    want = torch.topk(x, 5, 1).indices
    assert torch.equal(torch.gather(x, 1, r["top_ids"].long()), torch.gather(x, 1, want))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_rows_that_start_anywhere(dtype):
    """Rows a stride apart that leaves them on every alignment, what lies
    between them not read as theirs."""
    native = _native()
    rng = np.random.default_rng(32)
    for V, ld in ((1003, 1009), (9, 13), (8000, 8003)):
        whole = torch.full((9, ld), float("inf"), dtype=DT[dtype], device="cuda")
        whole[:, :V] = torch.from_numpy(rng.standard_normal((9, V)) * 3).to(DT[dtype]).cuda()
        run_and_check(native, whole[:, :V], rng.integers(0, V, (9, 1)), 9)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("V", [50, 5000])
def test_masks_infinities_and_ties(dtype, V):
    native = _native()
    rng = np.random.default_rng(33)
    x = torch.from_numpy(rng.standard_normal((12, V)) * 3).to(DT[dtype]).cuda()
    low = torch.finfo(DT[dtype]).min
    x[0, ::2] = -float("inf")
    x[1] = -float("inf")  # nothing left
    x[2] = -float("inf")
    x[2, V - 3] = -7.5  # one token left
    x[3] = low
    x[4, 1:] = low
    x[5] = 2.25  # all alike: the lowest ids
    x[6] = torch.round(x[6])  # many ties
    x[7, 20] = float("nan")
    x[8, 21] = float("inf")
    x[9, 5], x[9, 30] = float("inf"), float("nan")
    x[10] = torch.where(x[10] > 0, 0.0, -0.0)  # both zeros rank alike
    x[11] = torch.sort(x[11].float()).values.to(DT[dtype])  # the largest last
    ids = rng.integers(0, V, (12, 4))
    ids[:, 1], ids[:, 2] = -1, V
    ids[3, 3], ids[7, 3] = -2, 20
    run_and_check(native, x, ids, 32)
    run_and_check(native, x, ids, 1)


def test_far_values():
    native = _native()
    x = torch.zeros((4, 600), device="cuda")
    x[0], x[1, 3], x[2, 9] = 3e38, 3e38, -3e38
    x[3] = torch.linspace(-500, 500, 600)
    run_and_check(native, x, np.array([[0, 599]] * 4), 5)


def test_no_ids_and_one_id_a_row():
    native = _native()
    rng = np.random.default_rng(34)
    x = torch.from_numpy(rng.standard_normal((5, 900))).float().cuda()
    r = run_and_check(native, x, None, 3)
    assert r["logprobs"] is None
    one = native.token_logprobs(x, torch.arange(5, dtype=torch.int32, device="cuda"))
    two = native.token_logprobs(x, torch.arange(5, dtype=torch.int32, device="cuda")[:, None])
    assert one["logprobs"].shape == (5,) and torch.equal(one["logprobs"], two["logprobs"][:, 0])
    assert one["top_ids"].shape == (5, 0)


def test_more_rows_than_a_grid_has():
    native = _native()
    gen = torch.Generator(device="cuda").manual_seed(35)
    x = torch.randn((70001, 40), generator=gen, device="cuda")
    ids = torch.randint(0, 40, (70001,), generator=gen, device="cuda", dtype=torch.int32)
    r = native.token_logprobs(x, ids, 2)
    lp = torch.log_softmax(x.double(), 1)
    assert float((r["logprobs"] - lp.gather(1, ids.long()[:, None])[:, 0]).abs().max()) <= 2.0 ** -18
    assert torch.equal(r["top_ids"][:, 0].long(), x.argmax(1))


def test_rows_behind_32_bit_offsets():
    native = _native()
    V = 152064
    M = (1 << 32) // V + 3
    x = torch.zeros((M, V), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(36)
    rows = torch.from_numpy(rng.standard_normal((2, V)) * 3).bfloat16().cuda()
    x[0], x[-1] = rows[0], rows[1]
    ids = torch.full((M,), V - 1, dtype=torch.int32, device="cuda")
    r = native.token_logprobs(x, ids, 4)
    few = native.token_logprobs(rows, ids[:2].contiguous(), 4)
    for a, b in ((0, 0), (M - 1, 1)):
        assert torch.equal(r["top_ids"][a], few["top_ids"][b])
        assert abs(float(r["logprobs"][a] - few["logprobs"][b])) <= 2.0 ** -18


def test_streams_and_a_captured_call():
    native = _native()
    gen = torch.Generator(device="cuda").manual_seed(37)
    x = torch.randn((3, 50000), generator=gen, device="cuda")
    ids = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
    want = native.token_logprobs(x, ids, 10)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    got = [native.token_logprobs(x, ids, 10, stream=s) for s in side for _ in range(3)]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(r[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = native.token_logprobs(x, ids, 10)
    x.copy_(torch.randn((3, 50000), generator=gen, device="cuda"))
    want = native.token_logprobs(x, ids, 10)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(r[k], want[k]) for k in want)


def test_refusals():
    native = _native()
    x = torch.zeros((4, 100), device="cuda")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    for exc, a in ((ValueError, (x.t(), ids)), (ValueError, (x[0], ids)), (ValueError, (x.cpu(), ids)),
                   (TypeError, (x.double(), ids)), (TypeError, (x, ids.long())), (ValueError, (x, ids[:3])),
                   (native.EschaError, (x, ids, 33)), (native.EschaError, (x, ids, -1)),
                   (native.EschaError, (x[:, :8], ids, 9)), (native.EschaError, (x.flatten()[1:97].view(4, 24), ids)),
                   (ValueError, (x[:1].expand(4, 100), ids))):
        with pytest.raises(exc):
            native.token_logprobs(*a)


# by the way that rows are dealt out: a warp a row, a CTA, clusters of 4, 8 and 2, cut over all CTAs
WAYS = [(14, 50, d) for d in DT] + [(14, 5000, d) for d in DT] + [(14, 12001, d) for d in DT] + [
    (14, 30001, d) for d in DT] + [(70, 30004, d) for d in DT] + [(14, 1400001, "f16"), (14, 1400001, "bf16"), (14, 700001, "f32")]


@pytest.mark.parametrize("M,V,dtype", WAYS)
def test_finite_masks_and_far_maxima(M, V, dtype):
    """Tokens masked with finite values of every size, in runs longer than all
    that a lane, a warp and a CTA read; rows whose largest value is far from 0;
    values on both sides of 2^20 within reach of each other."""
    native = _native()
    rng = np.random.default_rng(41)
    x = torch.from_numpy(rng.standard_normal((M, V)) * 3).float().cuda()
    masks, far, edge = (1e9, 1e10, 1e20, 1e30, 1e36), (1e10, 1e30), 2.0 ** 20
    if dtype == "f16":  # as far as the type goes
        masks, far, edge = (6e4,) * 5, (6e4, 65504.0), 6e4
    keep = (slice(7, 12), slice(V - V // 4, V), slice(V - 3, V - 2), slice(V // 3, V // 3 + 9), slice(0, 1))
    for i in range(M):
        k, y = i % 14, x[i].clone()
        if k < 5:
            x[i] = -masks[k]
            x[i, keep[k]] = y[keep[k]]
        elif k == 5:  # three masks, and what is left
            x[i, :V // 5], x[i, V // 5:V // 2], x[i, V // 2:V - V // 5] = -masks[0], -masks[1], -masks[2]
        elif k == 6:
            x[i] = -far[0]
        elif k == 7:
            x[i] = far[1]
        elif k == 8:
            x[i, V // 2] = far[0]
        elif k == 9:
            x[i] = y * far[0] / 100 - far[0]
        elif k == 10:
            x[i] = y + edge
        elif k == 11:
            x[i] = y - edge
        elif k == 12:
            x[i] = y * 5 + 0.95 * edge
        else:
            x[i] = y * 5 - 0.95 * edge
    x = x.to(DT[dtype])
    if dtype == "f16":
        x = x.clamp(-65504, 65504)
    assert bool(x.isfinite().all())
    ids = rng.integers(0, V, (M, 4))
    ids[:, 0], ids[:, 1] = V - 3, 8
    r = run_and_check(native, x, ids, 32)
    none = native.token_logprobs(x, torch.from_numpy(ids.astype(np.int32)).cuda())
    assert all(torch.equal(r[k], none[k]) for k in ("lse", "entropy", "logprobs"))  # the sums do not hang on the top list


@pytest.mark.parametrize("M,V,dtype", WAYS[3:])
def test_masks_infinities_and_ties_every_way(M, V, dtype):
    """What bans tokens, breaks a row or fills the lists of its largest, over
    the ways that share a row among warps and CTAs; at both ends of a row and
    inside, so that each part of it has some."""
    native = _native()
    rng = np.random.default_rng(43)
    x = torch.from_numpy(rng.standard_normal((M, V)) * 3).to(DT[dtype]).cuda()
    low, inf, nan = torch.finfo(DT[dtype]).min, float("inf"), float("nan")
    for i in range(M):
        k, y = i % 14, x[i]
        if k == 0:
            y[::2] = -inf
        elif k == 1:
            y[:] = -inf  # nothing left
        elif k == 2:
            y[:V - 3], y[V - 2:] = -inf, -inf  # one token left
        elif k == 3:
            y[:] = low
        elif k == 4:
            y[:V // 2], y[V // 2 + 1:] = low, -inf
        elif k == 5:
            y[:] = 2.25  # all alike: the lowest ids
        elif k == 6:
            x[i] = torch.round(y)  # many ties
        elif k == 7:
            y[V - 2] = nan
        elif k == 8:
            y[V // 2] = inf
        elif k == 9:
            y[:], y[V - 1], y[3] = -inf, inf, nan
        elif k == 10:
            x[i] = torch.where(y > 0, 0.0, -0.0)  # both zeros rank alike
        elif k == 11:
            x[i] = torch.sort(y.float()).values.to(DT[dtype])  # the largest last
        elif k == 12:
            x[i] = torch.sort(y.float(), descending=True).values.to(DT[dtype])
        else:
            y[40:] = nan  # more of them than the list holds
    ids = rng.integers(0, V, (M, 4))
    ids[:, 1], ids[:, 2], ids[:, 3] = -1, V, V - 3
    run_and_check(native, x, ids, 32)
    run_and_check(native, x, ids, 1)
