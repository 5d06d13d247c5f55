"""GPU checks of escha_adjust_logits against its formula in 64 bits."""
import numpy as np
import pytest

import chunk_refs as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _native():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_trellis_quantized_gb300 import native

    return native


def make(seed, M, V, dtype, history=0, bias=0, masks=0, wide=0):
    rng = np.random.default_rng(seed)
    c = dict.fromkeys(("ids", "at", "prompt", "repetition", "frequency", "presence", "bias_ids", "bias", "bias_at",
                       "allowed", "allowed_rows"))
    if history:
        n = rng.integers(0, history + 1, M)
        n[0] = history
        c["at"] = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        c["ids"] = (rng.random(n.sum()) ** 3 * V).astype(np.int32)
        c["ids"][rng.random(n.sum()) < 0.02] = -1
        c["ids"][rng.random(n.sum()) < 0.02] = V
        c["prompt"] = rng.integers(0, n + 1).astype(np.int32)
        c["repetition"] = (1 + rng.random(M)).astype(np.float32)
        c["frequency"] = rng.random(M).astype(np.float32)
        c["presence"] = (rng.random(M) - 0.3).astype(np.float32)
    if bias:
        n = rng.integers(0, bias + 1, M)
        n[-1] = bias
        c["bias_at"] = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        c["bias_ids"] = rng.integers(-1, V + 1, n.sum()).astype(np.int32)  # (an id may come twice)
        c["bias"] = (4 * rng.standard_normal(n.sum())).astype(np.float32)
    if masks:
        c["allowed"] = rng.integers(-2 ** 31, 2 ** 31, (masks, (V + 31) // 32)).astype(np.int32)
        c["allowed_rows"] = rng.integers(-1, masks + 1, M).astype(np.int32)
    x = torch.from_numpy(rng.standard_normal((M, V + wide)) * 3).to(DT[dtype]).cuda()[:, :V]
    return x, c


def dev(c):
    return {k: None if v is None else torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in c.items()}


def check(x, c, got, dtype):
    """Five f32 operations at most but for biases, each within 2^-24 of the largest
    value on the way: 2^-21 of the sum of what is added, and half a step of the type."""
    x64 = x.double().cpu().numpy()
    want = ref.adjust_logits(x64, *(c[k] for k in ("ids", "at", "prompt", "repetition", "frequency", "presence", "bias_ids",
                                                   "bias", "bias_at", "allowed", "allowed_rows")))
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    size = np.where(np.isfinite(x64), np.abs(x64), 0)
    if c["repetition"] is not None:
        size = size * np.maximum(c["repetition"], 1)[:, None]
    for m in range(len(x64)):
        for lists, at, amount in (("ids", "at", None), ("bias_ids", "bias_at", "bias")):
            if c[lists] is None:
                continue
            a, b = (min(max(int(i), 0), len(c[lists])) for i in c[at][m:m + 2])
            ids = c[lists][a:b]
            ok = (ids >= 0) & (ids < x64.shape[1])
            if amount:
                np.add.at(size[m], ids[ok], np.abs(c["bias"][a:b][ok]))
            else:
                f = abs(float(c["frequency"][m])) if c["frequency"] is not None else 0
                p = abs(float(c["presence"][m])) if c["presence"] is not None else 0
                np.add.at(size[m], ids[ok], f + p)
    on = np.isfinite(want)
    tol = HALF[dtype] * np.abs(want[on]) * (1 + 2.0 ** -10) + 2.0 ** -21 * size[on] + (2.0 ** -25 if dtype == "f16" else 0)
    same = x64[on] == want[on]
    assert np.array_equal(got[on][same], want[on][same])
    assert np.all(np.abs(got[on] - want[on]) <= tol)


SIZES = [(1, 1, 3, 2, 1), (3, 20, 7, 5, 2), (2, 31, 40, 0, 2), (5, 33, 0, 3, 0), (4, 1000, 500, 20, 3), (2, 4097, 100, 300, 0),
         (3, 40003, 3000, 50, 3), (1, 152064, 900, 20, 0), (5, 152064, 2000, 5, 4), (7, 65537, 0, 0, 7), (200, 5003, 60, 10, 30),
         (2, 260001, 5000, 100, 1), (1, 9, 0, 0, 0)]


@pytest.mark.parametrize("M,V,history,bias,masks", SIZES)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_matches_the_formula(M, V, history, bias, masks, dtype):
    native = _native()
    for wide in (0, 5, 8):
        x, c = make(41 + wide, M, V, dtype, history, bias, masks, wide)
        raw, d = x.clone(), dev(c)
        got = native.adjust_logits(x, **d)
        assert torch.equal(x, raw)
        check(x, c, got, dtype)
        assert native.adjust_logits(x, **d, out=x) is x
        assert torch.equal(x, got)
        if wide:  # what lies between the rows stays
            behind = torch.as_strided(x, (M, wide), (V + wide, 1), V) if M > 1 else x[:0]
            before = torch.as_strided(make(41 + wide, M, V, dtype, history, bias, masks, wide)[0], (M, wide), (V + wide, 1), V) if M > 1 else x[:0]
            assert torch.equal(behind, before)
        other = torch.zeros((M, V + 3), dtype=x.dtype, device="cuda")[:, :V]  # rows aligned otherwise
        native.adjust_logits(raw, **d, out=other)
        assert torch.equal(other, got)


def test_each_part_alone_and_an_id_many_times():
    native = _native()
    x = torch.tensor([[2.0, -2.0, 0.0, -0.0, 5.0, 1.0]], device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    f32 = lambda a: torch.tensor(a, dtype=torch.float32, device="cuda")  # noqa: E731
    ids, at = i32([0, 1, 1, 4, 4, 4, 2]), i32([0, 7])
    out = native.adjust_logits(x, ids, at, repetition=f32([2.0]))
    assert out.tolist() == [[1.0, -4.0, 0.0, 0.0, 2.5, 1.0]]
    out = native.adjust_logits(x, ids, at, prompt=i32([2]), frequency=f32([0.5]))
    assert out.tolist() == [[2.0, -2.5, -0.5, 0.0, 3.5, 1.0]]
    out = native.adjust_logits(x, ids, at, prompt=i32([100]), presence=f32([0.25]), frequency=f32([9.0]))
    assert torch.equal(out, x)
    out = native.adjust_logits(x, ids, at, presence=f32([0.25]))
    assert out.tolist() == [[1.75, -2.25, -0.25, 0.0, 4.75, 1.0]]
    out = native.adjust_logits(x, bias_ids=i32([5, 5, 0, 5]), bias=f32([1e8, -1e8, 3.0, 0.5]), bias_at=i32([0, 4]))
    assert out.tolist() == [[5.0, -2.0, 0.0, 0.0, 5.0, 0.5]]  # in list order: (1 + 1e8) - 1e8 is 0 in f32
    out = native.adjust_logits(x, allowed=i32([[0b010011]]))
    assert out.tolist() == [[2.0, -2.0, float("-inf"), float("-inf"), 5.0, float("-inf")]]
    assert torch.equal(native.adjust_logits(x), x)
    many = i32([3] * 100000 + [4] * 7)
    out = native.adjust_logits(x, many, i32([0, 100007]), prompt=i32([1]), frequency=f32([0.25]))
    assert out[0].tolist() == [2.0, -2.0, 0.0, -0.25 * 99999, 5 - 0.25 * 7, 1.0]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_nan_infinity_and_the_lowest_value(dtype):
    """NaN stays but where it is banned; infinities keep their sign; the type's lowest value times a penalty is -infinity."""
    native = _native()
    x, c = make(43, 2, 3001, dtype, 600, 30, 1)
    c["allowed_rows"][:] = [0, -1]
    low = torch.finfo(DT[dtype]).min
    for i, v in enumerate((float("nan"), float("inf"), float("-inf"), low)):
        x[:, i::97] = v
    got = native.adjust_logits(x, **dev(c))
    x64, lowest = x.double().cpu().numpy(), float(low)
    want = ref.adjust_logits(x64, *(c[k] for k in ("ids", "at", "prompt", "repetition", "frequency", "presence", "bias_ids",
                                                   "bias", "bias_at", "allowed", "allowed_rows")))
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    for sign in (1, -1):
        assert np.all(got[want == sign * np.inf] == sign * np.inf)
    assert np.all(got[want < 1.01 * lowest] == -np.inf)


def test_bounds_of_the_lists_are_clamped_and_masks_out_of_range_are_none():
    native = _native()
    x, c = make(44, 4, 500, "f32", 50, 9, 2)
    c["at"][0], c["at"][-1] = -3, 1 << 30
    c["bias_at"][-1] = 1 << 30
    c["prompt"][1] = -9
    c["allowed_rows"][:] = [2, -(1 << 31), (1 << 31) - 1, 1]
    check(x, c, native.adjust_logits(x, **dev(c)), "f32")


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_more_biases_than_a_slice_lists_and_every_token_touched(dtype):
    native = _native()
    x, c = make(49, 2, 9001, dtype, 0, 3000, 1)
    c["bias_ids"][:600] = 7  # one token's, far apart
    check(x, c, native.adjust_logits(x, **dev(c)), dtype)
    n = 2 * 9001
    c.update(ids=np.tile(np.arange(9001, dtype=np.int32), 4), at=np.array([0, n, 2 * n], np.int32), prompt=np.array([9001, 100], np.int32),
             repetition=np.array([1.5, 2.0], np.float32), frequency=np.array([0.5, 0.1], np.float32), presence=np.array([0.0, 1.0], np.float32))
    got = native.adjust_logits(x, **dev(c))
    check(x, c, got, dtype)
    assert torch.equal(native.adjust_logits(x, **dev(c), out=x), got)


def test_no_masks_and_empty_lists():
    native = _native()
    x, _ = make(45, 3, 77, "bf16")
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    got = native.adjust_logits(x, z(0), z(4), prompt=z(3), repetition=z(3, t=torch.float32), bias_ids=z(0), bias=z(0, t=torch.float32),
                               bias_at=z(4), allowed=z(0, 3), allowed_rows=z(3))
    assert torch.equal(got, x)


def test_rows_behind_32_bit_offsets():
    native = _native()
    M, V = 17, 1 << 28
    x = torch.zeros((M, V), dtype=torch.float16, device="cuda")
    ids = torch.tensor([5, V - 1, 5], dtype=torch.int32, device="cuda")
    at = torch.zeros(M + 1, dtype=torch.int32, device="cuda")
    at[-1] = 3
    native.adjust_logits(x, ids, at, presence=torch.ones(M, device="cuda"), frequency=torch.ones(M, device="cuda"), out=x)
    assert int(torch.count_nonzero(x)) == 2
    assert float(x[-1, 5]) == -3 and float(x[-1, -1]) == -2


def test_streams_and_a_captured_step():
    native = _native()
    x, c = make(46, 9, 30011, "f32", 400, 10, 4)
    d = dev(c)
    want = native.adjust_logits(x, **d)
    torch.cuda.synchronize()
    for s in [torch.cuda.Stream() for _ in range(3)]:
        got = native.adjust_logits(x, **d, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(x)
    with torch.cuda.graph(graph):
        native.adjust_logits(x, **d, out=out)
    y, other = make(47, 9, 30011, "f32", 400, 10, 4)
    x.copy_(y)
    n = min(len(c["ids"]), len(other["ids"]))
    c["ids"][:n] = other["ids"][:n]
    d["ids"].copy_(torch.from_numpy(c["ids"]))
    graph.replay()
    torch.cuda.synchronize()
    check(x, c, out, "f32")


def test_refusals():
    native = _native()
    x, c = make(48, 3, 100, "f32", 20, 5, 3)
    d = dev(c)

    def bad(exc, logits=x, **kw):
        with pytest.raises(exc):
            native.adjust_logits(logits, **{**d, **kw})

    bad(ValueError, logits=x.cpu())
    bad(ValueError, logits=x.t())
    bad(TypeError, logits=x.double())
    bad(TypeError, ids=d["ids"].long())
    bad(ValueError, at=None)
    bad(ValueError, ids=None, at=None)
    bad(ValueError, at=d["at"][:3].clone())
    bad(ValueError, ids=d["ids"][None])
    bad(ValueError, bias=None)
    bad(TypeError, bias=d["bias"].half())
    bad(ValueError, allowed=d["allowed"][:2].clone(), allowed_rows=None)
    bad(ValueError, allowed=None)
    bad(ValueError, allowed=d["allowed"][:, :3].clone())
    bad(TypeError, frequency=d["frequency"].half())
    bad(ValueError, repetition=d["repetition"][:2].clone())
    bad(ValueError, out=torch.empty((3, 101), device="cuda"))
    bad(ValueError, out=torch.empty((3, 100), dtype=torch.float16, device="cuda"))
    bad(native.EschaError, out=torch.empty(400, device="cuda")[1:301].view(3, 100))


def _in_f32(x, ids, bias):
    """Biases added one by one in f32, in list order."""
    y = x.copy()
    for i, b in zip(ids, bias):
        if 0 <= i < len(y):
            y[i] = np.float32(y[i] + b)
    return y


@pytest.mark.parametrize("V,n,same", [(9001, 512, 512), (9001, 513, 513), (9001, 20000, 3000), (40000, 700, 1), (40000, 600, 600),
                                      (40000, 60000, 0), (100, 5000, 40)])
def test_biases_of_any_number_are_added_in_list_order(V, n, same):
    """Magnitudes far apart, so that another order of the f32 sums would show: equal bits. ``same`` of them are one token's."""
    native = _native()
    rng = np.random.default_rng(61)
    ids = rng.integers(-1, V + 1, 2 * n).astype(np.int32)
    ids[rng.permutation(n)[:same]] = 7
    bias = (rng.standard_normal(2 * n) * 10.0 ** rng.integers(-4, 5, 2 * n)).astype(np.float32)
    at = np.array([0, n, n, 2 * n], np.int32)
    x = rng.standard_normal((3, V)).astype(np.float32)
    allowed = rng.integers(-2 ** 31, 2 ** 31, (1, (V + 31) // 32)).astype(np.int32)
    d = dev(dict(bias_ids=ids, bias=bias, bias_at=at, allowed=allowed, allowed_rows=np.array([-1, 0, 0], np.int32)))
    want = np.stack([_in_f32(x[m], ids[at[m]:at[m + 1]], bias[at[m]:at[m + 1]]) for m in range(3)])
    i = np.arange(V)
    want[1:, (allowed[0].view(np.uint32)[i // 32] >> (i % 32).astype(np.uint32)) & 1 == 0] = -np.inf
    logits = torch.from_numpy(x).cuda()
    assert np.array_equal(native.adjust_logits(logits, **d).cpu().numpy(), want)
    native.adjust_logits(logits, **d, out=logits)
    assert np.array_equal(logits.cpu().numpy(), want)


def test_time_goes_by_the_number_of_biases():
    """One for every token of a row, and 512 of one token, take a time in proportion to the list: 0.77 and 0.02 ms, where a walk of
    the whole list by every token took 54 ms for the first."""
    native = _native()
    V = 152064
    x = torch.zeros((1, V), device="cuda")
    for n, ids, bound in ((V, torch.arange(V), 3.0), (512, torch.full((512,), 5), 0.25)):
        d = dict(bias_ids=ids.int().cuda(), bias=torch.ones(n, device="cuda"), bias_at=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        out = native.adjust_logits(x, **d)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            native.adjust_logits(x, **d, out=out)
        times = []
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        assert min(times) < bound, times
