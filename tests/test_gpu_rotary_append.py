"""GPU checks of escha_rotary_append against its formula in 64 bits."""
import numpy as np
import pytest

import chunk_refs as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _native():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_trellis_quantized_gb300 import native

    return native


def make(seed, new, old, Hq, Hkv, d, page, dtype, source, pad=0, fused=True):
    rng = np.random.default_rng(seed)
    lens = [a + b for a, b in zip(new, old)]
    need = [-(-max(x, 0) // page) for x in lens]
    n_pages, width = sum(need) + 3, max(max(need), 1)
    table, order, p = np.full((len(lens), width), -1, np.int32), rng.permutation(n_pages), 0
    for b, c in enumerate(need):
        table[b, :c], p = order[p:p + c], p + c
    T = sum(new) + pad
    x = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hkv, d))).to(DT[source]).cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pool = lambda: torch.from_numpy(rng.standard_normal((n_pages, Hkv, page, d))).to(DT[dtype]).cuda()  # noqa: E731
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(q=q, k=k, v=v, k_pool=pool(), v_pool=pool(), table=torch.from_numpy(table).cuda(),
                at=i32(np.cumsum([0] + new).tolist()), lens=i32(lens))


def f64(t):
    return t.double().cpu().numpy()


def check(c, got, before, rotary, positions=None):
    """A turned value is x c - y s with |c|, |s| <= factor: their error (the
    frequency's 2^-53 and 2^-65 p, the angle's 2^-24 of half a turn at most, the
    functions' 2^-22) and four roundings to f32 are within 2^-20 factor (|x| +
    |y|); then half a step of the type, in fp16 2^-25 near 0."""
    dt = "f16" if c["k_pool"].dtype is torch.float16 else "bf16"
    T = c["k"].shape[0]
    at, lens, table = (f64(c[x]).astype(np.int64) for x in ("at", "lens", "table"))
    seq, pos = ref.places(at, lens, T)
    by = pos if positions is None else f64(positions)
    if rotary is None:
        turned = {x: f64(c[x]) for x in "qkv" if c[x] is not None}
        slack = {x: 0 * np.abs(y) for x, y in turned.items()}
    else:
        angle = by[:, None].astype(np.float64) * rotary.frequencies
        turned = {x: ref.rotate(f64(c[x]), angle, rotary.factor, rotary.interleaved) for x in "qk" if c[x] is not None}
        turned["v"] = f64(c["v"])
        slack = {}
        for x in turned:
            size = np.abs(f64(c[x]))
            if x != "v":
                r = rotary.rot
                one, two = ((slice(0, r, 2), slice(1, r, 2)) if rotary.interleaved else (slice(0, r // 2), slice(r // 2, r)))
                both = (size[..., one] + size[..., two]) * rotary.factor
                size = np.zeros_like(size)
                size[..., one], size[..., two] = both, both
            else:
                size = 0 * size
            slack[x] = 2.0 ** -20 * size
    tiny = 2.0 ** -25 if dt == "f16" else 0
    tol = {x: HALF[dt] * np.abs(y) + slack[x] + tiny for x, y in turned.items()}
    on = seq >= 0
    if got is not None:
        assert np.all(np.abs(f64(got)[on] - turned["q"][on]) <= tol["q"][on])
    for x, b in (("k", before[0]), ("v", before[1])):
        want, room = f64(b), np.zeros(b.shape)
        zeros = np.zeros_like(want)
        ref.append(want, zeros, turned[x], turned[x], table, at, lens)
        ref.append(room, zeros, tol[x], tol[x], table, at, lens)
        assert np.all(np.abs(f64(c[x + "_pool"]) - want) <= room)  # (what is not stored to keeps its bits)


CASES = [
    # new, old, Hq, Hkv, d, page, dtype, source, rot, interleaved, pad
    ([1], [0], 2, 2, 64, 16, "f16", "f32", 64, False, 0),
    ([1], [699], 16, 2, 256, 64, "f16", "f32", 64, False, 0),
    ([1] * 37, [(i * 31) % 90 for i in range(37)], 16, 2, 256, 64, "bf16", "f32", 64, False, 5),
    ([5, 0, 17, 1, 0], [0, 3, 15, 16, 0], 5, 1, 128, 16, "bf16", "bf16", 128, True, 3),
    ([33, 2], [100, 7], 22, 2, 64, 17, "f16", "f16", 16, True, 0),
    ([130], [5], 3, 3, 256, 1, "bf16", "f32", 256, False, 1),
    ([9, 9], [0, 1], 64, 1, 64, 128, "f16", "f32", 48, False, 0),
    ([3] * 300, [i % 7 for i in range(300)], 8, 4, 128, 4, "f16", "f16", 96, True, 0),
    ([40], [8], 4, 2, 128, 16, "bf16", "bf16", 0, False, 0),
]


@pytest.mark.parametrize("new,old,Hq,Hkv,d,page,dtype,source,rot,interleaved,pad", CASES)
@pytest.mark.parametrize("scaling", [None, {"type": "linear", "factor": 8.0}, {"type": "yarn", "factor": 4.0, "original": 64}])
def test_matches_the_formula(new, old, Hq, Hkv, d, page, dtype, source, rot, interleaved, pad, scaling):
    native = _native()
    rotary = native.Rotary(rot, base=1e4, interleaved=interleaved, scaling=scaling) if rot else None
    for fused in (True, False):
        c = make(21, new, old, Hq, Hkv, d, page, dtype, source, pad, fused)
        before = c["k_pool"].clone(), c["v_pool"].clone()
        given = torch.full((sum(new) + pad, Hq, d), 7.0, dtype=DT[dtype], device="cuda")
        got = native.rotary_append(**c, rotary=rotary, out=given)
        torch.cuda.synchronize()
        assert got is given and bool((given[sum(new):] == 7).all())
        check(c, got, before, rotary)


def test_few_and_many_tokens_give_the_same_bits():
    """Tokens are dealt out by their number; a token's outputs do not depend on it."""
    native = _native()
    rotary = native.Rotary(64)
    c = make(22, [6000], [50], 16, 2, 256, 64, "f16", "f32")
    got = native.rotary_append(**c, rotary=rotary)
    for a, b in ((0, 1), (1234, 1300), (5000, 6000)):
        part = {**c, **{x: c[x][a:b] for x in "qkv"}, "k_pool": torch.zeros_like(c["k_pool"]), "v_pool": torch.zeros_like(c["v_pool"]),
                "at": torch.tensor([0, b - a], dtype=torch.int32, device="cuda"),
                "lens": torch.tensor([50 + b], dtype=torch.int32, device="cuda")}
        assert torch.equal(native.rotary_append(**part, rotary=rotary), got[a:b])
        pos = torch.arange(50 + a, 50 + b, device="cuda")
        pg = c["table"][0][pos // 64].long()
        for x in ("k_pool", "v_pool"):
            assert torch.equal(part[x][pg, :, pos % 64], c[x][pg, :, pos % 64])


@pytest.mark.parametrize("far", [131071, 2 ** 24 + 1, 2 ** 31 - 1, -3])
def test_far_positions(far):
    """Given positions up to the largest: 64-bit angles of p f are good to 2^-22 there."""
    native = _native()
    rotary = native.Rotary(128, base=1e6)
    c = make(23, [4], [0], 2, 1, 128, 16, "f16", "f32")
    before = c["k_pool"].clone(), c["v_pool"].clone()
    positions = torch.tensor([far, 0, 7, far // 2], dtype=torch.int32, device="cuda")
    got = native.rotary_append(**c, rotary=rotary, positions=positions)
    check(c, got, before, rotary, positions)


def test_tokens_without_a_place_are_turned_and_not_stored():
    native = _native()
    rotary = native.Rotary(32)
    c = make(24, [4, 6, 3, 2], [2, 10, 0, 5], 4, 2, 64, 4, "bf16", "bf16", pad=2)
    c["table"][1, 3] = -1  # a dropped page
    c["table"][1, 2] = c["k_pool"].shape[0]  # past the pool
    c["lens"][2] = 1  # two of three tokens before the start
    c["lens"][3] = 1 << 30  # behind the table
    c["lens"][0] = -5
    before = c["k_pool"].clone(), c["v_pool"].clone()
    got = native.rotary_append(**c, rotary=rotary)
    check(c, got, before, rotary)


def test_keys_and_values_alone_and_queries_in_place():
    native = _native()
    rotary = native.Rotary(64, interleaved=True)
    c = make(25, [11, 4], [3, 0], 6, 2, 64, 8, "f16", "f16", fused=False)
    twin = {**c, "k_pool": c["k_pool"].clone(), "v_pool": c["v_pool"].clone(), "q": None}
    want = native.rotary_append(**c, rotary=rotary)
    assert native.rotary_append(**twin, rotary=rotary) is None
    assert torch.equal(twin["k_pool"], c["k_pool"]) and torch.equal(twin["v_pool"], c["v_pool"])
    got = native.rotary_append(**c, rotary=rotary, out=c["q"])
    assert got.data_ptr() == c["q"].data_ptr() and torch.equal(got, want)


def test_pools_behind_32_bit_offsets():
    native = _native()
    Hkv, page, d = 8, 64, 256
    n_pages = (1 << 32) // (Hkv * page * d) + 5
    pools = [torch.zeros((n_pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    c = make(26, [70], [10], 8, Hkv, d, page, "bf16", "f32")
    c["table"] = torch.tensor([[n_pages - 1, 3]], dtype=torch.int32, device="cuda")
    native.rotary_append(c["q"], c["k"], c["v"], *pools, c["table"], c["at"], c["lens"])
    assert torch.equal(pools[0][n_pages - 1, :, 10:], c["k"][:54].bfloat16().transpose(0, 1))
    assert torch.equal(pools[1][3, :, :16], c["v"][54:].bfloat16().transpose(0, 1))
    assert int(torch.count_nonzero(pools[0][:, :, :, 0])) == 70 * Hkv


def test_nan_and_infinity_stay_in_their_pairs():
    native = _native()
    rotary = native.Rotary(64)
    c = make(27, [6], [0], 4, 2, 128, 8, "bf16", "f32")
    want = native.rotary_append(**c, rotary=rotary).clone()
    c["q"][2, 1, 5], c["q"][3, 0, 100] = float("nan"), float("inf")
    got = native.rotary_append(**c, rotary=rotary)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[2, 1, 5] = hit[2, 1, 37] = hit[3, 0, 100] = True
    assert torch.equal(got[~hit], want[~hit])
    assert bool(got[2, 1, [5, 37]].isnan().all()) and float(got[3, 0, 100]) == float("inf")


def test_streams_and_a_captured_step():
    native = _native()
    rotary = native.Rotary(64)
    c = make(28, [1] * 9, [5 + i for i in range(9)], 8, 2, 128, 16, "f16", "f32")
    want = native.rotary_append(**c, rotary=rotary)
    torch.cuda.synchronize()
    for s in [torch.cuda.Stream() for _ in range(3)]:
        got = native.rotary_append(**c, rotary=rotary, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        native.rotary_append(**c, rotary=rotary, out=out)
    c["lens"] += 1  # lengths are read by the replay
    before = c["k_pool"].clone(), c["v_pool"].clone()
    graph.replay()
    torch.cuda.synchronize()
    check(c, out, before, rotary)


def test_refusals():
    native = _native()
    c = make(29, [5, 3], [0, 2], 4, 2, 64, 8, "f16", "f32")
    rotary = native.Rotary(32)

    def bad(exc, **kw):
        with pytest.raises(exc):
            native.rotary_append(**{**c, "rotary": rotary, **kw})

    bad(ValueError, q=c["q"].half())
    bad(ValueError, v=c["v"][:, :1])
    bad(ValueError, v=c["v"].half())
    bad(ValueError, k=c["k"].cpu())
    bad(ValueError, k=c["k"].transpose(1, 2).contiguous().transpose(1, 2))
    bad(ValueError, k=c["k"][:1].expand(8, 2, 64))
    bad(ValueError, at=c["at"][:2].clone())
    bad(TypeError, lens=c["lens"].long())
    bad(TypeError, k_pool=c["k_pool"].float(), v_pool=c["v_pool"])
    bad(ValueError, q=None, out=torch.empty_like(c["q"]))
    bad(ValueError, positions=c["at"])
    bad(ValueError, rotary=native.Rotary(32, device="cpu"))
    bad(native.EschaError, rotary=native.Rotary(128))
    bad(native.EschaError, v_pool=c["k_pool"])
    bad(native.EschaError, k_pool=c["k_pool"].bfloat16(), v_pool=c["v_pool"].bfloat16(), q=c["q"].half(), k=c["k"].half(), v=c["v"].half())
    odd = torch.zeros((8, 2 * 64 + 1), device="cuda")
    bad(native.EschaError, k=odd[:, :128].unflatten(1, (2, 64)))
