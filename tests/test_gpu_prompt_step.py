"""A prompt's way through one attention layer and the head, as a user runs it:
the int8 projection's fused f32 output is rotated and appended, a chunk attends
over the cache, the MoE block follows, then the int8 head, the adjusted logits
and their log probabilities. Each operator's output is held to its formula on
the inputs it got in the run; a prompt at once, in parts, and token by token
reach the same cache."""
import numpy as np
import pytest

import chunk_refs as ref
import mixer_refs
from escha_synth import gen

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, DIM, PAGE, VOCAB = 512, 8, 2, 64, 16, 5003
EPS = 2.0 ** -11


class Model:
    def __init__(self, native, seed, slots, room):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.native = native

        def int8(n, k):
            w = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
            return w, torch.rand(n, generator=g, device="cuda") * 2e-3 / k ** 0.5 + 1e-4

        self.block = native.MoeBlock(gen.moe_layer(53, hidden=HIDDEN, inter=128, n_experts=16), topk=4)
        self.qkv, self.o, self.head = int8((HEADS + 2 * KV) * DIM, HIDDEN), int8(HIDDEN, HEADS * DIM), int8(VOCAB, HIDDEN)
        self.rotary = native.Rotary(32, base=1e4, scaling={"type": "yarn", "factor": 2.0, "original": 128})
        pages = slots * room
        self.k = torch.zeros(pages, KV, PAGE, DIM, dtype=torch.float16, device="cuda")
        self.v = torch.zeros_like(self.k)
        order = torch.from_numpy(np.random.default_rng(seed).permutation(pages).astype(np.int32)).cuda()
        self.table = order.view(slots, room).contiguous()
        self.embed = torch.randn(VOCAB, HIDDEN, generator=g, device="cuda")
        self.seen = torch.randint(0, VOCAB, (40,), generator=g, device="cuda", dtype=torch.int32)

    def __call__(self, ids, new, lens):
        """ids of all sequences' new tokens, how many are each's, and the lengths with them."""
        n, T, seen = self.native, ids.shape[0], {}
        i32 = lambda a: torch.tensor(a, dtype=torch.int32).to("cuda", non_blocking=True)  # noqa: E731
        at, lens = (new, lens) if isinstance(new, torch.Tensor) else (i32([0] + np.cumsum(new).tolist()), i32(lens))
        h = self.embed[ids.long()].clone()
        qkv = n.int8_w8a16_matvec(*self.qkv, n.residual_rmsnorm(h)).view(T, HEADS + 2 * KV, DIM)
        q = n.rotary_append(qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:], self.k, self.v, self.table, at, lens,
                            rotary=self.rotary)
        out, lse = n.chunk_attention(q, self.k, self.v, self.table, at, lens)
        x = torch.empty(T, HIDDEN, dtype=torch.float16, device="cuda")
        moe, _, _ = self.block.resid(h, n.int8_w8a16_matvec(*self.o, out.view(T, -1)), x)
        n.residual_add(h, moe / 64)
        logits = n.int8_w8a16_matvec(*self.head, n.residual_rmsnorm(h))
        spans = 40 * (torch.arange(T + 1, dtype=torch.int32, device="cuda") > 0).int()  # the first row has a history, the others none
        ones = torch.ones(T, device="cuda")
        adjusted = n.adjust_logits(logits, self.seen, spans, repetition=1.3 * ones, frequency=0.1 * ones, presence=0.2 * ones)
        lp = n.token_logprobs(adjusted, ids, top=5)
        seen.update(qkv=qkv, q=q, out=out, lse=lse, logits=logits, adjusted=adjusted, lp=lp, at=at, lens=lens)
        return seen


def f64(t):
    return t.double().cpu().numpy()


def check(m, s, ids):
    T = len(ids)
    at, lens, table = f64(s["at"]).astype(int), f64(s["lens"]).astype(int), m.table.cpu().numpy()
    seq, pos = ref.places(at, lens, T)
    x = f64(s["qkv"])
    turned = ref.rotate(x[:, :HEADS + KV], pos[:, None] * m.rotary.frequencies, m.rotary.factor, False)
    tol = EPS * np.abs(turned) + 2.0 ** -19 * np.abs(x[:, :HEADS + KV]).max() + 2.0 ** -25
    k = f64(m.k)
    place = table[seq, pos // PAGE], slice(None), pos % PAGE
    assert np.all(np.abs(f64(s["q"]) - turned[:, :HEADS]) <= tol[:, :HEADS])
    assert np.all(np.abs(k[place] - turned[:, HEADS:]) <= tol[:, HEADS:])
    assert torch.equal(m.v[place[0], :, place[2]], s["qkv"][:, HEADS + KV:].half())
    want, want_lse, mass, reach, most = ref.chunk_attention(f64(s["q"]), k, f64(m.v), table, at, lens, DIM ** -0.5)
    err = (DIM + 4) * 2.0 ** -24 * reach
    tol = EPS * np.abs(want) + (EPS * (1 + EPS) + 2 * err[..., None] + 2.0 ** -15) * mass + 2.0 ** -25 + 2.0 ** -36 * most[..., None]
    assert np.all(np.abs(f64(s["out"]) - want) <= tol)
    assert np.all(np.abs(f64(s["lse"]) - want_lse) <= err + 2.0 ** -20 + 2.0 ** -22 * np.abs(want_lse))
    spans = np.full(T + 1, 40)
    spans[0] = 0
    want = ref.adjust_logits(f64(s["logits"]), m.seen.cpu().numpy(), spans, None, np.full(T, np.float32(1.3)), np.full(T, np.float32(0.1)),
                             np.full(T, np.float32(0.2)), None, None, None, None, None)
    assert np.all(np.abs(f64(s["adjusted"]) - want) <= 2.0 ** -21 * (1.3 * np.abs(f64(s["logits"])) + 8))
    want = mixer_refs.logprobs(f64(s["adjusted"]), ids.cpu().numpy()[:, None], 5)
    assert np.array_equal(s["lp"]["top_ids"].cpu().numpy(), want["top_ids"])
    assert np.all(np.abs(f64(s["lp"]["logprobs"]) - want["logprobs"][:, 0]) <= 2.0 ** -17 + 2.0 ** -22 * np.abs(want["logprobs"][:, 0]))


def _native():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_trellis_quantized_gb300 import native

    return native


@pytest.mark.parametrize("steps", [[[37]], [[20, 1, 0], [3, 50, 7], [1, 1, 1]], [[5] * 12, [1] * 12]])
def test_chunks_of_ragged_prompts(steps):
    native = _native()
    m = Model(native, 71, len(steps[0]), 8)
    lens, g = [0] * len(steps[0]), torch.Generator(device="cuda").manual_seed(72)
    for new in steps:
        lens = [a + b for a, b in zip(lens, new)]
        ids = torch.randint(0, VOCAB, (sum(new),), generator=g, device="cuda", dtype=torch.int32)
        s = m(ids, new, lens)
        torch.cuda.synchronize()
        check(m, s, ids)


def test_a_prompt_at_once_in_parts_and_token_by_token():
    """The cache is written from the projection's outputs alone here, so that all three ways hold the same bits but for the
    projection's own (16 tokens and more go through the tensor cores); a decode step's attention agrees with the chunk's."""
    native = _native()
    ids = torch.randint(0, VOCAB, (90,), generator=torch.Generator(device="cuda").manual_seed(73), device="cuda", dtype=torch.int32)
    whole = Model(native, 74, 1, 6)
    a = whole(ids, [90], [90])
    for parts in ([40, 50], [1] * 90):
        m, done = Model(native, 74, 1, 6), 0
        for p in parts:
            s = m(ids[done:done + p].clone(), [p], [done + p])
            done += p
        for x, y in ((m.k, whole.k), (m.v, whole.v)):
            assert float((x.float() - y.float()).abs().max()) <= 2.0 ** -9 * float(y.float().abs().max())
        assert float((s["out"][-1].float() - a["out"][-1].float()).abs().max()) <= 2.0 ** -7 * float(whole.v.float().abs().max())
    q = a["q"][89:].contiguous()
    out, lse = native.paged_attention(q, whole.k, whole.v, whole.table, torch.tensor([90], dtype=torch.int32, device="cuda"))
    assert float((lse - a["lse"][89:]).abs().max()) <= 2.0 ** -16
    assert float((out.float() - a["out"][89:].float()).abs().max()) <= 4 * EPS * float(whole.v.float().abs().max())


def test_a_captured_step_gives_the_same_bits():
    native = _native()
    a, b = Model(native, 75, 3, 4), Model(native, 75, 3, 4)
    ids = torch.randint(0, VOCAB, (20,), generator=torch.Generator(device="cuda").manual_seed(76), device="cuda", dtype=torch.int32)
    at = torch.tensor([0, 7, 8, 20], dtype=torch.int32, device="cuda")
    lens = torch.tensor([30, 9, 12], dtype=torch.int32, device="cuda")
    b(ids, at, lens)  # warm
    b = Model(native, 75, 3, 4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            seen = b(ids, at, lens)
    for step in range(2):
        want = a(ids, at, lens)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and torch.equal(want["out"], seen["out"])
        assert torch.equal(want["adjusted"], seen["adjusted"])
        assert all(torch.equal(want["lp"][k], seen["lp"][k]) for k in want["lp"])
        lens += 1
        ids.copy_((ids * 7 + 1) % VOCAB)
