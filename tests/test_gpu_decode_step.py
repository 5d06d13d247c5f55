"""One decode step of a hybrid layer pair and its head, as a user runs it: a
delta-rule mixer and its MoE block, an attention mixer over the paged cache and
its MoE block, then the int8 head and the log probabilities. Every new
operator's output is held to its formula on the inputs it got in the run."""
import numpy as np
import pytest

import mixer_refs as ref
from escha_synth import gen

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, DIM, PAGE, DK, DV, DH = 512, 8, 2, 64, 16, 64, 64, 4


class Step:
    """Weights, caches and buffers of the two layers for B slots."""

    def __init__(self, native, B, lens, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.native, self.B = native, B

        def int8(n, k):
            w = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
            return w, torch.rand(n, generator=g, device="cuda") * 2e-3 / k ** 0.5 + 1e-4

        self.blocks = [native.MoeBlock(gen.moe_layer(s, hidden=HIDDEN, inter=128, n_experts=16), topk=4) for s in (51, 52)]
        self.wq, self.wk, self.wv = int8(DH * DK, HIDDEN), int8(DH * DK, HIDDEN), int8(DH * DV, HIDDEN)
        self.wo = int8(HIDDEN, DH * DV)
        self.aq, self.ak, self.av = int8(HEADS * DIM, HIDDEN), int8(KV * DIM, HIDDEN), int8(KV * DIM, HIDDEN)
        self.ao = int8(HIDDEN, HEADS * DIM)
        self.head = int8(5003, HIDDEN)
        self.g = -torch.rand(B, DH, generator=g, device="cuda") * 0.3
        self.beta = torch.rand(B, DH, generator=g, device="cuda")
        self.state = torch.randn(B, DH, DK, DV, generator=g, device="cuda") * 0.1
        self.at = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        need = [-(-n // PAGE) for n in lens]
        pages = sum(need)
        self.k = torch.randn(pages, KV, PAGE, DIM, generator=g, device="cuda").half()
        self.v = torch.randn(pages, KV, PAGE, DIM, generator=g, device="cuda").half()
        table = np.full((B, max(need)), -1, np.int32)
        order, p = np.random.default_rng(seed).permutation(pages), 0
        for b, n in enumerate(need):
            table[b, :n], p = order[p:p + n], p + n
        self.table = torch.from_numpy(table).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.h = torch.randn(B, HIDDEN, generator=g, device="cuda")
        self.ids = torch.randint(0, 5003, (B,), generator=g, device="cuda", dtype=torch.int32)

    def linear(self, w, x):
        return self.native.int8_w8a16_matvec(w[0], w[1], x)

    def moe(self, i, mixed):
        x = torch.empty(self.B, HIDDEN, dtype=torch.float16, device="cuda")
        out, _, _ = self.blocks[i].resid(self.h, mixed, x)
        self.native.residual_add(self.h, out / 64)  # random experts' outputs are large

    def __call__(self):
        n, B, seen = self.native, self.B, {}
        x = n.residual_rmsnorm(self.h)
        q, k, v = (self.linear(w, x).half().view(B, DH, d) for w, d in ((self.wq, DK), (self.wk, DK), (self.wv, DV)))
        seen["delta"] = (q, k, v, self.state.clone())
        seen["delta_out"] = n.delta_rule(q, k, v, self.g, self.beta, self.state, self.at)
        self.moe(0, self.linear(self.wo, seen["delta_out"].view(B, -1)))
        x = n.residual_rmsnorm(self.h)
        q, k, v = (self.linear(w, x).half().view(B, hh, DIM) for w, hh in ((self.aq, HEADS), (self.ak, KV), (self.av, KV)))
        out, lse = n.paged_attention(q, self.k, self.v, self.table, self.lens, k_new=k, v_new=v)
        seen["attention"] = (q, k, v, out, lse)
        self.moe(1, self.linear(self.ao, out.view(B, -1)))
        seen["logits"] = self.linear(self.head, n.residual_rmsnorm(self.h))
        seen["lp"] = n.token_logprobs(seen["logits"], self.ids, top=5)
        return seen


def _check(s, seen):
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    q, k, v, before = seen["delta"]
    want, state = ref.delta_rule(f64(q), f64(k), f64(v), f64(s.g), f64(s.beta), f64(before), s.at.cpu().numpy(), DK ** -0.5, 1e-6)
    # one token: sums of DK products in f32, sizes as in the operator's own tests
    tol = 2.0 ** -20 * np.sqrt(DK * 2)
    assert np.linalg.norm(f64(s.state) - state) <= tol * np.linalg.norm(state)
    assert np.all(np.abs(f64(seen["delta_out"]) - want) <= ref.HALF["f16"] * np.abs(want) + tol * np.abs(want).max() + 2.0 ** -25)
    q, k, v, out, lse = seen["attention"]
    for b, n in enumerate(s.lens.tolist()):
        assert torch.equal(s.k[s.table[b, (n - 1) // PAGE], :, (n - 1) % PAGE], k[b])
        assert torch.equal(s.v[s.table[b, (n - 1) // PAGE], :, (n - 1) % PAGE], v[b])
    want, want_lse, mass, reach = ref.attention(f64(q), f64(s.k), f64(s.v), s.table.cpu().numpy(), s.lens.cpu().numpy(), DIM ** -0.5)
    err = (DIM + 4) * 2.0 ** -24 * reach
    assert np.all(np.abs(f64(out) - want) <= ref.HALF["f16"] * np.abs(want) + (2 * err[..., None] + 2.0 ** -15) * mass + 2.0 ** -25)
    assert np.all(np.abs(f64(lse) - want_lse) <= err + 2.0 ** -20 + 2.0 ** -22 * np.abs(want_lse))
    want = ref.logprobs(f64(seen["logits"]), s.ids.cpu().numpy()[:, None], 5)
    assert np.array_equal(seen["lp"]["top_ids"].cpu().numpy(), want["top_ids"])
    for key in ("lse", "entropy", "top_logprobs"):
        assert np.all(np.abs(f64(seen["lp"][key]) - want[key]) <= 2.0 ** -17 + 2.0 ** -22 * np.abs(want[key])), key
    assert np.all(np.abs(f64(seen["lp"]["logprobs"]) - want["logprobs"][:, 0]) <= 2.0 ** -17 + 2.0 ** -22 * np.abs(want["logprobs"][:, 0]))


@pytest.mark.parametrize("lens", [[37], [1, 64, 65, 200], [5] * 24])
def test_a_decode_step(lens):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_trellis_quantized_gb300 import native

    s = Step(native, len(lens), lens, 61)
    for _ in range(2):  # a second token over the first one's state (its key overwrites the last position)
        seen = s()
        torch.cuda.synchronize()
        _check(s, seen)


def test_a_captured_step_gives_the_same_bits():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_trellis_quantized_gb300 import native

    a, b = (Step(native, 3, [37, 16, 129], 62) for _ in range(2))
    b()  # warm: the grouped path's stream, kernels loaded
    b = Step(native, 3, [37, 16, 129], 62)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            seen = b()
    for _ in range(2):
        want = a()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.h, b.h) and torch.equal(a.state, b.state) and torch.equal(a.k, b.k)
        assert torch.equal(want["logits"], seen["logits"])
        assert all(torch.equal(want["lp"][k], seen["lp"][k]) for k in want["lp"])
