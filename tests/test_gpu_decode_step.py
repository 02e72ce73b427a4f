"""The operators between a model's last block and its next token, run together as a decoder
runs them: embedding rows, the end of a block, logits by a matrix held in 4 bits, a drawn token,
which is the next step's input."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import log_sum_exp_gb300 as L  # noqa: E402


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Decoder:
    def __init__(self, V=2003, D=256, seed=0, dtype=torch.bfloat16):
        g = torch.Generator().manual_seed(seed)
        self.table = torch.randn((V, D), generator=g).to(dtype).cuda()
        self.block = (torch.randn((D, D), generator=g) * 0.05).to(dtype).cuda()
        self.weight, self.post = (torch.rand(D, generator=g).add(0.5).to(dtype).cuda() for _ in range(2))
        self.head = L.lse_quantize4((torch.randn((V, D), generator=g) * 0.1).to(dtype).cuda(), group=64)

    def step(self, ids, u, **settings):
        x = L.lse_embedding(self.table, ids, scale=0.5)
        s = L.lse_residual_norm(x, x @ self.block, self.weight, post_weight=self.post, scale=0.7)
        logits = L.lse_linear4(s.out, self.head, out_dtype=torch.float32)
        return logits, L.lse_sample(logits, u, **settings)

    def plain(self, ids):
        d = torch.float64
        x = (self.table[ids].float() * 0.5).to(self.table.dtype)
        y = (x @ self.block).to(d)
        a = y / torch.sqrt((y * y).mean(1, keepdim=True) + 1e-6) * self.post.to(d)
        h = x.to(d) + 0.7 * a
        out = (h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * self.weight.to(d)).to(self.table.dtype)
        return out.to(d) @ L.lse_dequantize4(self.head).to(d).t()


def test_steps():
    model = Decoder()
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(0, 2003, (12,), generator=g).cuda()
    for _ in range(6):
        u = torch.rand(12, generator=g).cuda()
        logits, drawn = model.step(ids, u, temperature=0.8, top_k=40, top_p=0.95)
        want = model.plain(ids)
        # bf16 rows into the matrix differ by a step where f32 and f64 round apart (2^-8 of each of
        # 256 terms, few of them), and the matrix's values are rounded to bf16 when read back.
        assert (logits.double() - want).abs().max() <= 2.0 ** -6 * want.abs().max()
        stats = L.lse_token_stats(logits, drawn.token, top_k=32)
        kept = logits.double().topk(40, 1).values / 0.8
        z = torch.logsumexp(kept, 1)
        lp = logits.double().gather(1, drawn.token[:, None])[:, 0] / 0.8 - z
        # kept by top-p: between the whole top 40 and 0.95 of it
        assert (drawn.logprob.double() >= lp - 1e-5).all() and (drawn.logprob.double() <= lp - torch.log(torch.tensor(0.95)) + 1e-5).all()
        assert (stats.logprob <= 0).all() and (drawn.token >= 0).all()
        ids = drawn.token


def test_greedy_is_the_first_alternative():
    model = Decoder(seed=2)
    ids = torch.arange(30, device="cuda")
    logits, drawn = model.step(ids, torch.zeros(30, device="cuda"), temperature=0.0)
    assert torch.equal(drawn.token, L.lse_token_stats(logits, top_k=1).top_index[:, 0])


def test_steps_in_a_graph_and_two_at_once():
    """A captured step replayed with new inputs, next to one on another stream."""
    model = Decoder(seed=3)
    ids = torch.arange(8, device="cuda")
    u = torch.full((8,), 0.37, device="cuda")
    want = model.step(ids, u, top_p=0.9)[1].token
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, got = model.step(ids, u, top_p=0.9)
    other = Decoder(seed=4)
    ids2 = torch.arange(100, 164, device="cuda")
    u2 = torch.rand(64, device="cuda")
    want2 = other.step(ids2, u2)[1].token
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    results = []
    for _ in range(20):
        graph.replay()
        with torch.cuda.stream(st):
            results.append(other.step(ids2, u2)[1].token)
    torch.cuda.synchronize()
    assert torch.equal(got.token, want) and all(torch.equal(r, want2) for r in results)
    ids.copy_(torch.arange(50, 58))
    graph.replay()
    assert torch.equal(got.token, model.step(torch.arange(50, 58, device="cuda"), u, top_p=0.9)[1].token)


def test_training_through_the_block_end():
    """Embedding, block end and token statistics differentiated together against 64 bits."""
    V, D, T = 301, 48, 40
    g = torch.Generator().manual_seed(5)
    table = torch.randn((V, D), generator=g).cuda().requires_grad_()
    out = (torch.randn((V, D), generator=g) * 0.2).cuda()
    w, p, gate = (torch.rand(D, generator=g).add(0.5).cuda().requires_grad_() for _ in range(3))
    ids, target = (torch.randint(0, V, (T,), generator=g).cuda() for _ in range(2))
    torch.backends.cuda.matmul.allow_tf32 = False

    def loss_of(embed, norm, stats):
        x = embed()
        h, n = norm(x, torch.tanh(x))
        return stats((n + 0.1 * h) @ out.to(n.dtype).t())

    loss = loss_of(lambda: L.embedding(ids, table), lambda x, y: L.residual_norm(x, y, w, p, gate, scale=0.6),
                   lambda z: -L.token_stats(z, target).logprob.mean())
    loss.backward()
    leaves = [t.detach().double().requires_grad_() for t in (table, w, p, gate)]

    def norm64(x, y):
        a = y / torch.sqrt((y * y).mean(1, keepdim=True) + 1e-6) * leaves[2]
        h = x + 0.6 * leaves[3] * a
        return h, h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * leaves[1]

    want = loss_of(lambda: leaves[0][ids], norm64,
                   lambda z: -torch.log_softmax(z, 1).gather(1, target[:, None]).mean())
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) < 1e-5
    # f32 products of 48- and 301-long sums: about 350 * 2^-24 = 2e-5 of the largest entry
    for t, r in zip((table, w, p, gate), leaves):
        assert (t.grad.double() - r.grad).abs().max() <= 1e-4 * r.grad.abs().max()
