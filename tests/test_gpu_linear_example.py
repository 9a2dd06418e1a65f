"""examples/decode_gdn.py: prompt, states, drawn tokens and steps together say what one pass over the whole text says, for
both kinds of layers; beams over linear attention too; and a model of linear attention has the gradients of its formula.

The models run in fp32, so that the ways differ by the order of fp32 sums alone, as in test_gpu_decode_example.py."""
import pytest
import torch

from test_gpu_decode_example import TOL, example, prompts  # noqa: F401  (example is a fixture)

pytestmark = pytest.mark.gpu


@torch.no_grad()
@pytest.mark.parametrize("kind", ["Model", "LinearModel"])
@pytest.mark.parametrize("heat", [1.0, 0.6])
def test_shares_are_those_of_the_whole_text(example, kind, heat):  # noqa: F811
    model = getattr(example, kind)(vocab=300, width=128, dtype=torch.float32)
    prompt = prompts(3, 70, 1)
    tokens, shares = example.generate(model, prompt, steps=6, copies=2, seed=3, temperature=heat)
    assert tokens.shape == (3, 2, 6) and len({tuple(t) for t in tokens.flatten(0, 1).tolist()}) > 1
    for b in range(3):
        for i in range(2):
            logits, _ = model.prefill(torch.cat([prompt[b], tokens[b, i].long()]).unsqueeze(0))
            logp = torch.log_softmax(logits[0, 69:75].double() / heat, -1)
            assert (logp.gather(1, tokens[b, i].long().unsqueeze(1))[:, 0] - shares[b, i]).abs().max() < 2 * TOL / heat


@torch.no_grad()
def test_one_choice_is_the_largest(example):  # noqa: F811
    """top_k = 1, and a mask that forbids what is largest."""
    model = example.LinearModel(vocab=300, width=128, dtype=torch.float32)
    prompt = prompts(4, 33, 2)
    tokens, shares = example.generate(model, prompt, steps=4, top_k=1)
    greedy, _ = example.generate(model, prompt, steps=4, temperature=0.0)
    assert torch.equal(tokens, greedy) and (shares == 0).all()
    mask = torch.ones(1, 300, dtype=torch.bool, device="cuda")
    mask[0, tokens.flatten().long()] = False
    others, _ = example.generate(model, prompt, steps=4, top_p=0.9, mask=mask)
    assert not set(others.flatten().tolist()) & set(tokens.flatten().tolist())


@torch.no_grad()
def test_beams_over_linear_attention(example):  # noqa: F811
    model = example.LinearModel(vocab=300, width=128, dtype=torch.float32)
    prompt = prompts(2, 70, 4)
    tokens, scores = example.beam_search(model, prompt, beams=3, steps=4)
    for b in range(2):
        for i in range(3):
            logits, _ = model.prefill(torch.cat([prompt[b], tokens[b, i].long()]).unsqueeze(0))
            logp = torch.log_softmax(logits[0, 69:73].double(), -1).gather(1, tokens[b, i].long().unsqueeze(1))
            assert abs(logp.sum().item() - scores[b, i].item()) < 5 * TOL


def test_gradients(example):  # noqa: F811
    """Through two layers of the model, against the same model with each layer's sums written out in 64 bits."""
    model = example.LinearModel(vocab=300, width=128, dtype=torch.float32)
    text = prompts(2, 90, 5)
    weights = [w.requires_grad_() for w in model.w_in + model.w_out]

    def plain(layer, q, k, v, g):
        G, T = v.shape[2] // q.shape[2], q.shape[1]
        q, k, v = (t.double() for t in (q.repeat_interleave(G, 2), k.repeat_interleave(G, 2), v))
        age = torch.arange(T, device="cuda").unsqueeze(1) - torch.arange(T, device="cuda")
        decay = torch.exp(age.clamp(min=0) * g.double()[:, None, None]).tril()
        a = torch.einsum("bihk,bjhk->bhij", q, k) * decay * q.shape[-1] ** -0.5
        return torch.einsum("bhij,bjhv->bihv", a, v).float()

    def loss(mix):
        logits = model.forward(text, mix)
        return torch.nn.functional.cross_entropy(logits[:, :-1].flatten(0, 1), text[:, 1:].flatten())

    ours = torch.autograd.grad(loss(lambda layer, *x: model.through(*x)[0]), weights)
    want = torch.autograd.grad(loss(plain), weights)
    for a, b in zip(ours, want):
        assert (a - b).abs().max() <= TOL * b.abs().max()
