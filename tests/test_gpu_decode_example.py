"""examples/decode_gdn.py: what it generates token by token equals what one prefill over the whole text says.

The model runs in fp32 here, so that the two ways differ by the order of fp32 sums alone: logits of size ~3 after
two layers, held to 2e-3 (their fp32 rounding is 1e-6; the operators are each held to 1e-5 of their size)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOL = 2e-3


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decode_gdn", os.path.join(ROOT, "examples", "decode_gdn.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.fixture(scope="module")
def model(example):
    return example.Model(vocab=300, width=128, dtype=torch.float32)


def prompts(B, T, seed):
    return torch.randint(0, 300, (B, T), generator=torch.Generator().manual_seed(seed)).cuda()


@torch.no_grad()
@pytest.mark.parametrize("end", [None, 7])
def test_beam_scores_are_those_of_the_whole_text(example, model, end):
    if end is not None:  # a token that is chosen now and then
        model.head[end] *= 1.5
    prompt = prompts(3, 70, 1)
    tokens, scores = example.beam_search(model, prompt, beams=4, steps=5, end=end)
    assert (scores[:, :-1] >= scores[:, 1:]).all()
    for b in range(3):
        assert len({tuple(t) for t in tokens[b].tolist()}) == 4
        for i in range(4):
            said = [t for t in tokens[b, i].tolist() if t >= 0]
            assert all(t == -1 for t in tokens[b, i, len(said):].tolist())
            assert len(said) == 5 or said[-1] == end
            logits, _ = model.prefill(torch.cat([prompt[b], torch.tensor(said, device="cuda")]).unsqueeze(0))
            logp = torch.log_softmax(logits[0, 69:69 + len(said)].double(), -1)
            whole = sum(logp[j, t].item() for j, t in enumerate(said))
            assert abs(whole - scores[b, i].item()) < 5 * TOL
    if end is not None:
        model.head[end] /= 1.5


@torch.no_grad()
def test_drafts(example, model):
    """The tree's logits are those of each path as a text; the states afterwards are those of the accepted path."""
    prompt = prompts(2, 33, 2)
    greedy, _ = example.beam_search(model, prompt, beams=1, steps=3)
    right = greedy[:, 0].long()
    wrong = (right + 1) % 300
    drafts = torch.stack([wrong[:, 0], right[:, 0], right[:, 1], wrong[:, 2], right[:, 2], right[:, 0]], dim=1)
    drafts[1, 4] = wrong[1, 2]  # the second row's tree has two tokens that are right
    parents = torch.tensor([-1, -1, 1, 2, 2, 0], dtype=torch.int32, device="cuda").expand(2, 6).contiguous()
    last, states = model.prefill(prompt)
    path, logits = example.verify_drafts(model, states, drafts, parents, last[:, -1])
    assert path.tolist() == [[1, 2, 4, -1, -1, -1], [1, 2, -1, -1, -1, -1]]
    ways = {0: [0], 1: [1], 2: [1, 2], 3: [1, 2, 3], 4: [1, 2, 4], 5: [0, 5]}
    for b in range(2):
        for t, way in ways.items():
            whole, _ = model.prefill(torch.cat([prompt[b], drafts[b, way]]).unsqueeze(0))
            assert (whole[0, -1] - logits[b, t]).abs().max() < TOL
        taken = [t for t in path[b].tolist() if t >= 0]
        _, after = model.prefill(torch.cat([prompt[b], drafts[b, taken]]).unsqueeze(0))
        for layer in range(model.layers):
            assert (after[layer][0] - states[layer][b]).abs().max() < TOL


def test_main(example, capsys):
    example.main()
    out = capsys.readouterr().out
    assert out.count("best:") == 3 and out.count("accepted:") == 3
