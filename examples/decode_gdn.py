"""Generating from a small model of gated delta rule layers, or of linear attention: prefill, sampling, beam search,
drafted trees.

The model is random (there is nothing to learn here); what it shows is how the calls fit together.  One pool of
states per layer, a slot per hypothesis:

    prefill      chunk_gated_delta_rule (chunk_linear_attention) leaves a state per prompt
    sampling     sample_tokens draws the next token of every row, recurrent_gated_delta_rule
                 (recurrent_linear_attention) moves the row's state by it
    beam search  recurrent_gated_delta_rule moves every beam by a token, beam_search_step selects,
                 reorder_states lets the states follow the selection
    drafts       tree_gated_delta_rule answers a tree of drafted tokens without touching the states,
                 recurrent_gated_delta_rule(None, ..., token_indices=path) moves them along what was accepted

    python examples/decode_gdn.py            # needs a GPU
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_50_gb300 as gdn  # noqa: E402


class Model:
    """Embedding, layers x += Wo GDN(Wq x, Wk x, Wv x, gates), logits from the normalised x."""

    def __init__(self, vocab=1000, width=256, layers=2, Hq=2, Hv=4, K=128, V=128, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, device="cuda", generator=gen) * shape[-1] ** -0.5).to(dtype)

        self.Hq, self.Hv, self.K, self.V, self.layers = Hq, Hv, K, V, layers
        self.embed = torch.randn(vocab, width, device="cuda", generator=gen).to(dtype)
        # one projection per layer: q, k, v and the two gates of a token side by side
        self.w_in = [weight(2 * Hq * K + Hv * V + 2 * Hv, width) for _ in range(layers)]
        self.w_out = [weight(width, Hv * V) for _ in range(layers)]
        self.head = weight(vocab, width) * 3

    def inputs(self, layer, x):
        """q, k, v, g, beta of a layer from x [B, T, width]; q and k are normalised."""
        B, T, _ = x.shape
        Hq, Hv, K, V = self.Hq, self.Hv, self.K, self.V
        x = torch.nn.functional.rms_norm(x.float(), x.shape[-1:]).to(x.dtype)
        qk, v, g, beta = (x @ self.w_in[layer].t()).split([2 * Hq * K, Hv * V, Hv, Hv], dim=-1)
        q, k = torch.nn.functional.normalize(qk.float().view(B, T, 2 * Hq, K), dim=-1).to(x.dtype).split(Hq, dim=2)
        return q, k, v.view(B, T, Hv, V), -torch.nn.functional.softplus(g.float()), torch.sigmoid(beta.float())

    def forward(self, tokens, mix):
        """Logits [B, T, vocab] of tokens [B, T]; mix(layer, q, k, v, g, beta) is the layer's mixing along the tokens."""
        x = self.embed[tokens]
        for layer in range(self.layers):
            o = mix(layer, *self.inputs(layer, x))
            x = x + o.flatten(2) @ self.w_out[layer].t()
        x = torch.nn.functional.rms_norm(x.float(), x.shape[-1:]).to(x.dtype)
        return x @ self.head.t()

    def through(self, *inputs):
        """(o, final state) of a layer's whole text."""
        return gdn.chunk_gated_delta_rule(*inputs, output_final_state=True)

    def step(self, state, *inputs):
        """o of a token or a few behind the states, which are moved."""
        return gdn.recurrent_gated_delta_rule(*inputs, state)

    def prefill(self, tokens):
        """(logits of all tokens, a state per prompt and layer [B, Hv, K, V])."""
        states = []

        def mix(layer, *inputs):
            o, state = self.through(*inputs)
            states.append(state)
            return o

        return self.forward(tokens, mix), states

    def further(self, tokens, states):
        """Logits [B, T, vocab] of tokens [B, T] behind the states, which are moved."""
        return self.forward(tokens, lambda layer, *inputs: self.step(states[layer], *inputs))


class LinearModel(Model):
    """The same with linear attention: head i of n forgets by 1 - 2^(-1 - 8 i / n) a token."""

    def inputs(self, layer, x):
        q, k, v, _, _ = super().inputs(layer, x)
        heads = torch.arange(self.Hv, device="cuda", dtype=torch.float64)
        return q, k, v, torch.log1p(-torch.exp2(-1 - 8 * heads / self.Hv)).float()

    def through(self, *inputs):
        return gdn.chunk_linear_attention(*inputs, output_final_state=True)

    def step(self, state, *inputs):
        return gdn.recurrent_linear_attention(*inputs, state)


@torch.no_grad()
def generate(model, prompt, steps=8, copies=1, seed=0, **filters):
    """`copies` drawn continuations of every prompt [B, T]: (tokens [B, copies, steps], the logarithms of their shares,
    the same).  filters: what sample_tokens takes, temperature, top_k, top_p, min_p, mask."""
    B = prompt.shape[0]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    logits, states = model.prefill(prompt)
    states = [s.repeat_interleave(copies, 0) for s in states]  # slot b * copies + i
    logits = logits[:, -1].repeat_interleave(copies, 0)
    tokens, shares = [], []
    for step in range(steps):
        if step:
            logits = model.further(tokens[-1].unsqueeze(1), states)[:, -1]
        token, share = gdn.sample_tokens(logits, torch.rand(B * copies, device="cuda", generator=gen), **filters)
        tokens.append(token)
        shares.append(share)
    return torch.stack(tokens, 1).view(B, copies, steps), torch.stack(shares, 1).view(B, copies, steps)


@torch.no_grad()
def beam_search(model, prompt, beams=4, steps=8, end=None):
    """The best `beams` continuations of every prompt [B, T]: (tokens [B, beams, steps], scores [B, beams]).  A
    hypothesis that has chosen the token `end` is carried along; its further tokens are -1."""
    B = prompt.shape[0]
    logits, states = model.prefill(prompt)
    states = [s.repeat_interleave(beams, 0) for s in states]  # slot b * beams + i
    scores = torch.full((B, beams), float("-inf"), device="cuda")
    scores[:, 0] = 0  # at first every search has one beam
    finished = torch.zeros(B, beams, dtype=torch.bool, device="cuda")
    logits = logits[:, -1:].expand(B, beams, -1)
    chosen = torch.empty(B, beams, 0, dtype=torch.int32, device="cuda")
    for step in range(steps):
        scores, tokens, parents = gdn.beam_search_step(logits, scores, finished=finished)
        gdn.reorder_states(states, parents)
        at = parents.long()
        chosen = torch.cat([chosen.gather(1, at.unsqueeze(-1).expand(-1, -1, step)), tokens.unsqueeze(-1)], dim=-1)
        finished = finished.gather(1, at) | (tokens == (-2 if end is None else end))
        if step + 1 < steps:  # finished beams run along: what they would say is not looked at
            logits = model.further(tokens.clamp(min=0).view(B * beams, 1), states).view(B, beams, -1)
    return chosen, scores


@torch.no_grad()
def verify_drafts(model, states, drafts, parents, last_logits):
    """Answers a drafted tree per row and moves the states along the longest path that the model would have taken
    itself.  drafts, parents [B, T] as tree_gated_delta_rule takes them; last_logits [B, vocab] what the model said
    after the token before the tree.  Returns (path [B, T], -1 past its end; logits [B, T, vocab] of the nodes)."""
    seen = []

    def mix(layer, *inputs):
        seen.append(inputs)
        return gdn.tree_gated_delta_rule(*inputs, parents, states[layer])

    logits = model.forward(drafts, mix)
    said, before = logits.argmax(-1).tolist(), last_logits.argmax(-1).tolist()
    path = torch.full(drafts.shape, -1, dtype=torch.int32)
    for b, (row, up) in enumerate(zip(drafts.tolist(), parents.tolist())):
        at, want, length = -1, before[b], 0
        for t in range(len(row)):  # parents come before their children
            if up[t] == at and row[t] == want:
                path[b, length], at, want, length = t, t, said[b][t], length + 1
    path = path.cuda()
    for layer, (_, k, v, g, beta) in enumerate(seen):
        gdn.recurrent_gated_delta_rule(None, k, v, g, beta, states[layer], token_indices=path)
    return path, logits


def main():
    torch.manual_seed(0)
    model = Model()
    prompt = torch.randint(0, 1000, (3, 40), device="cuda")
    tokens, scores = beam_search(model, prompt, beams=4, steps=6)
    for b in range(3):
        print("prompt", b, "best:", tokens[b, 0].tolist(), "score %.3f" % scores[b, 0].item())
    for kind in (model, LinearModel()):
        tokens, shares = generate(kind, prompt, steps=6, temperature=0.8, top_k=50, top_p=0.95)
        print(type(kind).__name__, "draws:", tokens[0, 0].tolist(), "logarithm of its share %.3f" % shares[0, 0].sum().item())
    # drafts for every row: the right next tokens in one branch, wrong ones beside it
    greedy, _ = beam_search(model, prompt, beams=1, steps=3)
    logits, states = model.prefill(prompt)
    right = greedy[:, 0].long()
    wrong = (right + 1) % 1000
    drafts = torch.stack([wrong[:, 0], right[:, 0], right[:, 1], wrong[:, 2], right[:, 2]], dim=1)
    parents = torch.tensor([-1, -1, 1, 2, 2], dtype=torch.int32, device="cuda").expand(3, 5).contiguous()
    path, _ = verify_drafts(model, states, drafts, parents, logits[:, -1])
    for b in range(3):
        taken = [t for t in path[b].tolist() if t >= 0]
        print("prompt", b, "drafts accepted:", drafts[b, taken].tolist(), "of", drafts[b].tolist())


if __name__ == "__main__":
    main()
