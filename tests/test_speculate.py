"""The speculative decoding example: its host side, and decoding with trees of
drafts against decoding token by token."""
import pytest
import torch

from block_scaled_fp4_softmax_gb300 import speculate as S


def test_lookup_builds_a_tree():
    tokens, parents = S.lookup([7, 1, 2, 3, 7, 1, 4, 7, 1, 2, 5, 7], depth=3)
    assert tokens[0] == 7 and parents[0] == -1 and len(tokens) == len(parents)
    assert all(p < i for i, p in enumerate(parents))
    paths = set()
    for i in range(1, len(tokens)):
        path, at = [], i
        while at > 0:
            path.append(tokens[at])
            at = parents[at]
        paths.add(tuple(reversed(path)))
    # what followed the latest three sevens: 1 2 5, 1 4 7 and 1 2 3, each prefix once
    assert paths == {(1,), (1, 2), (1, 2, 5), (1, 4), (1, 4, 7), (1, 2, 3)}
    assert len(tokens) == 1 + len(paths)
    assert S.lookup([3]) == ([3], [-1])
    assert S.lookup([3, 4]) == ([4], [-1])


def test_ancestors_and_accept():
    parents = [-1, 0, 0, 1, 1, 3]
    bits, depth = S.ancestors(parents)
    assert bits == [0b1, 0b11, 0b101, 0b1011, 0b10011, 0b101011]
    assert depth == [0, 1, 1, 2, 2, 3]
    tokens = [9, 1, 2, 3, 4, 5]
    assert S.accept(tokens, parents, [1, 4, 0, 0, 8, 0]) == ([0, 1, 4], 8)
    assert S.accept(tokens, parents, [6, 0, 0, 0, 0, 0]) == ([0], 6)
    assert S.accept(tokens, parents, [1, 3, 0, 5, 0, 7]) == ([0, 1, 3, 5], 7)


# All experts are selected, so that no near-tie of the router can part the two ways.
WHOLE = dict(experts=4, top_k=4)


@pytest.mark.gpu
@pytest.mark.parametrize("layers", [1, 2])
def test_trees_decode_what_single_tokens_decode(layers):
    """Trees that hold the right continuation among wrong branches: the tokens and
    the logits are those of plain decoding.  A layer rounds nine times to BF16
    (input, q/k/v, rotated q, weights, attention, projection, experts' input, and the
    two projections' sums), each off by at most 2^-8, and so does the other
    way; the head adds two.  Taken as independent: sqrt(2 (9 layers + 2)) 2^-8 of the norm."""
    cfg = S.Config(layers=layers, budget=256, slack=64, **WHOLE)
    g = torch.Generator().manual_seed(5)
    prompts = [torch.randint(cfg.vocab, (n,), generator=g).tolist() for n in (1, 70, 9)]
    count = 40
    plain = S.Decoder(cfg, 3, seed=11)
    at = [list(p) for p in prompts]
    for k in range(0, 69, cfg.most):
        plain.prefill([p[:-1][k:k + cfg.most] for p in prompts])
    logits = [[] for _ in prompts]
    for _ in range(count + 8):
        took, of = plain.step([([t[-1]], [-1]) for t in at])
        for b in range(3):
            at[b] += took[b]
            logits[b].append(of[b])
    plain.check()
    logits = [torch.cat(x) for x in logits]

    drafted = S.Decoder(cfg, 3, seed=11)
    for k in range(0, 69, cfg.most):
        drafted.prefill([p[:-1][k:k + cfg.most] for p in prompts])
    text = [list(p) for p in prompts]
    bound = (2 * (9 * layers + 2)) ** 0.5 * 2.0 ** -8
    steps = 0
    while min(len(t) - len(p) for t, p in zip(text, prompts)) < count:
        trees = []
        for b, t in enumerate(text):
            right = at[b][len(t):len(t) + 3]
            wrong = [(x + 1) % cfg.vocab for x in right]
            # root, a wrong branch, the right one with a wrong sibling at each step
            tokens, parents, last = [t[-1]], [-1], 0
            for r, w in zip(right, wrong):
                tokens += [w, r]
                parents += [last, last]
                last = len(tokens) - 1
            trees.append((tokens, parents))
        took, of = drafted.step(trees)
        steps += 1
        for b in range(3):
            done = len(text[b]) - len(prompts[b])
            want = logits[b][done:done + len(took[b])]
            n = min(len(want), len(took[b]))
            got = of[b][:n]
            err = ((got - want[:n]).norm(dim=1) / want[:n].norm(dim=1)).max().item() if n else 0.0
            assert err <= bound, (steps, b, err, bound)
            text[b] += took[b]
    drafted.check()
    assert steps <= count // 3  # most steps take the three drafts and a fourth token
    for b in range(3):
        n = min(len(text[b]), len(at[b]))
        # a near-tie of the logits may part the two ways; it would have shown above
        assert text[b][:n] == at[b][:n]


@pytest.mark.gpu
def test_example_keeps_its_budget():
    cfg = S.Config()
    g = torch.Generator().manual_seed(3)
    prompts = [torch.randint(cfg.vocab, (n,), generator=g).tolist() for n in (1, 150, 33, 2)]
    decoder = S.Decoder(cfg, 4, seed=3)
    text, steps = S.generate(decoder, prompts, 160)
    assert all(len(t) - len(p) >= 160 for t, p in zip(text, prompts))
    assert steps <= max(len(t) - len(p) for t, p in zip(text, prompts))
    for b, t in enumerate(text):
        n = decoder.lens[b]
        assert n < cfg.budget + cfg.slack and decoder.next_pos[b] == len(t) - 1
        for layer in decoder.layers:
            for h in range(cfg.kv_heads):
                pos = layer.slot_pos[b, h, :n].tolist()
                assert len(set(pos)) == n and max(pos) == len(t) - 2
                # the first positions and the last ones are there whatever their weight
                assert set(range(cfg.sinks)) <= set(pos)
                assert set(range(len(t) - 1 - cfg.recent, len(t) - 1)) <= set(pos)
                w = layer.weight[b, h, :n]
                assert torch.isfinite(w).all() and (w >= 0).all()
    # deterministic, and drafts of nothing lead to the same end as far as nothing was evicted
    again, _ = S.generate(S.Decoder(cfg, 4, seed=3), prompts, 160)
    assert again == text


@pytest.mark.gpu
def test_steps_that_do_not_fit_are_refused():
    decoder = S.Decoder(S.Config(layers=1, **WHOLE), 1)
    for tree in (([], []), ([1] * 65, [-1] + [0] * 64), ([1, 2], [-1])):
        with pytest.raises(ValueError):
            decoder.step([tree])
    with pytest.raises(ValueError):
        decoder.prefill([[1] * 65])
    # a full tree whose last node is bit 63
    took, logits = decoder.step([([1] * 64, [-1] + list(range(63)))])
    assert len(took[0]) == len(logits[0]) and decoder.lens == [len(took[0])]
    decoder.check()


@pytest.mark.gpu
def test_weights_are_what_was_looked_at():
    """Every accepted token hands out one unit of weight per query head."""
    cfg = S.Config(layers=1, budget=256, slack=64, decay=1.0, **WHOLE)
    decoder = S.Decoder(cfg, 2, seed=8)
    prompts = [[5, 6, 7, 8], [9] * 20]
    text, _ = S.generate(decoder, prompts, 30)
    for b, t in enumerate(text):
        n, layer = decoder.lens[b], decoder.layers[0]
        per_head = layer.weight[b, :, :n].double().sum(-1)
        want = n * (cfg.q_heads // cfg.kv_heads)
        # each of the n steps' sums is 1 up to its own FP32 exponentials and lse
        assert ((per_head - want).abs() <= want * 2.0 ** -16).all(), (per_head, want)
