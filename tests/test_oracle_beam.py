"""The oracle of the beam search's choice against a loop over all continuations, and worked examples."""
import math

import numpy as np

import oracle


def test_worked_example():
    # two beams, three tokens: probabilities 1/2 1/4 1/4 and 1/5 3/5 1/5
    logits = np.log([[2.0, 1, 1], [1, 3, 1]])
    scores = np.array([[-1.0, -1.0]])
    s, parents, tokens, done, _ = oracle.oracle_beam_select(logits, scores, eos=1)
    assert parents.tolist() == [[1, 0]] and tokens.tolist() == [[1, 0]] and done.tolist() == [[True, False]]
    assert np.allclose(s, [[-1 + math.log(0.6), -1 + math.log(0.5)]])
    # the second beam has ended: it stands with its score, above all others
    s, parents, tokens, done, _ = oracle.oracle_beam_select(logits, scores, np.array([[False, True]]), eos=2, keep=4)
    assert parents.tolist() == [[1, 0, 0, 0]] and tokens.tolist() == [[2, 0, 1, 2]] and done.tolist() == [[True, False, False, True]]
    assert s[0, 0] == -1


def test_brute_force_and_ties():
    rng = np.random.default_rng(0)
    G, B, V, keep = 3, 4, 7, 9
    logits = rng.integers(-2, 3, (G * B, V)).astype(float)
    logits[rng.random((G * B, V)) < 0.2] = -np.inf
    scores = -rng.integers(0, 3, (G, B)).astype(float)
    scores[1, 2] = -np.inf
    s, parents, tokens, _, ranked = oracle.oracle_beam_select(logits, scores, keep=keep)
    for g in range(G):
        every = []
        for b in range(B):
            total = math.fsum(math.exp(x) for x in logits[g * B + b])
            for v in range(V):
                c = scores[g, b] + logits[g * B + b, v] - (math.log(total) if total else math.inf)
                every.append((-round(c, 9) if c > -math.inf else math.inf, b, v))
        every.sort()
        assert [(g * B + b, v) for _, b, v in every[:keep]] == list(zip(parents[g], tokens[g]))
        assert np.allclose(s[g], [-x[0] for x in every[:keep]])
        assert np.all(np.diff(ranked[g][np.isfinite(ranked[g])]) <= 0)
