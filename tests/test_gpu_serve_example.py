"""The serving example: the page plan, cache, attention and logit adjustment run together with the
low-bit products.  Prompts read whole, in chunks or one token at a time give the same answers, and
the grammar holds."""
import os
import sys

import numpy as np
import pytest

import bit_matvec_lb_gb300 as lb

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_chunks_and_batches_agree():
    import serve_step as s

    rng = np.random.default_rng(3)
    prompts = [rng.integers(0, s.VOCAB, n).tolist() for n in (50, 1, 17, 90)]
    odd = range(1, s.VOCAB, 2)
    whole = s.Server(4, grammar=s.grammar_of(odd)).generate(prompts, 6)
    chunks = s.Server(4, grammar=s.grammar_of(odd)).generate(prompts, 6, chunk=13)
    alone = [s.Server(1, grammar=s.grammar_of(odd)).generate([p], 6, chunk=1)[0] for p in prompts[:2]]
    assert lb.lb_device_status() == 0
    assert whole == chunks and whole[:2] == alone
    assert all(t % 2 == 1 for a in whole for t in a) and all(len(a) == 6 for a in whole)


def test_example_runs(capsys, monkeypatch):
    import serve_step as s

    monkeypatch.setattr(sys, "argv", ["serve_step.py", "--steps", "3"])
    s.main()
    assert capsys.readouterr().out.count("prompt tokens ->") == 3
