"""The operators together, as examples/verify_step.py runs them: drafts change how many steps a
generation takes, not what it says; a banned token is never said; an eviction keeps going."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "verify_step", os.path.join(ROOT, "examples", "verify_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def prompts(V):
    g = torch.Generator().manual_seed(1)
    return [torch.randint(0, V, (n,), generator=g).tolist() * 3 for n in (5, 9, 12, 7)]


@pytest.mark.parametrize("repetition", [1.0, 1.2])
def test_drafts_do_not_change_the_tokens(example, repetition):
    plain, steps = example.generate(prompts(example.V), 40, 0, repetition=repetition)
    assert steps == 40
    for k in (2, 5):
        drafted, ran = example.generate(prompts(example.V), 40, k, repetition=repetition)
        assert drafted == plain and ran <= steps


def test_bans_hold_with_and_without_eviction(example):
    free, _ = example.generate(prompts(example.V), 40, 4)
    banned = sorted({t for row in free for t in row[:3]})
    for budget in (0, 40):
        got, _ = example.generate(prompts(example.V), 40, 4, budget=budget, recent=12,
                                  banned=banned)
        assert not {t for row in got for t in row} & set(banned)
        assert all(0 <= t < example.V for row in got for t in row)


def test_an_eviction_that_drops_nothing_changes_nothing(example):
    free, _ = example.generate(prompts(example.V), 30, 3)
    kept, _ = example.generate(prompts(example.V), 30, 3, budget=200)
    assert kept == free
