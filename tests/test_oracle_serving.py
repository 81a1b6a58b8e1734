"""The oracle's window mask, head norm and rotation, pinned by brute force, closed forms and
identities (CPU)."""

import math

import numpy as np
import pytest

import oracle
from oracle import serving


@pytest.mark.parametrize("Nq,Lk,window,sinks", [(1, 1, 1, 0), (3, 9, 2, 1), (9, 9, 4, 0), (4, 20, 7, 5), (5, 5, 100, 9),
                                                (2, 30, 1, 30)])
def test_window_mask_by_brute_force(Nq, Lk, window, sinks):
    m = serving.window_mask(Nq, Lk, window, sinks)
    for t in range(Nq):
        p = Lk - Nq + t
        for j in range(Lk):
            assert m[t, j] == (j <= p and (j > p - window or j < sinks))
        assert m[t, p]          # a row always sees itself


def test_wide_window_and_many_sinks_are_causal_attention():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(2, 4, 4, 8)), rng.normal(size=(2, 12, 2, 8)), rng.normal(size=(2, 12, 2, 8))
    lens = [12, 7]
    ref = oracle.attention(q, k, v, 0.3, True, lens)
    for window, sinks in ((12, 0), (1, 12), (5000, 5000)):
        got = serving.attention_window(q, k, v, 0.3, lens, window, sinks)
        assert np.allclose(got[0], ref[0], atol=1e-13) and np.allclose(got[1], ref[1], atol=1e-13)


def test_window_of_one_without_sinks_returns_the_own_value():
    rng = np.random.default_rng(4)
    q, k, v = rng.normal(size=(1, 6, 2, 4)), rng.normal(size=(1, 6, 2, 4)), rng.normal(size=(1, 6, 2, 4))
    o, lse = serving.attention_window(q, k, v, 0.5, [6], 1, 0)
    assert np.allclose(o, v) and np.allclose(lse[0].T, 0.5 * (q[0] * k[0]).sum(-1))


def test_head_norm_closed_forms():
    assert np.allclose(serving.head_norm(np.full(8, -3.0), np.ones(8), 0.0), -1.0)
    x = np.array([3.0, 4.0])
    assert np.allclose(serving.head_norm(x, np.array([1.0, 2.0]), 0.0), [3 / math.sqrt(12.5), 8 / math.sqrt(12.5)])
    assert np.allclose(serving.head_norm(np.zeros(4), np.ones(4), 1e-6), 0.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_relative_positions(interleaved):
    rng = np.random.default_rng(5)
    d, rot = 16, 8
    q, k = rng.normal(size=(1, 1, 1, d)), rng.normal(size=(1, 1, 1, d))

    def turn(x, p):
        return serving.rotate(x, np.array([[p]]), rot, interleaved=interleaved)

    assert np.allclose(turn(q, 0), q)
    assert np.allclose((turn(q, 37) ** 2).sum(), (q ** 2).sum())
    assert np.array_equal(turn(q, 37)[..., rot:], q[..., rot:])
    dots = [(turn(q, p + 5) * turn(k, p)).sum() for p in (0, 11, 4000)]
    assert np.allclose(dots, dots[0], atol=1e-9)
    # pair 0 turns by p radians
    e = np.zeros((1, 1, 1, d))
    e[..., 0] = 1.0
    y = turn(e, 2)[0, 0, 0]
    assert np.allclose([y[0], y[1 if interleaved else rot // 2]], [math.cos(2), math.sin(2)])
