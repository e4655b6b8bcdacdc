"""The fp64 statements of the serving operators against values worked out by hand and
against differently written ones."""
import numpy as np
import pytest

from oracle import draft, serve


def test_norm_by_hand():
    x = np.array([[3.0, 4.0, 0.0, 0.0]])
    np.testing.assert_allclose(serve.norm(x, np.array([1, 2, 1, 1.0]), 0.0), [[1.2, 3.2, 0, 0]])  # rms = 2.5
    np.testing.assert_allclose(serve.norm(x, np.ones(4), 2.75), [[1.0, 4 / 3, 0, 0]])             # sqrt(6.25 + 2.75) = 3
    assert serve.norm(x, None, 1.0) is not None and (serve.norm(x, None, 1.0) == x).all()


def test_turn_by_hand():
    q = np.zeros((1, 1, 8))
    q[0, 0] = [1, 2, 3, 4, 5, 6, 7, 8]
    f = np.array([np.pi / 2, 0.0], np.float32)  # a quarter turn, none
    half, _ = serve.turn(q, [1], f, False)      # pairs (0, 2), (1, 3)
    np.testing.assert_allclose(half[0, 0], [-3, 2, 1, 4, 5, 6, 7, 8], atol=1e-6)
    near, size = serve.turn(q, [1], f, True)    # pairs (0, 1), (2, 3)
    np.testing.assert_allclose(near[0, 0], [-2, 1, 3, 4, 5, 6, 7, 8], atol=1e-6)
    np.testing.assert_allclose(size[0, 0], [3, 3, 7, 7, 5, 6, 7, 8])


@pytest.mark.parametrize("pos", [0, 1, -5, 131071, 2**31 - 1])
def test_far_angles(pos):
    """Against whole turns taken out in exact fractions."""
    from fractions import Fraction
    f = np.float32(0.123456)
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021")
    t = Fraction(float(f)) * pos
    t = float(t - two_pi * (t // two_pi))
    u = np.zeros((1, 1, 2))
    u[0, 0, 0] = 1.0
    got, _ = serve.turn(u, [pos], [f], False)
    np.testing.assert_allclose(got[0, 0], [np.cos(t), np.sin(t)], atol=1e-9)


def test_paged_is_prompt_attention_of_gathered_keys():
    rng = np.random.default_rng(0)
    page, lq, lk = 16, [3, 1, 20], [40, 16, 20]
    table = np.array([[5, 0, 7], [2, -1, -1], [1, 6, -1]])
    kp, vp = rng.standard_normal((8, page, 2, 4)), rng.standard_normal((8, page, 2, 4))
    q = rng.standard_normal((24, 4, 4))
    cu_q = np.cumsum([0] + lq)
    k = np.concatenate([kp[table[b, :(n + 15) // 16]].reshape(-1, 2, 4)[:n] for b, n in enumerate(lk)])
    v = np.concatenate([vp[table[b, :(n + 15) // 16]].reshape(-1, 2, 4)[:n] for b, n in enumerate(lk)])
    for window in (0, 9):
        want, _ = draft.attn_prompt(q, k, v, cu_q, np.cumsum([0] + lk), window, 0.7)
        got, _ = serve.attn_paged(q, kp, vp, table, lk, cu_q, window, 0.7)
        np.testing.assert_allclose(got, want)


def test_paged_keys_without_a_page():
    """A page that is none, and keys past the table, are kept by no row."""
    rng = np.random.default_rng(1)
    kp, vp = rng.standard_normal((3, 16, 1, 4)), rng.standard_normal((3, 16, 1, 4))
    q = rng.standard_normal((1, 1, 4))
    for bad in (-1, 3, 1 << 30):
        got, _ = serve.attn_paged(q, kp, vp, np.array([[0, bad, 2]]), [45], None, 0, 1.0)
        want, _ = draft.attend(q[:, 0], np.concatenate([kp[0, :, 0], kp[2, :13, 0]]),
                               np.concatenate([vp[0, :, 0], vp[2, :13, 0]]), np.ones((1, 29), bool), 1.0)
        np.testing.assert_allclose(got[:, 0], want)
    got, _ = serve.attn_paged(q, kp, vp, np.array([[1]]), [40], None, 0, 1.0)
    want, _ = draft.attend(q[:, 0], kp[1, :, 0], vp[1, :, 0], np.ones((1, 16), bool), 1.0)
    np.testing.assert_allclose(got[:, 0], want)
    assert not serve.attn_paged(q, kp, vp, np.array([[-1]]), [5], None, 0, 1.0)[0].any()


def test_rows_of_sequences():
    seq, pos = serve.rows_of([1, 3, 3, 4], [10, 7, 1], 6)
    assert seq.tolist() == [-1, 0, 0, 2, -1, -1] and pos[1:4].tolist() == [8, 9, 0]
    seq, pos = serve.rows_of(None, [10, 0, -4], 3)
    assert seq.tolist() == [0, 1, 2] and pos.tolist() == [9, -1, -1]


def test_lora_by_hand():
    y = np.zeros((4, 2))
    x = np.array([[1.0, 2.0]] * 4)
    a = np.array([[[1.0, 1.0]], [[2.0, 0.0]]])
    b = np.array([[[1.0], [10.0]], [[3.0], [0.0]]])
    out, size, low, status = serve.lora(y, x, a, b, [0, 1, -1, 2], [1.0, 0.5])
    assert out.tolist() == [[3, 30], [3, 0], [0, 0], [0, 0]] and status == 1
    assert low.tolist() == out.tolist()
