"""The fp64 statements of the prompt and draft operators against worked examples."""
import numpy as np

from oracle import draft


def test_attend_two_keys_by_hand():
    # scores 0 and log 3: weights 1/4 and 3/4
    q = np.array([[1.0, 0.0]])
    k = np.array([[0.0, 5.0], [np.log(3.0), 7.0]])
    v = np.array([[4.0, 0.0], [8.0, -4.0]])
    out, ab = draft.attend(q, k, v, np.array([[True, True]]), 1.0)
    np.testing.assert_allclose(out, [[7.0, -3.0]], rtol=1e-14)
    np.testing.assert_allclose(ab, [[7.0, 3.0]], rtol=1e-14)


def test_attend_ignores_what_is_not_kept():
    v = np.array([[1.0], [np.nan]])
    out, _ = draft.attend(np.ones((2, 1)), np.array([[1.0], [np.inf]]), v, np.array([[True, False], [False, False]]), 1.0)
    assert out[0, 0] == 1.0 and out[1, 0] == 0.0


def test_prompt_positions_and_window():
    # one-hot values give the kept sets; zero queries give equal weights
    T = 5
    q, k = np.zeros((3, 1, T)), np.zeros((T, 1, T))
    v = np.eye(T)[:, None, :]
    out, _ = draft.attn_prompt(q, k, v, [0, 3], [0, 5], 2, 1.0)
    want = [[0, .5, .5, 0, 0], [0, 0, .5, .5, 0], [0, 0, 0, .5, .5]]
    np.testing.assert_allclose(out[:, 0], want)
    out, _ = draft.attn_prompt(q, k[:2], v[:2], [0, 3], [0, 2], 0, 1.0)  # more queries than keys
    np.testing.assert_allclose(out[:, 0], [[0] * 5, [1, 0, 0, 0, 0], [.5, .5, 0, 0, 0]])


def test_tree_chains_and_keeps():
    parents = [-1, 0, 0, 1, 9, -2, 5]
    assert draft.tree_chain(parents, 3) == [3, 1, 0]
    assert draft.tree_chain(parents, 4) == [4]        # a parent after the node counts as none
    assert draft.tree_chain(parents, 5) == []
    assert draft.tree_chain(parents, 6) == [6, 5]
    keep = draft.tree_keep(parents, 3, None, 4, 0)
    assert keep[3].tolist() == [True, True, True, False] + [True, True, False, True, False, False, False]
    keep = draft.tree_keep(parents, 3, [4, 1, 2, -1], 4, 2)  # ring: slot 0 holds a later position
    assert keep[0].tolist() == [False, False, True, False] + [True] + [False] * 6
    assert keep[3].tolist() == [False] * 4 + [False, True, False, True, False, False, False]


def test_logprobs_by_hand():
    x = np.log(np.array([[1.0, 2.0, 1.0, 4.0]], np.float64)).astype(np.float32)
    lp, ent, top, ids, st = draft.logprobs(x, [1], 3)
    np.testing.assert_allclose(lp, np.log(0.25), rtol=1e-6)
    np.testing.assert_allclose(ent, 2 * 0.125 * np.log(8) + 0.25 * np.log(4) + 0.5 * np.log(2), rtol=1e-6)
    assert ids.tolist() == [[3, 1, 0]] and st == 0
    _, ent, top, ids, st = draft.logprobs(np.array([[-np.inf, -np.inf]]), [5], 3)
    assert ent[0] == 0 and np.all(top == -np.inf) and ids.tolist() == [[0, 1, -1]] and st == 1


def test_kv_commit_wraps_and_refuses():
    L, B, T, N, W = 2, 1, 3, 4, 8
    kc, vc = np.zeros((L, B, T, W)), np.zeros((L, B, T, W))
    kt = np.arange(L * N, dtype=float).reshape(L, B, N, 1) + np.ones(W)
    kp = np.array([[3, 4, 2]])
    k2, v2, kp2, st = draft.kv_commit(kc, vc, kp, kt, kt, [[0, 2, 3, 0]], [3], [5])
    assert kp2.tolist() == [[6, 7, 5]] and st == 0
    assert k2[0, 0, :, 0].tolist() == [3.0, 4.0, 1.0]
    _, _, _, st = draft.kv_commit(kc, vc, None, kt, kt, [[0, 9, 1, 1]], [4], [1])
    assert st == 1
