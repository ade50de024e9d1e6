"""Pins of oracle/scored.py and oracle/lora.py: hand cases and special values."""

import math

import numpy as np

from oracle import lora, router, scored

LOG3 = math.log(3.0)


def test_softmax_hand_case():
    # exp: 1, 3, 3, 1 -> scores 1/8, 3/8, 3/8, 1/8; the tie goes to the lower index
    r = scored.route([[0.0, LOG3, LOG3, 0.0]], 2, renormalize=False, scale=2.0)
    assert r["topk_ids"].tolist() == [[1, 2]] and np.allclose(r["topk_w"], [[0.75, 0.75]])
    r = scored.route([[0.0, LOG3, LOG3, 0.0]], 3)
    assert r["topk_ids"].tolist() == [[1, 2, 0]] and np.allclose(r["topk_w"], [[3 / 7, 3 / 7, 1 / 7]])


def test_sigmoid_with_bias_chooses_by_the_sum_and_weighs_by_the_score():
    # scores 1/2, 3/4, 1/4, 1/2; bias lifts expert 2 to 0.95 and expert 3 to 0.6
    r = scored.route([[0.0, LOG3, -LOG3, 0.0]], 2, "sigmoid", bias=[0.0, 0.0, 0.7, 0.1])
    assert r["topk_ids"].tolist() == [[2, 1]] and np.allclose(r["topk_w"], [[0.25, 0.75]])
    assert r["expert_off"].tolist() == [0, 0, 1, 2, 2] and r["sorted_pairs"].tolist() == [1, 0]


def test_groups():
    # groups {0, 1}, {2, 3}, {4, 5}: by the largest value {4, 5} is first, by the two largest {2, 3}
    l = [[0.0, 0.0, LOG3, LOG3, 2 * LOG3, -8.0]]
    assert scored.route(l, 2, "sigmoid", groups=3, keep=1, top=1)["topk_ids"].tolist() == [[4, 5]]
    assert scored.route(l, 2, "sigmoid", groups=3, keep=1, top=2)["topk_ids"].tolist() == [[2, 3]]
    assert scored.route(l, 3, "sigmoid", groups=3, keep=2, top=2)["topk_ids"].tolist() == [[2, 3, 0]]


def test_plain_softmax_is_the_router_of_the_package():
    lg = np.random.default_rng(0).standard_normal((9, 12)).astype(np.float32)
    r, q = scored.route(lg, 4), router.route(lg, 4)
    assert np.array_equal(r["topk_ids"], q["ids"]) and np.allclose(r["topk_w"], q["weights"])
    assert np.array_equal(r["pair_pos"], q["pair_pos"])


def test_masks_and_special_values():
    inf, nan = math.inf, math.nan
    for score in ("softmax", "sigmoid"):
        r = scored.route([[-inf] * 4], 2, score)
        assert r["topk_ids"].tolist() == [[0, 1]] and r["topk_w"].tolist() == [[0.0, 0.0]]
        r = scored.route([[-inf, 1.0, -inf, -inf]], 2, score)
        assert r["topk_ids"].tolist() == [[1, 0]] and r["topk_w"].tolist() == [[1.0, 0.0]]
        r = scored.route([[nan, -inf, 0.0]], 3, score)
        assert r["topk_ids"].tolist() == [[2, 1, 0]] and np.isnan(r["topk_w"]).all()
    # a bias chooses among masked experts
    assert scored.route([[-inf] * 3], 1, "sigmoid", bias=[0.0, 0.5, nan])["topk_ids"].tolist() == [[1]]


def test_lora_hand_case():
    x = np.array([[1.0, 2.0], [3.0, 0.0], [1.0, 1.0]])
    a = np.array([[[1.0, 1.0]], [[0.0, 2.0]]])          # [L 2, R 1, K 2]
    b = np.array([[[1.0], [10.0]], [[2.0], [0.5]]])     # [L, N 2, R 1]
    d, lim = lora.delta(x, a, b, [0, 2, 1], [2.0, 1.0])
    assert d.tolist() == [[6.0, 60.0], [0.0, 0.0], [4.0, 1.0]]
    assert (lim[1] == 0).all() and (lim[0] > 0).all() and (lim[[0, 2]] < 1e-4).all()


def test_whole_sums_would_show_a_lost_part():
    """The inner sum of the GPU tests that take it whole: each of its three bf16 parts, dropped, changes what they expect."""
    h = np.float32(1 + 2.0 ** -12 + 2.0 ** -23)
    parts = []
    for _ in range(3):
        p = (np.array([h], np.float32).view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)[0]
        parts.append(float(p))
        h = np.float32(h - p)
    assert parts == [1.0, 2.0 ** -12, 2.0 ** -23] and h == 0
    for lost in range(3):
        left = sum(p for i, p in enumerate(parts) if i != lost)
        assert 1024 * (left - 1) != 0.25 + 2.0 ** -13 and 1024 * (left - 1 - 2.0 ** -12) != 2.0 ** -13
