"""The ragged attention oracle: closed forms, agreement with the decode
oracle row by row, a library cross-check, and causality."""
import numpy as np
import pytest
import torch

from oracle import paged_attention as OPA
from oracle import prompt as OP


def _case(seed, lens, hkv=2, group=2, d=8, bs=4):
    rng = np.random.default_rng(seed)
    width = max(-(-n // bs) for n in lens) + 1
    order = rng.permutation(sum(-(-n // bs) for n in lens) + 3)
    tab = -np.ones((len(lens), width), dtype=np.int64)
    at = 0
    for b, n in enumerate(lens):
        w = -(-n // bs)
        tab[b, :w] = order[at:at + w]
        at += w
    k = rng.standard_normal((len(order), hkv, bs, d))
    v = rng.standard_normal((len(order), hkv, bs, d))
    return rng, tab, k, v, hkv * group


def test_causal_rows_equal_the_decode_oracle_at_their_length():
    lens, news = [11, 4, 0, 9], [5, 4, 0, 1]
    rng, tab, k, v, hq = _case(0, lens)
    start = np.concatenate([[0], np.cumsum(news)])
    q = rng.standard_normal((start[-1] + 2, hq, 8))
    out, spread = OP.attend_rows(q, k, v, tab, start, lens, 0.4, True)
    for b in range(4):
        for i in range(news[b]):
            n = lens[b] - news[b] + i + 1
            ref = OPA.decode(q[start[b] + i][None], k, v, tab[b:b + 1], [n], 0.4)[0]
            assert np.allclose(out[start[b] + i], ref, atol=1e-13)
    assert np.isnan(out[start[-1]:]).all()
    assert (spread[:start[-1]] >= np.abs(out[:start[-1]]) - 1e-12).all()


def test_cross_rows_and_empty_encoder():
    lens, news = [7, 0], [3, 2]
    rng, tab, k, v, hq = _case(1, lens)
    q = rng.standard_normal((5, hq, 8))
    out, _ = OP.attend_rows(q, k, v, tab, [0, 3, 5], lens, 0.3, False)
    for i in range(3):
        assert np.allclose(out[i], OPA.decode(q[i][None], k, v, tab[:1], [7], 0.3)[0], atol=1e-13)
    assert (out[3:] == 0).all()


@pytest.mark.parametrize("causal", [False, True])
def test_library_cross_check(causal):
    n = 13
    rng, tab, k, v, hq = _case(2, [n], group=1)
    q = rng.standard_normal((n, hq, 8))
    out, _ = OP.attend_rows(q, k, v, tab, [0, n], [n], 0.5, causal)
    kk = OPA.gather_sequence(k, tab[0], n, 4).transpose(1, 0, 2)
    vv = OPA.gather_sequence(v, tab[0], n, 4).transpose(1, 0, 2)
    ref = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q.transpose(1, 0, 2).copy()), torch.from_numpy(kk.copy()),
        torch.from_numpy(vv.copy()), is_causal=causal, scale=0.5)
    assert np.allclose(out, ref.numpy().transpose(1, 0, 2), atol=1e-12)


def test_later_tokens_do_not_reach_earlier_queries():
    rng, tab, k, v, hq = _case(3, [9])
    q = rng.standard_normal((9, hq, 8))
    a, _ = OP.attend_rows(q, k, v, tab, [0, 9], [9], 1.0, True)
    k2, v2 = k.copy(), v.copy()
    blk, off = tab[0][6 // 4], 6 % 4
    k2[blk, :, off] += 5
    v2[blk, :, off] -= 7
    b, _ = OP.attend_rows(q, k2, v2, tab, [0, 9], [9], 1.0, True)
    assert (a[:6] == b[:6]).all() and not np.allclose(a[6:], b[6:])
