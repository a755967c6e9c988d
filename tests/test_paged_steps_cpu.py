"""The bounds that the serving steps are held to notice mistakes: each of these, made in 64 bits,
falls outside them at every step and sequence."""

import math

import pytest
import torch

import paged_steps as ps
from paged_plain import attention64


def no_output(q, k, v):
    return torch.zeros_like(q)


def newest_key_left_out(q, k, v):
    n, m = q.shape[0], k.shape[0]
    return attention64(q, k[:-1], v[:-1], 1 / math.sqrt(ps.D), True, m - n - 1)[0]


def values_reversed(q, k, v):
    return ps.exact(q, k, v.flip(0))[0]


def keys_turned_twice(q, k, v):
    return ps.exact(q, ps.turned(k, 0)[0], v)[0]


def last_page_again(q, k, v):
    """The last whole page's keys in place of the first page's."""
    k, v = k.clone(), v.clone()
    at = k.shape[0] // ps.PAGE * ps.PAGE
    k[:ps.PAGE], v[:ps.PAGE] = k[at - ps.PAGE:at].clone(), v[at - ps.PAGE:at].clone()
    return ps.exact(q, k, v)[0]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("mistake", [no_output, newest_key_left_out, values_reversed,
                                     keys_turned_twice, last_page_again])
def test_mistakes_fall_outside_the_bounds(mistake, e4m3):
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    done = [0] * len(ps.TOTAL)
    data = ps.inputs()
    for new in ps.STEPS:
        done = [a + n for a, n in zip(done, new)]
        for s, (n, m) in enumerate(zip(new, done)):
            if n == 0 or (mistake is last_page_again and m < 2 * ps.PAGE):
                continue
            q = ps.turned(data[s][0][m - n:m], m - n)[0].to(torch.bfloat16).double()
            k = (ps.turned(data[s][1][:m], 0)[0] * 8).to(dtype).double() / 8
            v = (data[s][2][:m].double() * 8).to(dtype).double() / 8
            o, lse, a, size = ps.exact(q, k, v)
            o_tol, _ = ps.attention_bound(o, lse, a, size, m, v.abs().max(), e4m3)
            assert ((mistake(q, k, v) - o).abs() > o_tol).any()
