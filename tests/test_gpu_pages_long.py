"""add_norm, append_pages and attend_pages at lengths where offsets pass 32 bits, and a prompt's queries at once."""
import pytest
import torch

import deepseek_v4_compressed_csa_gb300 as csa
from tests import _pages as P
from tests.test_gpu_pages import append_ref, build, call, gen, i32, normal, verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("small,X", [(False, 4096), (True, 128)])
def test_add_norm_of_more_values_than_an_int_counts(small, X):
    """The rows in front of and behind value 2^31, and the last ones, as they are by themselves."""
    L = P.layer(small)
    N = 2 ** 31 // X + 37
    x = torch.zeros(N, X, dtype=L.dtype, device="cuda")
    w = 1 + 0.1 * normal(gen(1), X)
    spots = [0, 5, 2 ** 30 // X - 1, 2 ** 30 // X, 2 ** 31 // X - 1, 2 ** 31 // X, 2 ** 31 // X + 1, N - 1]
    x[spots] = normal(gen(2), len(spots), X, dtype=L.dtype)
    want = csa.add_norm(L, x[spots], x[spots], w, group=64)
    got = csa.add_norm(L, x, x, w, group=64)
    for a, b in zip(got, want):
        assert torch.equal(a[spots], b)
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[spots] = False
    assert not got.scales[rest].any() and not got.codes.view(N, -1).any(1)[rest].any()


def test_append_pages_of_more_values_than_an_int_counts():
    """A long prompt's rows, 2^31 values and more."""
    L = P.layer()
    T, page = 2 ** 31 // L.D + 70, 64
    x = torch.zeros(1, T, L.D, dtype=L.dtype, device="cuda")
    spots = [0, 2 ** 30 // L.D, 2 ** 31 // L.D - 1, 2 ** 31 // L.D, T - 1]
    x[0, spots] = normal(gen(3), len(spots), L.D, dtype=L.dtype)
    n = -(-T // page)
    codes = torch.full((n, page, L.D), 0x7F, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, page), -1.0, device="cuda")
    table = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")[None]
    freq = P.inv_freq(L)
    assert csa.append_pages(L, x, csa.Pages(codes, scales), table, i32([0]), norm=True, inv_freq=freq).item() == 0
    at = torch.tensor([(n - 1 - t // page) * page + t % page for t in spots], device="cuda")
    y, e = append_ref(L, x[0, spots], torch.tensor(spots, device="cuda"), freq, None, 1)
    P.check_codes(codes.view(-1, L.D)[at], scales.view(-1)[at], y, e)
    flat = scales.view(-1)
    flat[at] = 0
    behind = [(n - 1 - t // page) * page + t % page for t in range(T, n * page)]
    assert (flat[behind] == -1).all()
    flat[behind] = 0
    assert not flat.any()


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("keys,first", [("window", 4), ("select", 0)])
def test_a_prompt(small, keys, first):
    """More than a thousand queries of a sequence in one call, a shorter and an empty one beside it."""
    L = P.layer(small, topk=24)
    args = build(L, 3, 1300, [700, 90, 30], 16, keys, first, [1300, 411, 0], seed=31)
    assert call(L, *args).item() == 0
    verify(L, *args)
