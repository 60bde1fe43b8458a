"""A program's own plan: what Routing takes and refuses (no GPU calls)."""
import pytest
import torch

ex = pytest.importorskip("tensor_gemm_reduce_amd.experts")

T, K, E = 4, 2, 3


def parts(**kw):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    p = dict(weights=torch.zeros(T, K), experts=i(T, K), offsets=i(E + 1), tokens=i(T * K), slots=i(T, K), E=E)
    return dict(p, **kw)


def test_a_whole_plan_is_taken():
    r = ex.Routing(**parts())
    assert (r.T, r.k, r.E, r.rows) == (T, K, E, T * K)
    assert ex.Routing(**parts(weights=None)).weights is None


@pytest.mark.parametrize("name,value,error", [
    ("offsets", torch.zeros(E, dtype=torch.int32), ValueError),            # short: the last expert's end would be read behind it
    ("offsets", torch.zeros(E + 1, dtype=torch.int64), TypeError),
    ("offsets", torch.zeros(2 * E + 2, dtype=torch.int32)[::2], ValueError),
    ("tokens", torch.zeros(T * K - 1, dtype=torch.int32), ValueError),
    ("tokens", torch.zeros((T, K), dtype=torch.int32), ValueError),
    ("tokens", torch.zeros(T * K, dtype=torch.int64), TypeError),
    ("slots", torch.zeros(T * K, dtype=torch.int32), ValueError),
    ("slots", torch.zeros((K, T), dtype=torch.int32).t(), ValueError),
    ("experts", torch.zeros((T, K), dtype=torch.int64), TypeError),
    ("experts", torch.zeros(T * K, dtype=torch.int32), ValueError),
    ("weights", torch.zeros((T, K), dtype=torch.float64), TypeError),
    ("weights", torch.zeros((T, 1)), ValueError),
    ("E", 0, ValueError),
    ("E", E + 1, ValueError),
])
def test_a_plan_of_other_types_or_shapes_is_refused(name, value, error):
    with pytest.raises(error, match=name if name != "E" else "E|offsets"):
        ex.Routing(**parts(**{name: value}))
