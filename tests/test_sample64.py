"""The sampling definition the GPU tests compare with, on hand examples."""
import numpy as np

from tests import sample64 as S

X = np.log([4.0, 1.0, 2.0, 1.0, 8.0])


def test_index_order_and_u():
    for u, want in ((0.0, 0), (3.9 / 16, 0), (4.1 / 16, 1), (6.9 / 16, 2), (7.1 / 16, 3), (8.1 / 16, 4), (0.999, 4), (1.0, 4), (-1.0, 0)):
        assert S.draw(X, u)[0] == want
    assert abs(S.draw(X, 0.3)[1] - 1 / 16) < 1e-15


def test_filters():
    assert [int(i) for i in S.kept(X, 1.0, 2, None, None)[0]] == [0, 4]
    assert [int(i) for i in S.kept(X, 1.0, 4, None, None)[0]] == [0, 1, 2, 4]  # of the equal ones, the lower index
    assert [int(i) for i in S.kept(X, 1.0, None, 0.5, None)[0]] == [4]
    assert [int(i) for i in S.kept(X, 1.0, None, 0.51, None)[0]] == [0, 4]
    assert [int(i) for i in S.kept(X, 1.0, None, 0.0, None)[0]] == [4]
    assert [int(i) for i in S.kept(X, 1.0, 3, 0.86, None)[0]] == [0, 2, 4]  # of 14
    assert [int(i) for i in S.kept(X, 1.0, None, None, 0.2)[0]] == [0, 2, 4]
    assert [int(i) for i in S.kept(X, 0.5, None, None, 0.2)[0]] == [0, 4]
    assert S.draw(X, 0.9, temperature=0.0)[0] == 4


def test_ends():
    inf = np.inf
    assert S.draw([-inf, -inf], 0.5) == (-1, 0.0)
    assert S.draw([np.nan, 1.0, -inf], 0.99) == (1, 1.0)
    assert S.draw([0.0, inf, 3.0, inf], 0.6) == (3, 0.5)
