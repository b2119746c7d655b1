"""The bounds of oracle/kv4_oracle.py's attention: they follow what a row sees, and a wrong output of
its size does not pass."""
import numpy as np
import pytest

from oracle import kv4_oracle as ko

from kv4_util import Call

SCALE = 128 ** -0.5


def grown(new, lens, q_size):
    """Value scales that rise and fall by 2^36 along the sequences."""
    c = Call(20, new, lens, q_heads=4, heads=2, page=16, q_size=q_size)
    for b, n in enumerate(c.lens):
        at = np.arange(n)
        size = np.exp2(18 * np.sin(at / 150.0) - 5)[:, None].astype(np.float32)
        c.cache[3][c.table[b, at // 16], at % 16] *= size / 8
    return c


def test_bounds_do_not_follow_tokens_that_a_row_does_not_see():
    c = Call(1, [6, 70], [40, 200], q_heads=4, heads=2, page=16, q_size=0.05)
    first = ko.attention(c.q, c.cache, *c.sequences(), True, SCALE)
    rows = np.zeros(c.rows, bool)
    for b, n in enumerate(c.new):
        at = np.arange(c.lens[b] - n // 2, c.lens[b])
        c.cache[3][c.table[b, at // 16], at % 16] *= np.float32(2.0 ** 20)
        rows[c.cu_q[b]:c.cu_q[b + 1] - n // 2] = True
    later = ko.attention(c.q, c.cache, *c.sequences(), True, SCALE)
    for a, b in zip(first, later):
        assert np.array_equal(a[rows], b[rows])
    assert not np.array_equal(first[1][~rows], later[1][~rows])


@pytest.mark.parametrize("new", [1, 250])
def test_zeros_and_halves_do_not_pass_for_small_outputs(new):
    """Where value scales span 2^36, rows' outputs stand above their bounds, those that attend to
    small values among them (all but a few whose largest weight meets a small value beside a visible
    large one)."""
    c = grown([new, new], [1300, 900], 0.3)
    out, tol, _, _ = ko.attention(c.q, c.cache, *c.sequences(), True, SCALE)
    finite = np.isfinite(out) & np.isfinite(tol)
    size = np.where(finite, np.abs(out), 0).max(-1)
    off = np.where(finite, np.abs(out) / 2 - tol, -1).max(-1)
    normal = (size > 2.0 ** -14) & finite.all(-1)    # not below fp16's normal numbers
    assert (off > 0)[normal].mean() > 0.95
    if new > 1:
        assert (size[normal].max() > 2.0 ** 20 * size[normal].min()) and normal.mean() > 0.5
