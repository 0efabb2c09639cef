"""Refusals of the linear-attention binding that test_lin_oracle.py has no case of (no GPU)."""
import pytest

from test_lin_oracle import F32, I32, I64, form, plan

ONE = dict(cu=form((2,), I64), read=form((1,), I32), write=form((1,), I32), interval=64)


def one(T, rows):
    """A call of one sequence of T tokens without offsets, with so many rungs."""
    return plan(**ONE, q=form((T, 2, 64)), k=form((T, 2, 64)), v=form((T, 4, 128)), g=form((T, 4), F32),
                ckpt=None if rows is None else form((rows, 4, 64, 128), F32))


def test_rungs_of_one_sequence_need_their_rows():
    """Without offsets the sequence's rungs start at row 0, and there are T // interval of them at most."""
    for T, rows in ((640, 10), (703, 10), (640, 12), (63, 0), (640, None)):
        one(T, rows)
    for T, rows in ((640, 9), (704, 10), (640, 0), (64, 0)):
        with pytest.raises(ValueError, match="ckpt_out"):
            one(T, rows)
