"""Elementwise comparison that says where and by how much a bound is missed."""
import numpy as np


def within(got, want, bound, what=""):
    got, want, bound = np.asarray(got), np.asarray(want), np.broadcast_to(bound, np.shape(want))
    err = np.abs(got - want)
    bad = ~(err <= bound)
    if bad.any():
        ratio = np.where(bad, err / np.maximum(bound, 1e-300), 0.0)
        at = np.unravel_index(np.nanargmax(np.where(np.isnan(ratio), np.inf, ratio)), ratio.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside, worst at {tuple(int(i) for i in at)}: got "
                             f"{got[at]!r}, want {want[at]!r}, bound {bound[at]!r}; first {np.argwhere(bad)[:3].tolist()}, "
                             f"last {np.argwhere(bad)[-3:].tolist()}")
