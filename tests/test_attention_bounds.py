"""The bound of the long attention tests tells a wrong output from a right one:
it rejects zeros, uniform weights, sums that are off by 2^-10 of their size, and
a sequence without its first or last position (the first or last 32 of 9001 and
more), in every form that the GPU tests run.  (No GPU.)"""

import numpy as np
import pytest

from attention_cases import ENOUGH, FORMS, short, split, whole


@pytest.mark.parametrize("form,D,group", FORMS)
@pytest.mark.parametrize("kind", [whole, lambda *a: whole(*a, window=2500), split])
def test_bound_rejects_wrong_outputs(form, D, group, kind):
    case = kind(form, D, group)
    for i in (0, 2):
        wrong = {}
        heads = range(0, case.heads, max(1, case.heads // 6))
        for h in heads:
            out, lse, bound, lb, p, v = case.reference(i, h)
            assert (bound < 0.05 * np.max(np.abs(out))).all() and lb < 1e-4
            k = 32 if len(p) > 5000 else 1
            for name, y in (("zeros", 0 * out), ("uniform", v.mean(0)), ("off", out + 2.0 ** -10 * (p @ np.abs(v))),
                            ("last", p[:-k] @ v[:-k] / p[:-k].sum()), ("first", p[k:] @ v[k:] / p[k:].sum())):
                wrong[name] = wrong.get(name, 0) + int(np.sum(np.abs(y - out) > bound))
        assert all(wrong.values()), (i, wrong)
        assert wrong["zeros"] > 0.5 * len(heads) * D and wrong["off"] > 0.3 * len(heads) * D, wrong


@pytest.mark.parametrize("form,D,group", FORMS)
def test_bound_rejects_wrong_short_outputs(form, D, group):
    case = short(form, D, group)
    for i, n in enumerate(case.lens):
        wrong = {}
        for h in range(case.heads):
            out, lse, bound, lb, p, v = case.reference(i, h)
            ys = [("zeros", 0 * out)]
            if n > 1:
                ys += [("uniform", v.mean(0)), ("last", p[:-1] @ v[:-1] / p[:-1].sum()),
                       ("first", p[1:] @ v[1:] / p[1:].sum())]
            for name, y in ys:
                wrong[name] = wrong.get(name, 0) + int(np.sum(np.abs(y - out) > bound))
        assert all(wrong.values()), (n, wrong)
        assert wrong["zeros"] > 0.6 * case.heads * D, (n, wrong)


def test_sequences_reach_the_long_state():
    """Rows that are not split have 256 pages (32 chunks for each of 4 waves)."""
    for form, D, group in FORMS:
        for window in (0, 2500):
            case = whole(form, D, group, window)
            assert len(case.lens) * case.kv_heads >= ENOUGH[form, D] and case.lens[0] // case.page >= 256
            assert (case.window or case.width * case.page) <= 4096
