"""Every form of the AdamW step on inputs that are the same in every run: what
fails here fails again. Tolerances: test_gpu_adamw.py."""

from __future__ import annotations

import pytest

from test_gpu_adamw import FORMS, SIZES, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("offset", [0, 1, 3, 8])
@pytest.mark.parametrize("seed", [1, 2])
def test_step(form, offset, seed):
    c = Case([form, offset, seed], [(n, *FORMS[form]) for n in SIZES], offset)
    decay = [0.1 * (i % 3) for i in range(len(SIZES))]
    for t in (1, 2, 3):
        before = c.before()
        c.step(decay)
        c.check(before, t, decay)
