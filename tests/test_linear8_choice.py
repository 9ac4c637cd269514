"""The sizes that the GPU tests give the 8-bit products reach every form of the
tile kernels that the choice of tile and split can send a product to (no GPU
needed: the choice is made on the host)."""
import math
import random

import pytest

from linear8_forms import FORMS, choice


def name(form):
    return "-".join(str(int(v) if isinstance(v, bool) else v) for v in form)


@pytest.mark.parametrize("form, size", FORMS.items(), ids=[name(f) for f in FORMS])
def test_each_size_runs_in_its_form(form, size):
    got, stages, splits = choice(form.product, *size)
    assert got == form
    assert stages // (splits * form.groups) >= 8
    t, n, k = size
    np_, nq, kd = ((n, t, k), (k, t, n), (k, n, t))[form.product]
    assert np_ % form.tile and nq % form.tile and kd % (64 if form.product == 0 else 32)


def test_no_other_form_exists():
    """Over random sizes, every product of at least eight stages per wave group
    and splits runs in one of the listed forms, and most of them come up."""
    rng = random.Random(3)
    seen = set()
    for _ in range(40000):
        kind = rng.randrange(3)
        size = [int(math.exp(rng.uniform(0, math.log(20000)))) for _ in range(3)]
        if rng.random() < 0.5:
            size = [max(16, v // 16 * 16) for v in size]
        form, stages, splits = choice(kind, *size, pad=rng.choice((0, 16)))
        if form and stages // (splits * form.groups) >= 8:
            assert form in FORMS, (form, size)
            seen.add(form)
    assert len(seen) >= 45


@pytest.mark.parametrize("t, n, k, few", [(1, 18944, 16384, True), (16, 100, 8192, True), (16, 100, 8193, False),
                                          (16, 16384, 60000, True), (32, 1024, 4096, True), (32, 4097, 4096, False),
                                          (32, 100, 4097, False), (33, 100, 64, False), (64, 100, 33, False)])
def test_where_the_few_rows_kernel_ends(t, n, k, few):
    assert (choice(0, t, n, k)[0] is None) == few
    assert choice(1, t, n, k)[0] is not None and choice(2, t, n, k)[0] is not None
