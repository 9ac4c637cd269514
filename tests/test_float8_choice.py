"""The sizes of tests/float8_forms.py reach every form that a product of the 8-bit
floating-point layer can take, so that tests/test_gpu_float8_forms.py runs each
kernel; no GPU needed."""
import random

from float8_common import GRAD_WEIGHT, MATMUL, choice, workspace
from float8_forms import SIZES, every_form, form


def test_sizes_reach_every_form():
    missing = every_form() - {form(*s) for s in SIZES}
    assert not missing, missing


def test_choices_are_sound():
    """Random sizes: tiles of one workgroup and split ones make up the output,
    no split is empty, and the workspace holds what the choice lays there."""
    r = random.Random(3)
    for _ in range(4000):
        size = lambda top: int(top ** r.random())  # noqa: E731
        product, bf16, t, n, k = r.randrange(3), r.randrange(2), size(20000), size(20000), size(20000)
        experts = r.choice([0, 0, 1, size(1000)])
        a_cols = k if product == MATMUL else n
        lda = (a_cols + 15) // 16 * 16 if product == MATMUL else a_cols
        c = choice(product, 1 << 20, lda, experts > 0, max(experts, 1), t, n, k, bf16)
        need = workspace(product, 1 << 20, lda, experts > 0, max(experts, 1), t, n, k, bf16)
        packed = (t * ((n * 2 + 15) // 16 * 16) + 255) // 256 * 256 if c["pack"] else 0
        if c["few"]:
            assert product == MATMUL and need == 0 and c["splits"] == 1
            continue
        T = c["tile"]
        rows, cols = (n if product == GRAD_WEIGHT else t), (n if product == MATMUL else k)
        tiles = -(-rows // T) * -(-cols // T)
        assert c["direct"] + c["split"] == tiles or experts
        stages = -(-k // 128) if product == MATMUL else -(-(t if product == GRAD_WEIGHT else n) // 32)
        if c["splits"] > 1:
            assert not experts and c["split"] > 0 and c["splits"] * c["groups"] <= stages
            assert need == packed + c["split"] * c["splits"] * T * T * 4
        else:
            assert need == packed and (experts or c["split"] == 0)
        assert c["groups"] == {64: 4, 256: 1}.get(T, c["groups"]) and not (experts and c["groups"] > 1)
