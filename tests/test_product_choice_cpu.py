"""Which form of the products a size takes: the sizes of the other tests and of the
smoke run cover what they are there for, and every form is reached."""
import pytest

import product_forms

MANY = (0, 0)


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    return product_forms.load(tmp_path_factory.mktemp("forms"), 1_000_000)


@pytest.mark.parametrize("rows,cols,depth,experts,form", [
    # few rows, the depth split as far as there are blocks to fill
    (1, 128, 128, 1, (16, 1)), (300, 136, 656, 3, (16, 2)), (17, 520, 400, 1, (16, 4)),
    (16, 512, 2048, 1, (16, 8)), (16, 7168, 2048, 1, (16, 4)),
    (1003, 520, 272, 1, (32, 1)), (800, 136, 4112, 3, (32, 2)), (300, 136, 4112, 3, (32, 4)),
    (200, 136, 8208, 3, (32, 8)), (512, 4096, 7168, 32, (32, 2)),
    (3000, 136, 128, 3, (64, 1)), (1024, 4096, 7168, 32, (64, 2)), (1000, 136, 16400, 3, (64, 4)),
    (1500, 136, 16400, 3, (64, 8)),
    # many rows, and the smoke run's product
    (1100, 1288, 656, 1, MANY), (20000, 272, 128, 1, MANY), (12000, 608, 64, 1, MANY),
    (20480, 384, 512, 1, MANY), (8192, 7168, 2048, 1, MANY), (16384, 4096, 7168, 32, MANY)])
def test_form_of_a_size(L, rows, cols, depth, experts, form):
    assert product_forms.choice(L, rows, cols, depth, experts) == form


def test_a_split_has_a_block_of_the_depth_for_each_part(L):
    for depth in (16, 128, 144, 256, 272, 384, 528, 1024):
        for rows in (1, 40, 70, 300):
            for experts in (1, 7):
                tokens, split = product_forms.choice(L, rows, 128, depth, experts)
                assert split == 0 or split <= -(-depth // 128)
