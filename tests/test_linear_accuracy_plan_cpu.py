"""The long sums of the accuracy tests reach every kernel instance of moe_linear (no GPU)."""
from tests.linear_accuracy_shapes import LONG, SEGMENTED
from tests.linear_plan_shapes import PRODUCTS
from tests.test_linear_plan_cpu import plans  # noqa: F401  (fixture)


def test_long_sums_run_on_the_instance_they_are_listed_for(plans):  # noqa: F811
    assert set(LONG) == set(PRODUCTS)
    for plan, sizes in LONG.items():
        assert plans(sizes) == [plan] * len(sizes), plan


def test_segmented_sizes_run_on_the_pair_kernels(plans):  # noqa: F811
    for plan, sizes in SEGMENTED.items():
        assert plans(sizes) == [plan] * len(sizes), plan
