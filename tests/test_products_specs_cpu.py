"""What the binding keeps of a configuration: a server whose calls have a thousand different row counts, in turn, makes
each one's specs once."""
import pytest

from mixture_experts_ffn_gemm_gb300 import binding as B

MAKERS = {
    "_product_specs": lambda r: B.make_product_config(r, 4, 64, 128),
    "_quantize_specs": lambda r: B.make_micro_config(r, 128, "nv", groups=4),
    "_dequantize_specs": lambda r: B.make_micro_config(r, 128, "mx", groups=4),
    "_micro_product_specs": lambda r: B.make_micro_product_config(r, 4, 64, 128, "nv"),
}


@pytest.mark.parametrize("name", MAKERS)
def test_specs_of_a_thousand_row_counts_are_made_once(name):
    specs = getattr(B, name)
    specs.cache_clear()
    keys = [bytes(MAKERS[name](r)) for r in range(1, 1001)]
    first = [specs(k) for k in keys]
    again = [specs(k) for k in keys]
    assert specs.cache_info().misses == 1000
    assert all(a is b for a, b in zip(first, again))
    assert len({s for s in first}) == 1000  # each its own
    specs.cache_clear()
