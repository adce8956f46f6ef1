"""Calls with nothing to do: an empty batch gives empty results and never reaches
the library, whose pointers would be null."""
import pytest

from mla_latent_kv_05_gb300 import binding
from tests.test_binding_cpu import FakeTensor
from tests.test_operators_cpu import FORMATS, STREAM, Rows, fake  # noqa: F401


@pytest.mark.parametrize("fmt", FORMATS)
def test_tree_decode_of_no_sequence(fake, fmt):  # noqa: F811
    q, qr, cache = FakeTensor((0, 6, 128, 512)), FakeTensor((0, 6, 128, 64)), FakeTensor((9, 64, binding._ROW_WIDTH[fmt]))
    out, lse = FakeTensor((0, 6, 128, 512)), FakeTensor((0, 6, 128))
    got = getattr(binding, "mla_decode_tree_" + fmt)(q, qr, cache, FakeTensor((0, 5)), FakeTensor((0,)), FakeTensor((0, 6)),
                                                     0.25, out=out, lse=lse, workspace=FakeTensor((999,)), stream=STREAM)
    assert got == (out, lse) and fake.calls == []


def test_prefill_of_no_query(fake):  # noqa: F811
    q, qr, k, kr = Rows((0, 128, 128)), Rows((0, 128, 64)), Rows((4, 128, 128)), Rows((4, 64))
    out, lse = FakeTensor((0, 128, 128)), FakeTensor((0, 128))
    assert binding.mla_prefill_bf16(q, qr, k, kr, k, FakeTensor((3,)), FakeTensor((3,)), 0.5, out=out, lse=lse,
                                    workspace=FakeTensor((4096,)), stream=STREAM) == (out, lse)
    assert fake.calls == []
