"""The direct-to-LDS loads of the dense operators' tiles set M0 in inline asm
(as those of the grouped GEMMs): the compiler must emit no use of M0 of its
own in the same source.  Compiled to assembly with the library's flags."""
import pytest

from test_asm_m0 import _assemble, m0_uses


@pytest.mark.timeout(600)
def test_compiler_leaves_m0_alone_in_the_dense_tiles(tmp_path):
    inside, outside = m0_uses(_assemble("dense_ffn.hip", str(tmp_path / "dense_ffn.s")))
    assert inside, "no inline-asm write of m0 found"
    assert not outside, outside[:5]
