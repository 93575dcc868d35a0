"""Where the quantisers' loads leave the caches first: rows that are read once and whose
codes a product reads next, and nowhere else.  (Rows quantised by themselves, gathered
ones and the few rows that all CTAs of a kernel read lose up to 20% by it.)"""
import os
import re

import pytest

from tests.test_early_launch_loads import CSRC, FILES, code

HINT = r"evict_first|no_allocate|kLeaving"
OPS = code(os.path.join(CSRC, "mxfp4_ops.cuh"))


def test_only_one_form_of_the_load_has_the_hint():
    body = OPS[OPS.index("void load16_raw"):OPS.index("void load16_raw") + 1600]
    assert re.findall(r"if \(ALIGN == kLeaving\)\s+MOE_LOAD32\(([^)]*)\);\s+else\s+MOE_LOAD32\(([^)]*)\);", body) == \
        [('".L1::no_allocate.L2::evict_first"', '""')]
    assert len(re.findall("evict_first", OPS)) == 1


@pytest.mark.parametrize("path", [f for f in FILES if not f.endswith(("mxfp4_ops.cuh", "mxfp4_quant.cu"))], ids=os.path.basename)
def test_kernels_that_read_rows_more_than_once_have_no_hint(path):
    assert not re.search(HINT, code(path))


def test_quantising_asks_for_it_for_products_of_rows_as_they_lie():
    source = code(os.path.join(CSRC, "mxfp4_quant.cu"))
    assert re.findall(r"leaving = (.*?) &&\s+R\.rows", source) == ["for_product && tiled && !R.row_index"]
    assert re.findall(r"align = (.*?);", source) == ["leaving && R.align() == 32 ? kLeaving : R.align()"]
    calls = re.findall(r"launch_mxfp4_quantize\(R, codes, scales, (.*?), (?:st|static_cast)", source)
    assert calls == ["tiled != 0, false"]
    assert not re.search(HINT, source[source.index("launch_mxfp4_quantize_once(const"):])
