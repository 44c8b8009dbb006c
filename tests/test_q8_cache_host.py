"""QuantizedCache refuses sizes that no call takes before it allocates anything (tensors without memory,
no GPU)."""
import pytest

from kv_cache_compression_probe_gb300 import kvc
from kv_cache_compression_probe_gb300.pipeline import QuantizedCache


def _params(**over):
    kw = dict(B=2, L=4, H=2, G=4, d=128, P=1, W=1, dtype=kvc.KVC_BF16, n_max=64, S_max=1)
    return kvc.make_params(**{**kw, **over})


REFUSED = [
    (dict(tokens=100, page_rows=48), "page_rows"),
    (dict(tokens=100, page_rows=8), "page_rows"),
    (dict(tokens=100, page_rows=256), "page_rows"),
    (dict(tokens=100, page_rows=0), "page_rows"),
    (dict(tokens=0), "at least one token"),
    (dict(tokens=-5), "at least one token"),
    (dict(tokens=100, T=0), "at a time"),
    (dict(tokens=100, T=65537), "at a time"),
    (dict(tokens=1 << 27), "rows"),                          # 16 (b, l, h): 2^31 rows
    (dict(tokens=1 << 26, B=1, L=32, H=1), "rows"),
    (dict(tokens=(1 << 27) + 1, B=1, L=1, H=1), "rows"),
    (dict(tokens=32768 * 16 + 1, page_rows=16, n_sel=8), "32768"),
    (dict(tokens=100, n_sel=32769), "32768"),
    (dict(tokens=100, n_sel=2, first=1, recent=2), "must fit"),
    (dict(tokens=100, n_sel=2, first=-1, recent=2), "must fit"),
    (dict(tokens=100, n_sel=-1), "must fit"),
]


@pytest.mark.parametrize("kw,message", REFUSED)
def test_sizes_that_no_call_takes(kw, message):
    over = {k: kw.pop(k) for k in ("B", "L", "H") if k in kw}
    with pytest.raises(ValueError, match=message):
        QuantizedCache(_params(**over), device="meta", **kw)
