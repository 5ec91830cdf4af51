"""pa_tree_decode where the largest tree is far above the batch's."""
import pytest

import paged_kv_cache_232_gb300 as pa
from test_gpu_tree import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (8, 2, 128), (16, 1, 128), (4, 1, 64), (3, 1, 96), (4, 2, 256), (16, 1, 256)])
@pytest.mark.parametrize("ns,most", [([1, 3], 300), ([1, 300, 2], 300), ([130, 0, 1, 7], 513), ([5], 2000)])
def test_largest_tree_far_above_the_batch(hq, hkv, d, ns, most):
    """max_q_len is a bound (a captured call keeps it): blocks of tokens in which a sequence has no rows are passed over."""
    b = Batch("bf16", hq, hkv, d, 16, ns, [(211 * i + 40) % 700 for i in range(len(ns))], seed=most + d,
              extra_words=-(-most // 64) - max(1, -(-max(ns) // 64)))
    b.max_n = most
    pa.pa_device_errors(clear=True)
    out = b.run()
    assert pa.pa_device_errors(clear=True) == 0
    b.check(out)
