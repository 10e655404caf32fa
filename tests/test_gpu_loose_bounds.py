"""max_new_tokens is an upper bound: a loose one, up to the
type's largest, changes nothing but the launch."""
import numpy as np
import pytest

from gpu_util import dev
from test_gpu_e4m3 import Case

pytestmark = pytest.mark.gpu

INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("page,h,d", [(16, 2, 64), (1, 1, 128), (256, 1, 64)])
@pytest.mark.parametrize("bound", [1 << 20, INT_MAX])
def test_append(pkv, cuda_dev, page, h, d, bound):
    """Pages far past the context are not touched, whatever the bound."""
    c = Case(pkv, cuda_dev, [300, 17, 0, 256], h, h, d, page)
    pkv.pf_device_status(reset=True)
    for new in ([200, 17, 0, 255], [100, 0, 0, 1]):
        new = np.array(new, np.int32)
        c.at = c.at + new
        offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        k, v = c.rows(int(offs[-1])), c.rows(int(offs[-1]))
        pkv.pf_append_kv(c.pool, 1, dev(k, cuda_dev), dev(v, cuda_dev), c.table_dev, dev(c.at, cuda_dev),
                         dev(offs, cuda_dev), bound)
        c.km.append(k, c.table, c.at, offs)
        c.vm.append(v, c.table, c.at, offs)
        c.check_pool()
    assert pkv.pf_device_status(reset=True) == 0
