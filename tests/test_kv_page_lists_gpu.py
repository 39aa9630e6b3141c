"""Page lists of attention that a caller may pass by accident or as padding."""
import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests.test_kv_attend_gpu import filled
from tests.test_kv_cache_gpu import dev32, randn

pytestmark = pytest.mark.gpu


def test_an_empty_page_list_is_refused(lib):
    # as the C call refuses n_sel 0: the address of an empty tensor is null, which would mean all pages
    rng = np.random.default_rng(1)
    lens = [100, 40]
    pair, table = filled(rng, 2, 64, 16, lens)
    q = randn(rng, 2, 4, 64)
    none = torch.empty(2, 2, 0, dtype=torch.int32, device="cuda")
    with pytest.raises(api.QmvError) as e:
        api.kv_attend(pair.dev, q, dev32(table), dev32(lens), pages=none)
    assert e.value.code == -2
    # a list that names no page is not an empty one: nothing is seen
    out = api.kv_attend(pair.dev, q, dev32(table), dev32(lens), pages=dev32(np.full((2, 2, 1), -1)))
    assert (out == 0).all() and api.get_device_error() == 0
