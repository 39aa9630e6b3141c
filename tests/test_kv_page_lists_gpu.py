"""Page lists of attention that a caller may pass by accident or as padding."""
import numpy as np
import pytest
import torch

from moe_matvec_gb300 import api
from tests.test_kv_attend_gpu import check, filled, wide
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,P,G", [(64, 16, 3), (128, 64, 12), (256, 32, 2)])
def test_lists_of_tokens_that_no_sequence_covers_are_not_looked_at(lib, dtype, D, P, G):
    # the ids of such tokens are what was in memory: nothing of them is read or flagged, their rows are not written
    rng = np.random.default_rng(2)
    lens, starts = [7 * P + 1, 3 * P], [2, 5, 6]  # tokens 0, 1 and 6, 7 of eight are padding
    pair, table = filled(rng, 2, D, P, lens)
    q = randn(rng, 8, 2 * G, D, dtype=dtype)
    ids = np.full((8, 2, 4), 2 ** 30, np.int32)
    ids[2:5], ids[5] = [0, 3, 6, 7], [1, 2, -1, 0]
    for t in (table, wide(table, P)):
        out = torch.full_like(q, 7)
        api.kv_attend(pair.dev, q, dev32(t), dev32(lens), dev32(starts), pages=dev32(ids), out=out)
        assert api.get_device_error() == 0
        pad = [0, 1, 6, 7]
        assert (out[pad] == 7).all()
        check(pair, q[2:6], table, lens, [0, 3, 4], out[2:6], pages=ids[2:6])


def test_selection_then_attention_on_a_padded_batch(lib):
    # the selection leaves the padding's ids as they are
    rng = np.random.default_rng(3)
    lens, starts = [200, 77], [0, 1, 2]
    pair, table = filled(rng, 2, 64, 16, lens)
    q = randn(rng, 5, 4, 64)
    ids = torch.full((5, 2, 3), 10_000_000, dtype=torch.int32, device="cuda")
    api.kv_select(pair.dev, q, dev32(table), dev32(lens), 3, dev32(starts), ids=ids)
    assert (ids[2:] == 10_000_000).all() and (ids[:2] < 13).all()
    out = api.kv_attend(pair.dev, q, dev32(table), dev32(lens), dev32(starts), pages=ids)
    assert api.get_device_error() == 0
    check(pair, q[:2], table, lens, None, out[:2], pages=ids[:2].cpu().numpy())
