"""Caches without layers have no accepted rows: refused, not answered with lengths nobody wrote."""
import pytest
import torch

from tiled_online_softmax_sm_gb300 import binding as fb

import _tree as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e4m3", [False, True])
def test_accept_refuses_no_layers(e4m3):
    def caches(layers):
        shape = (layers, 4, 2, 16, 64)
        k, v = (torch.zeros(shape, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda") for _ in "kv")
        ks, vs = (torch.zeros(shape[:4], dtype=torch.uint8, device="cuda") if e4m3 else None for _ in "kv")
        return k, v, ks, vs

    rest = (T.i32([[2, 1]]), T.i32([30]), T.i32([0, 5]), T.i32([[0, 2]]), T.i32([2]))
    for layers in (1, 2):
        k, v, ks, vs = caches(layers)
        assert fb.paged_kv_accept(k, v, *rest, ks, vs).tolist() == [27]
    k, v, ks, vs = caches(0)
    with pytest.raises(fb.FaError) as e:
        fb.paged_kv_accept(k, v, *rest, ks, vs)
    assert e.value.status == fb.FA_ERR_INVALID_ARG
    fb.paged_copy_pages(k, v, T.i32([[1, 2]]), ks, vs)      # (no pages to copy is no error)
    assert fb.fa_get_device_status() == 0
