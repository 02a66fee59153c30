"""Int arguments of the Python binding that do not fit the C call's 32 bits."""
import numpy as np
import pytest
import torch

import paged_fp8_kv_attn_b200 as pkv

from test_gpu_cache_ops import KINDS, Cache, attention_case, cuda, run_attention, run_tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(2**31, 0), (2**32 + 20, 3), (2**63, 2**40), (20, 2**32),
                                          (7, 2**33 + 1)])
def test_windows_and_sinks_past_any_length(cuda_device, kind, window, sinks):
    """They hide nothing, as one of the table's length does."""
    p, q, table, lens = attention_case(kind, [90, 1, 200], 2, 2, 64, 16, seed=4)
    run_attention(p, q, table, lens, window, sinks)
    tags = np.arange(p.shape[0], dtype=np.uint32)
    expected = tags[np.maximum(table, 0)]
    expected[2, 3] += np.uint32(1)          # a page between the sinks and a window of 20
    abort = torch.full((3,), 9, dtype=torch.uint8, device="cuda")
    pkv.kv_tag_check_window(cuda(tags), cuda(table), cuda(expected), cuda(lens), 16, window, sinks, abort)
    assert abort.tolist() == [0, 0, 1]


def test_other_arguments_are_refused(cuda_device):
    p, q, table, lens = attention_case("int4", [30], 2, 2, 64, 16, seed=1)
    c = Cache(p)
    gq, gt, gl = cuda(q), cuda(table), cuda(lens)
    with pytest.raises(ValueError, match="num_ctas"):
        c.attend(gq, gt, gl, 0.1, c.workspace(1, 4), num_ctas=2**32 + 1)
    with pytest.raises(pkv.PagedKVError, match="window"):
        c.attend(gq, gt, gl, 0.1, c.workspace(1, 4), window=-2**32)
    with pytest.raises(pkv.PagedKVError, match="sinks"):
        c.attend(gq, gt, gl, 0.1, c.workspace(1, 4), window=4, sinks=-2**32 + 4)
    z, one = np.zeros(1, np.int32), np.ones(1, np.int32)
    for P, NP, name in ((2**32 + 16, 9, "page_size"), (16, 2**32 + 9, "num_pages")):
        with pytest.raises(ValueError, match=name):
            run_tables(z, one, P, np.array([5], np.int32), 1, np.zeros((1, 1), np.int32), NP, 1)
    with pytest.raises(ValueError, match="page_size"):
        pkv.kv_tag_check_window(gt[0], gt, gt, gl, 2**32 + 16, 4, 0, torch.zeros(1, dtype=torch.uint8, device="cuda"))
