"""The operators' error words: one set for all streams and threads of a device,
each error taken by one check."""
import threading

import numpy as np
import pytest
import torch

import fp4_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


def raise_index_errors():
    """in the quantiser's word, and in that of the product for few rows"""
    x = torch.ones(4, 64, dtype=torch.bfloat16, device=DEV)
    bad = torch.from_numpy(np.array([0, 9], dtype=np.int32)).to(DEV)
    w, s = torch.zeros(8, 32, dtype=torch.uint8, device=DEV), torch.zeros(1, 1, 1, 512, dtype=torch.uint8, device=DEV)
    moe.mxfp4_quantize(x, row_index=bad)
    moe.mxfp4_linear(x, w, s, row_index=bad)
    torch.cuda.synchronize()


def test_a_check_on_another_stream_takes_every_words_error():
    moe.ops_check()
    raise_index_errors()
    s = torch.cuda.Stream()
    with pytest.raises(moe.MoeFp4Error):
        moe.ops_check(s)
    moe.ops_check(s)
    moe.ops_check()


def test_an_error_is_reported_by_one_of_several_checks():
    moe.ops_check()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(50):
        raise_index_errors()
        reports, together = [], threading.Barrier(len(streams))

        def check(stream):
            together.wait()
            try:
                moe.ops_check(stream)
            except moe.MoeFp4Error:
                reports.append(stream)

        threads = [threading.Thread(target=check, args=(s,)) for s in streams]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert len(reports) == 1
    moe.ops_check()
