"""Wrong operands of latent attention's Python calls, GPU tensors all: each is
refused before anything is enqueued."""
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from tests.test_gpu_ops_refusals import BOTH, F32, I32, U8, z

pytestmark = pytest.mark.gpu


def decode(**kw):
    t = {"q": z(2, 16, 576), "cache": z(8, 64, 576), "block_table": z(2, 4, dtype=I32), "lengths": z(2, dtype=I32),
         "scale": 0.1}
    return moe.latent_decode(**{**t, **kw})


def attention(**kw):
    t = {"q": z(8, 4, 192), "kv": z(9, 4, 256), "k_rope": z(9, 64), "q_offsets": z(3, dtype=I32), "k_offsets": z(3, dtype=I32),
         "scale": 0.1}
    return moe.latent_attention(**{**t, **kw})


REFUSED = {
    "attention: q of fp32": lambda: attention(q=z(8, 4, 192, dtype=F32)),
    "attention: q's width": lambda: attention(q=z(8, 4, 128)),
    "attention: q of two dimensions": lambda: attention(q=z(32, 192)),
    "attention: no heads": lambda: attention(q=z(8, 0, 192), kv=z(9, 0, 256)),
    "attention: many heads": lambda: attention(q=z(8, 1025, 192), kv=z(9, 1025, 256)),
    "attention: other heads": lambda: attention(kv=z(9, 1, 256)),
    "attention: one head for all": lambda: attention(kv=z(9, 1, 256).expand(9, 4, 256)),
    "attention: q off 16 bytes": lambda: attention(q=z(8, 4, 196)[:, :, 4:]),
    "attention: q's columns apart": lambda: attention(q=z(8, 192, 4).transpose(1, 2)),
    "attention: kv's width": lambda: attention(kv=z(9, 4, 320)),
    "attention: k_rope's rows": lambda: attention(k_rope=z(8, 64)),
    "attention: k_rope's width": lambda: attention(k_rope=z(9, 32)),
    "attention: k_rope of heads": lambda: attention(k_rope=z(9, 4, 64)),
    "attention: k_rope off 16 bytes": lambda: attention(k_rope=z(9, 68)[:, 4:]),
    "attention: k_rope's columns apart": lambda: attention(k_rope=z(64, 9).t()),
    "attention: offsets' number": lambda: attention(q_offsets=z(2, dtype=I32)),
    "attention: no offsets' elements": lambda: attention(q_offsets=z(0, dtype=I32), k_offsets=z(0, dtype=I32)),
    "attention: offsets' type": lambda: attention(k_offsets=z(3, dtype=torch.int64)),
    "attention: no offsets": lambda: attention(q_offsets=None),
    "attention: scale": lambda: attention(scale=None),
    "attention: causal neither": lambda: attention(causal=BOTH),
    "attention: small workspace": lambda: attention(workspace=z(moe.latent_attention_workspace_bytes() - 1, dtype=U8)),
    "attention: workspace's type": lambda: attention(workspace=z(1 << 26)),
    "attention: out's shape": lambda: attention(out=z(8, 4, 192)),
    "attention: out's type": lambda: attention(out=z(8, 4, 128, dtype=F32)),
    "attention: out's strides": lambda: attention(out=z(4, 8, 128).transpose(0, 1)),
    "decode: q of fp32": lambda: decode(q=z(2, 16, 576, dtype=F32)),
    "decode: q's width": lambda: decode(q=z(2, 16, 512)),
    "decode: q of two dimensions": lambda: decode(q=z(32, 576)),
    "decode: no heads": lambda: decode(q=z(2, 0, 576)),
    "decode: many heads": lambda: decode(q=z(2, 1025, 576)),
    "decode: q's columns apart": lambda: decode(q=z(2, 576, 16).transpose(1, 2)),
    "decode: q off 16 bytes": lambda: decode(q=z(2, 16, 577)[:, :, 1:]),
    "decode: heads over one another": lambda: decode(q=z(2, 1, 576).expand(2, 16, 576)),
    "decode: q not a tensor": lambda: decode(q=[1.0]),
    "decode: cache's width": lambda: decode(cache=z(8, 64, 512)),
    "decode: cache of fp32": lambda: decode(cache=z(8, 64, 576, dtype=F32)),
    "decode: cache's strides": lambda: decode(cache=z(8, 64, 640)[:, :, :576]),
    "decode: cache of two dimensions": lambda: decode(cache=z(512, 576)),
    "decode: table's type": lambda: decode(block_table=z(2, 4, dtype=torch.int64)),
    "decode: table's rows": lambda: decode(block_table=z(3, 4, dtype=I32)),
    "decode: table's columns apart": lambda: decode(block_table=z(4, 2, dtype=I32).t()),
    "decode: one row of the table for all": lambda: decode(block_table=z(1, 4, dtype=I32).expand(2, 4)),
    "decode: lengths' number": lambda: decode(lengths=z(3, dtype=I32)),
    "decode: lengths' type": lambda: decode(lengths=z(2, dtype=torch.int64)),
    "decode: no lengths": lambda: decode(lengths=None),
    "decode: scale": lambda: decode(scale="small"),
    "decode: out's shape": lambda: decode(out=z(2, 16, 576)),
    "decode: out's type": lambda: decode(out=z(2, 16, 512, dtype=F32)),
    "decode: out's strides": lambda: decode(out=z(2, 16, 1024)[:, :, :512]),
    "decode: small workspace": lambda: decode(workspace=z(moe.latent_decode_workspace_bytes(16) - 1, dtype=U8)),
    "decode: workspace's type": lambda: decode(workspace=z(1 << 26)),
}


@pytest.mark.parametrize("name", list(REFUSED))
def test_refused(name):
    with pytest.raises(ValueError):
        REFUSED[name]()
    moe.ops_check()


def test_sizes_that_the_library_refuses():
    for call in (lambda: decode(cache=z(8, 40, 576)), lambda: decode(cache=z(8, 8, 576)), lambda: decode(cache=z(0, 64, 576)),
                 lambda: decode(block_table=z(2, 0, dtype=I32)), lambda: decode(scale=float("nan")),
                 lambda: attention(scale=0.0), lambda: attention(scale=-1.0), lambda: attention(scale=float("nan"))):
        with pytest.raises(moe.MoeFp4Error):
            call()
    moe.ops_check()
