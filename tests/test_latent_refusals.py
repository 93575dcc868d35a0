"""Refusals of latent attention, without a GPU: every bad argument is caught on the
host, before anything is enqueued; and no read-only loads in the sources
(test_early_launch_loads.py says why)."""
import ctypes
import glob
import os
import re

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import fp4_mixture_experts_gb300 as moe
from fp4_mixture_experts_gb300 import build as build_mod
from fp4_mixture_experts_gb300._ops import LatentAttentionArgs, LatentDecodeArgs
from tests.test_early_launch_loads import CSRC, code

FAKE = 0x100000  # never dereferenced
BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.lib_path()):
        build_mod.build()
    return moe.load_library()


def test_decode(lib):
    base = dict(B=2, H=16, page=64, pages=10, width=4, scale=0.1, q_stride=16 * 576, q_head_stride=576, table_stride=4, q=FAKE,
                cache=FAKE, table=FAKE, lengths=FAKE, out=FAKE)

    def call(work=FAKE, size=1 << 30, **kw):
        a = LatentDecodeArgs()
        for k, v in {**base, **kw}.items():
            setattr(a, k, v)
        return lib.moe_fp4_latent_decode(ctypes.byref(a), work, size, None)

    assert lib.moe_fp4_latent_decode(None, FAKE, 1 << 30, None) == -1
    need = moe.latent_decode_workspace_bytes(16)
    assert need > 0 and moe.latent_decode_workspace_bytes(0) == 0 and moe.latent_decode_workspace_bytes(1025) == 0
    for bad in (dict(B=-1), dict(H=0), dict(H=1025), dict(page=0), dict(page=8), dict(page=40), dict(page=-64), dict(pages=0),
                dict(width=0), dict(scale=float("nan")), dict(scale=float("-inf")), dict(scale=3e38), dict(table_stride=3), dict(q=None), dict(cache=None), dict(table=None),
                dict(lengths=None), dict(out=None), dict(q=FAKE + 8), dict(cache=FAKE + 2), dict(table=FAKE + 2),
                dict(lengths=FAKE + 2), dict(out=FAKE + 8), dict(q_stride=575), dict(q_stride=16 * 576 + 4),
                dict(q_head_stride=570), dict(q_head_stride=580), dict(q_stride=1 << 39), dict(work=None), dict(work=FAKE + 16)):
        assert call(**bad) == -1, bad
    for big in (dict(pages=1 << 25), dict(width=1 << 25, table_stride=1 << 25), dict(B=1 << 30), dict(B=(1 << 24) + 1)):
        assert call(**big) == -2, big
    assert call(size=need - 1) == -3
    assert call(B=0, q=None, cache=None, work=None) == 0


def test_attention(lib):
    base = dict(B=2, H=16, causal=1, scale=0.1, Tq=40, Tk=60, q_stride=16 * 192, q_head_stride=192, kv_stride=16 * 256,
                kv_head_stride=256, rope_stride=64, q=FAKE, kv=FAKE, k_rope=FAKE, q_offsets=FAKE, k_offsets=FAKE, out=FAKE)

    def call(work=FAKE, size=1 << 30, **kw):
        a = LatentAttentionArgs()
        for k, v in {**base, **kw}.items():
            setattr(a, k, v)
        return lib.moe_fp4_latent_attention(ctypes.byref(a), work, size, None)

    assert lib.moe_fp4_latent_attention(None, FAKE, 1 << 30, None) == -1
    assert call(work=None) == -1 and call(work=FAKE + 16) == -1
    assert call(size=moe.latent_attention_workspace_bytes() - 1) == -3
    for bad in (dict(B=-1), dict(H=0), dict(H=1025), dict(causal=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(scale=3e38), dict(Tq=-1), dict(Tk=-1), dict(q=None), dict(kv=None), dict(k_rope=None),
                dict(q_offsets=None), dict(k_offsets=None), dict(out=None), dict(q=FAKE + 8), dict(kv=FAKE + 8),
                dict(k_rope=FAKE + 8), dict(out=FAKE + 8), dict(q_offsets=FAKE + 2), dict(k_offsets=FAKE + 2), dict(q_stride=188),
                dict(q_stride=196), dict(q_head_stride=184), dict(kv_stride=248), dict(kv_head_stride=260), dict(rope_stride=56),
                dict(rope_stride=66), dict(q_stride=1 << 39)):
        assert call(**bad) == -1, bad
    for big in (dict(Tq=2**31), dict(Tk=2**31), dict(Tq=2**31 - 1000, H=1024), dict(B=2**31 - 1, Tq=2**30), dict(B=2**24 + 1)):
        assert call(**big) == -2, big
    assert call(Tq=0, q=None, kv=None, out=None) == 0 and call(B=0, q=None) == 0


def on(device, *shape, dtype=BF):
    with FakeTensorMode():
        return torch.empty(*shape, dtype=dtype, device=device)


def decode(**other):
    t = {"q": on("cuda:0", 2, 16, 576), "cache": on("cuda:0", 8, 64, 576), "block_table": on("cuda:0", 2, 4, dtype=I32),
         "lengths": on("cuda:0", 2, dtype=I32), "scale": 0.1}
    return moe.latent_decode(**{**t, **other})


def attention(**other):
    t = {"q": on("cuda:0", 8, 4, 192), "kv": on("cuda:0", 9, 4, 256), "k_rope": on("cuda:0", 9, 64), "scale": 0.1,
         "q_offsets": on("cuda:0", 3, dtype=I32), "k_offsets": on("cuda:0", 3, dtype=I32)}
    return moe.latent_attention(**{**t, **other})


def calls(o):
    return {
        "attention kv": lambda: attention(kv=on(o, 9, 4, 256)),
        "attention k_rope": lambda: attention(k_rope=on(o, 9, 64)),
        "attention q_offsets": lambda: attention(q_offsets=on(o, 3, dtype=I32)),
        "attention k_offsets": lambda: attention(k_offsets=on(o, 3, dtype=I32)),
        "attention out": lambda: attention(out=on(o, 8, 4, 128)),
        "attention workspace": lambda: attention(workspace=on(o, 1 << 26, dtype=U8)),
        "decode cache": lambda: decode(cache=on(o, 8, 64, 576)),
        "decode block_table": lambda: decode(block_table=on(o, 2, 4, dtype=I32)),
        "decode lengths": lambda: decode(lengths=on(o, 2, dtype=I32)),
        "decode out": lambda: decode(out=on(o, 2, 16, 512)),
        "decode workspace": lambda: decode(workspace=on(o, 1 << 26, dtype=U8)),
    }


@pytest.mark.parametrize("other,message", [("cuda:1", "same GPU"), ("cpu", "GPU tensors")])
@pytest.mark.parametrize("name", list(calls("cpu")))
def test_operands_elsewhere_are_refused(name, other, message):
    with pytest.raises(ValueError, match=message):
        calls(other)[name]()


FILES = sorted(glob.glob(os.path.join(CSRC, "latent*.cu*")))


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
@pytest.mark.parametrize("what", [r"__ldg\b", r"ld\.global(\.\w+)*\.nc\b", r"__restrict__"])
def test_no_read_only_loads(path, what):
    assert not re.search(what, code(path))
