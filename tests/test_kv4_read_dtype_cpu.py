"""kv4_read's type: ``dtype``, else that of whichever output is given, else
bf16. Asked of a cache in host memory, which the call refuses last of all."""

import pytest
import torch

from sequence_exact_attention_gb300 import binding

F32, BF16 = torch.float32, torch.bfloat16


def read(**kw):
    cache = binding.kv4_cache(1, 2, 16, 64, "cpu")
    return binding.kv4_read(cache, None, 3, **kw)


def out(dtype):
    return torch.zeros(1, 3, 2, 64, dtype=dtype)


@pytest.mark.parametrize("kw", [dict(), dict(k=out(F32)), dict(v=out(F32)), dict(v=out(BF16)), dict(dtype=F32),
                                dict(k=out(F32), v=out(F32)), dict(dtype=F32, v=out(F32))])
def test_one_type_is_taken(lib, kw):
    with pytest.raises(ValueError, match="CUDA"):
        read(**kw)


@pytest.mark.parametrize("kw", [dict(k=out(F32), v=out(BF16)), dict(k=out(BF16), v=out(F32)),
                                dict(dtype=F32, v=out(BF16)), dict(dtype=BF16, k=out(F32))])
def test_two_types_are_refused(lib, kw):
    with pytest.raises(ValueError, match="must be torch"):
        read(**kw)
