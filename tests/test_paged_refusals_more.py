"""CPU checks of calls of the q/k norm and the paged cache that the first refusal tests leave out."""
import pytest
import torch

from shared_prefix_packed_b200 import _lib
from tests.test_paged_refusals import BWD, DECODE, NORM, P, RESIZE, STORE, _call


def _cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("ws", [torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 12, 2, dtype=torch.uint8)[:, 0]])
def test_workspace_must_own_its_bytes(ws):
    """A broadcast or strided tensor counts more bytes than it holds in one piece."""
    kp, vp = _cpu(4, 2, 16, 128, dtype=torch.int8), _cpu(4, 2, 128, 16, dtype=torch.int8)
    f = lambda *s: _cpu(*s, dtype=torch.float32)
    i = lambda *s: _cpu(*s, dtype=torch.int32)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        _lib.pp_paged_decode(_cpu(2, 4, 128), kp, vp, f(4, 2), f(4, 2), i(2), i(3), i(3), i(3, 2), _cpu(2, 4, 128), f(4, 2), ws)
    x = f(3, 4, 64)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        _lib.pp_qk_norm_rope_bwd(x, x, None, None, i(3), x, x, x, x, None, None, ws)


@pytest.mark.parametrize("name,base,args", [
    ("pp_qk_norm_rope", NORM, ["pos"]),
    ("pp_qk_norm_rope_bwd", BWD, ["pos", "dwq", "dwk"]),
    ("pp_pages_resize", RESIZE, ["gs", "sg", "old", "new", "table", "free", "nin", "nout", "slots", "pos", "counts"]),
    ("pp_cache_store", STORE, ["slots", "ksc", "vsc"]),
    ("pp_paged_decode", DECODE, ["ksc", "vsc", "gs", "sg", "lens", "table", "lse"]),
])
def test_words_must_be_aligned(name, base, args):
    """An int32 or float array at an address that the GPU could not read it from."""
    for arg in args:
        for off in (1, 2):
            st, msg = _call(name, base, **{arg: P + off})
            assert st == "PP_ERR_INVALID_ARG" and "4-byte aligned" in msg, (arg, msg)


def test_streams_of_another_device():
    """The calls that allocate for themselves refuse them, as the plain calls do."""
    class Stream:
        device, cuda_stream = torch.device("cuda:1"), 0

    with pytest.raises(ValueError, match="the stream is of cuda:1, the tensors of cuda:0"):
        _lib.stream_scope(torch.device("cuda:0"), Stream())
