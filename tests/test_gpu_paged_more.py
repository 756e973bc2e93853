"""GPU checks of the paged 8-bit cache at calls that its first tests leave out: repeated calls with others between, slots
of a page with gaps, far-off query sizes, warps with many jobs, and page ids that do not fit."""
import numpy as np
import pytest
import torch

from tests.paged_util import random_cache

pytestmark = pytest.mark.gpu


def _decode_args(c, hq, seed, q=None):
    """A cache and its queries on the GPU, with outputs and scratch of their own."""
    import shared_prefix_packed_b200 as pp
    n = int(c["start"][-1]) - (len(c["start"]) - 1)
    if q is None:
        q = torch.from_numpy(1.5 * np.random.default_rng(seed).standard_normal((n, hq, 128))).to(torch.bfloat16)
    d = {k: c[k].cuda() for k in ("k", "v", "start", "seg_group", "lens_t", "table_t")}
    sk, sv = (torch.from_numpy(c[x]).cuda() for x in ("k_scale", "v_scale"))
    ws = torch.empty(pp.pp_paged_decode_bytes(n, hq, sk.shape[1]), dtype=torch.uint8, device="cuda")
    return [q.cuda(), d["k"], d["v"], sk, sv, d["start"], d["seg_group"], d["lens_t"], d["table_t"],
            torch.empty(n, hq, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(hq, n, device="cuda"), ws]


@pytest.mark.parametrize("num,lens,heads,page,codes", [
    ([1], [37, 19], (32, 8), 16, "e4m3"),
    ([4, 4], [1400, 70, 33, 64, 1, 900, 5, 0, 128, 257], (28, 4), 128, "int8"),
    ([8, 8, 8], [300] + [90] * 8 + [500] + [11] * 8 + [65] + [200] * 8, (32, 8), 64, "e4m3"),
])
def test_decode_repeats_bit_for_bit(num, lens, heads, page, codes):
    """The same inputs give the same bits, with a call on other inputs and the same scratch between."""
    import shared_prefix_packed_b200 as pp
    hq, hkv = heads
    a = _decode_args(random_cache(num, lens, page, hkv, codes, 1), hq, 2)
    b = _decode_args(random_cache(num, [n // 2 for n in lens], page, hkv, codes, 3), hq, 4)
    b[11] = a[11]
    pp.pp_paged_decode(*a)
    o, lse = a[9].clone(), a[10].clone()
    for i in range(12):
        if i % 2:
            pp.pp_paged_decode(*b)
        a[9].fill_(7)
        a[10].fill_(7)
        pp.pp_paged_decode(*a)
        assert torch.equal(a[9], o) and torch.equal(a[10], lse)
    pp.pp_get_status()
