"""GPU checks of the paged 8-bit cache at calls that its first tests leave out: repeated calls with others between, slots
of a page with gaps, far-off query sizes, warps with many jobs, and page ids that do not fit."""
import numpy as np
import pytest
import torch

from oracle import paged_cache as pc
from tests.paged_util import decode_bounds, random_cache
from tests.test_gpu_paged import _store_both

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


def _call_decode(a):
    import shared_prefix_packed_b200 as pp
    pp.pp_paged_decode(*a)
    pp.pp_get_status()


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


@pytest.mark.parametrize("top,k_exp", [(127, -126), (126, -126), (125, -124), (-120, 118), (-126, 120)])
def test_decode_queries_at_the_ends_of_bf16(top, k_exp):
    """Rows whose largest |q| lies in [2^top, 2^(top + 1)), with key scales that make their scores ordinary."""
    num, lens, page, hq, hkv = [2, 1], [40, 10, 20, 5, 130], 32, 4, 2
    c = random_cache(num, lens, page, hkv, "e4m3", 9)
    c["k_scale"][:] = 2.0 ** k_exp
    x = np.random.default_rng(3).standard_normal((3, hq, 128)) / 4
    x = np.where(np.abs(x) < 2.0 ** -6, 0, x)                # no element that f16 would lose bits of
    x[:, :, 7] = 1.9
    q = torch.from_numpy(x * 2.0 ** top).to(torch.bfloat16)
    assert torch.isfinite(q.float()).all()
    a = _decode_args(c, hq, 0, q)
    _call_decode(a)
    want = pc.decode(q.double().numpy(), c["k_vals"], c["v_vals"], c["k_scale"].astype(np.float64),
                     c["v_scale"].astype(np.float64), num, lens, c["table"])
    assert 1 < np.abs(want[3]).max() < 1e4
    bo, bl = decode_bounds(*want, n_keys=sum(lens), scale_exp=7)
    assert np.all(np.abs(a[9].double().cpu().numpy() - want[0]) <= bo)
    assert np.all(np.abs(a[10].double().cpu().numpy() - want[1]) <= bl)


def test_decode_scores_beyond_fp32_beside_low_ones():
    """A segment whose scores all pass fp32's range to -inf weighs nothing, however low the other segment's scores are; alone it
    has no softmax."""
    import shared_prefix_packed_b200 as pp
    page, n = 64, 64
    vals = np.zeros((2, 1, page, 128))
    vals[0, 0, :, 1] = np.arange(64) / 8 + 24                # the prefix: scores of some -1300
    vals[1, 0, :, 0] = -448                                  # the response: below -2^128
    k = torch.from_numpy(vals).float().to(torch.float8_e4m3fn).cuda()
    v_vals = np.random.default_rng(1).integers(-8, 9, (2, 1, 128, page)).astype(np.float64)
    v = torch.from_numpy(v_vals).float().to(torch.float8_e4m3fn).cuda()
    sk, sv = torch.tensor([[2.0 ** -106], [1.0]], device="cuda"), torch.ones(2, 1, device="cuda")
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0], q[0, 0, 1] = 2.0 ** 127, -2.0 ** 115
    o, lse = torch.empty_like(q), torch.empty(1, 1, device="cuda")
    ws = torch.empty(pp.pp_paged_decode_bytes(1, 1, 1), dtype=torch.uint8, device="cuda")
    for lens, seen in (([n, n], True), ([n, 0], True), ([0, n], False)):
        pp.pp_paged_decode(q, k, v, sk, sv, t([0, 2]), t([0, 0]), t(lens), t([[0], [1]]), o, lse, ws)
        pp.pp_get_status()
        if not seen:
            assert torch.isnan(o.float()).all() and torch.isneginf(lse).all()
            continue
        x = -(2.0 ** 9) * k[0, 0, :, 1].float().double().cpu().numpy() / 128 ** 0.5
        z = np.max(x) + np.log(np.sum(np.exp(x - np.max(x))))
        p = np.exp(x - z)
        want, spread = v_vals[0, 0] @ p, np.abs(v_vals[0, 0]) @ p
        bo, bl = decode_bounds(want[None, None], np.array([[z]]), spread[None, None], np.array([[np.max(np.abs(x))]]), n, 1)
        assert np.all(np.abs(o.double().cpu().numpy() - want) <= bo) and np.abs(lse.item() - z) <= bl[0, 0]


def test_decode_many_jobs_to_a_warp():
    """83,616 jobs, some 47 to each of 1776 warps, so that every warp decodes its jobs in three or four lots of 16; jobs of
    up to 8 and of up to 16 query rows, items that end inside a lot, that are cut between warps, and of one job."""
    import shared_prefix_packed_b200 as pp
    num, lens, page, r, hkv = [3, 1], [60000, 30000, 7, 12000, 45000, 20000], 128, 4, 32
    gen = torch.Generator(device="cuda").manual_seed(3)
    pages = [-(-n // page) for n in lens]
    total = sum(pages)
    k, v = (torch.randint(-127, 128, s, generator=gen, device="cuda", dtype=torch.int8) for s in ((total, hkv, page, 128), (total, hkv, 128, page)))
    sk, sv = (2.0 ** torch.randint(lo, lo + 3, (total, hkv), generator=gen, device="cuda").float() for lo in (-8, -6))
    ids, at = torch.randperm(total, generator=gen, device="cuda").to(torch.int32), 0
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32, device="cuda")
    for s, n in enumerate(pages):
        table[s, :n] = ids[at:at + n]
        at += n
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    q = torch.randn(4, r * hkv, 128, generator=gen, device="cuda").to(torch.bfloat16)
    o, lse = torch.empty_like(q), torch.empty(r * hkv, 4, device="cuda")
    ws = torch.empty(pp.pp_paged_decode_bytes(4, r * hkv, hkv), dtype=torch.uint8, device="cuda")
    pp.pp_paged_decode(q, k, v, sk, sv, t([0, 4, 6]), t([0] * 4 + [1] * 2), t(lens), table, o, lse, ws)
    pp.pp_get_status()
    for i, segs in enumerate(((0, 1), (0, 2), (0, 3), (4, 5))):
        place = [(table[s].long()[torch.arange(lens[s], device="cuda") // page], torch.arange(lens[s], device="cuda") % page) for s in segs]
        pg, off = (torch.cat(x) for x in zip(*place))
        for h in range(hkv):
            kk = k[pg, h, off].double() * sk[pg, h][:, None].double()
            vv = v[pg, h, :, off].double() * sv[pg, h][:, None].double()
            qq = q[i, r * h:r * h + r].double()
            x = qq @ kk.T / 128 ** 0.5
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - z[:, None])
            size = (qq.abs() @ kk.abs().T / 128 ** 0.5).amax(-1)
            want, spread = p @ vv, p @ vv.abs()
            bo, bl = decode_bounds(*(y.cpu().numpy() for y in (want, z, spread, size)), sum(lens), 6)
            got, got_l = o[i, r * h:r * h + r].double(), lse[r * h:r * h + r, i].double()
            assert np.all((got - want).abs().cpu().numpy() <= bo) and np.all((got_l - z).abs().cpu().numpy() <= bl)


def test_cache_keeps_its_device():
    """A cache made on "cuda" stays on the device that was current then."""
    import shared_prefix_packed_b200 as pp
    cache = pp.PagedCache([1], 4, 2, 4, 64)
    assert cache.device == cache.k_pages.device == torch.device("cuda", torch.cuda.current_device())
    for stream in (None, torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        slots, pos, counts = cache.resize([5, 3], stream=stream)
        torch.cuda.synchronize()
        assert slots.device == cache.device and counts[3] == 1
        cache.resize([0, 0], stream=stream)
        torch.cuda.synchronize()


# ------------------------------------------------------------------------------------------------------------- append
def _rows(rng, n, heads, dtype):
    """Rows of far-apart sizes, so that each decides a scale of its own."""
    size = np.exp(rng.uniform(-6, 6, (n, heads, 1)))
    return [torch.from_numpy(rng.standard_normal((n, heads, 128)) * size).to(dtype).cuda() for _ in range(2)]


APART = {                                                    # slots of page 1, as offsets; None skips a row
    "a gap": [3, 5],
    "a gap from the start": [0, 1, 3, 4],
    "a skipped row": [3, None, 4],
    "skipped rows and gaps": [1, None, None, 4, 5, 6, 7, 8, 9, None, 12],
    "descending": [9, 7, 3, 2],
    "the smallest last": [5, 6, 7, 8, 9, 10, 0],
    "twice": [4, 4, 6, 5, 6],
    "as far apart as may be": [2] + [None] * 255 + [3, 9],
    "again and again": ([2] + [None] * 200) * 3 + [8, 9, 10, 11, 12, 13],
}


@pytest.mark.parametrize("dtype,page,codes", [(torch.bfloat16, 16, "e4m3"), (torch.float32, 64, "int8"), (torch.bfloat16, 128, "int8")])
@pytest.mark.parametrize("what", list(APART))
def test_store_rows_of_a_page_apart(what, dtype, page, codes):
    """Rows of one page with gaps between their slots, skipped rows between them, or in another order are one append: one
    scale over all of them, alone in a call, behind other pages' rows, and where a block's window of 8 rows ends."""
    rng = np.random.default_rng(len(what))
    mine = [-1 if o is None else page + o for o in APART[what]]
    for before in ([], [0, 1, 2, 3, 4], [page * 3 + page - 1, -1, -1, 2 * page, 2 * page + 1]):
        slots = before + mine + [-1, 4 * page, 4 * page + 1, 4 * page + 2]
        _store_both(*_rows(rng, len(slots), 3, dtype), slots, page, 5, codes, 3)


@pytest.mark.parametrize("dtype,page,codes", [(torch.bfloat16, 16, "int8"), (torch.bfloat16, 64, "e4m3"), (torch.float32, 32, "e4m3"),
                                              (torch.bfloat16, 128, "e4m3")])
def test_store_many_rows_apart(dtype, page, codes):
    """Enough rows for windows of a page: whole pages, runs and pages with gaps, their rows across the windows' ends,
    stretches of skipped rows, and the end of a call inside a page."""
    rng = np.random.default_rng(page)
    slots, num_pages = [], 4000 // page + 200
    for pg in rng.permutation(num_pages):
        if len(slots) > 4000:
            break
        first = int(rng.integers(0, page)) if rng.random() < 0.5 else 0
        take = np.arange(first, int(rng.integers(first, page)) + 1)
        kind = rng.integers(0, 4)
        if kind == 1:
            take = take[rng.random(len(take)) < 0.7]
        if kind == 2:
            take = rng.permutation(take)
        for o in take:
            slots.append(int(pg) * page + int(o))
            if kind == 3 and rng.random() < 0.2:
                slots += [-1] * int(rng.integers(1, 4))
        if rng.random() < 0.1:
            slots += [-1] * int(rng.integers(1, 400))
    _store_both(*_rows(rng, len(slots), 3, dtype), slots, page, num_pages, codes, 5)


# ------------------------------------------------------------------------------------------------------------- resize
def _resize_args(old, new, table, free, n_free, page, capacity):
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    n = t([n_free])
    return [t([0, len(old)]), t([0] * len(old)), t(old), t(new), page, t(table), t(free), n, n, t([9] * capacity), t([9] * capacity), t([9] * 4)]


@pytest.mark.parametrize("bad", [-1, 12, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("new", [[3, 0, 20], [3, 0, 60], [3, 16, 20]])
def test_resize_refuses_to_take_back_pages_outside_the_pool(new, bad):
    """A shrinking segment whose row names a page that the pool does not have: nothing changes, and it is reported."""
    import shared_prefix_packed_b200 as pp
    old, table, free = [3, 40, 20], [[0, -1, -1, -1], [1, 2, bad, -1], [3, 4, -1, -1]], [5, 6, 7, 8, 9, 10, 11, -5, -5, -5, -5, -5]
    a = _resize_args(old, new, table, free, 7, 16, 50)
    pp.pp_pages_resize(*a)
    with pytest.raises(pp.PPError, match="cache pages"):
        pp.pp_get_status()
    assert a[11].tolist() == [0] * 4 and a[8].tolist() == [7] and (a[9] == -1).all() and (a[10] == 0).all()
    assert a[5].tolist() == table and a[6].tolist() == free
    a[5][1, 2] = 11                                          # (and no longer on the free list)
    a[7].fill_(6)
    pp.pp_pages_resize(*a)                                   # the next call, with a row that fits, is made
    assert a[11].tolist()[3] == 1
    pp.pp_get_status()


@pytest.mark.parametrize("new,n_free,capacity,word", [
    ([3, 40, 100], 4, 99, "more pages or slots"), ([3, 40, 60], 7, 30, "more pages or slots"), ([3, -1, 20], 7, 99, "cache pages"),
    ([3, 40, 100], 13, 99, "cache pages"), ([3, -1, 100], 4, 99, "cache pages"),
])
def test_resize_tells_a_full_pool_from_bad_input(new, n_free, capacity, word):
    import shared_prefix_packed_b200 as pp
    table = [[0] + [-1] * 7, [1, 2, 3] + [-1] * 5, [4, 5] + [-1] * 6]
    free = [6, 7, 8, 9, 10, 11, 12, -5, -5, -5, -5, -5]
    a = _resize_args([3, 40, 20], new, table, free, n_free, 16, capacity)
    pp.pp_pages_resize(*a)
    with pytest.raises(pp.PPError, match=f"DEVICE_INPUT.*{word}"):
        pp.pp_get_status()
    assert a[11].tolist() == [0] * 4 and a[8].tolist() == [n_free] and a[5].tolist() == table and a[6].tolist() == free


@pytest.mark.parametrize("at", [None, 0, 1023, 1024, 5000, 8999])
def test_resize_takes_back_many_pages_or_none(at):
    """9,000 pages given back, more than one CTA of the cluster looks at: all or, with one that does not fit, none."""
    import shared_prefix_packed_b200 as pp
    table = np.random.default_rng(3).permutation(9000).reshape(3000, 3)
    if at is not None:
        table[at // 3, at % 3] = 9000
    free = [-7] * 9000
    a = _resize_args([40] * 3000, [0] * 3000, table.tolist(), free, 0, 16, 5)
    pp.pp_pages_resize(*a)
    if at is None:
        pp.pp_get_status()
        assert a[11].tolist() == [0, 0, 9000, 1] and a[6].tolist() == table.reshape(-1).tolist() and a[8].item() == 9000
    else:
        with pytest.raises(pp.PPError, match="cache pages"):
            pp.pp_get_status()
        assert a[11].tolist() == [0] * 4 and a[6].tolist() == free and a[8].item() == 0
    assert a[5].tolist() == table.tolist()


@pytest.mark.parametrize("hq,hkv", [(32, 8), (28, 4)])
def test_decode_one_long_response_among_many_short(hq, hkv):
    """More than 2304 heads in all, so a warp of the second kernel takes a head, of which some have many records: a long
    prefix with one response, a long response behind a short prefix, responses of nothing beside them."""
    num = [1, 2] + [7] * 12
    lens = [9000, 40, 64, 7000, 0] + [x for _ in range(12) for x in [33] + [20, 0, 64, 65, 1, 130, 7]]
    c = random_cache(num, lens, 64, hkv, "int8", 12)
    n = sum(num)
    assert n * hq > 2304
    a = _decode_args(c, hq, 4)
    _call_decode(a)
    q = a[0]
    want = pc.decode(q.double().cpu().numpy(), c["k_vals"], c["v_vals"], c["k_scale"].astype(np.float64),
                     c["v_scale"].astype(np.float64), num, lens, c["table"])
    bo, bl = decode_bounds(*want, n_keys=sum(lens), scale_exp=7)
    assert np.all(np.abs(a[9].double().cpu().numpy() - want[0]) <= bo)
    assert np.all(np.abs(a[10].double().cpu().numpy() - want[1]) <= bl)


def test_cache_lengths_follow_only_changes_that_are_made():
    """PagedCache.lens after a change that is made, one that is refused, and one captured into a graph of which both are
    replayed; the lengths given are not written to."""
    import shared_prefix_packed_b200 as pp
    cache = pp.PagedCache([2], 4, 2, 6, 64, 16)
    new = torch.tensor([20, 3, 1], dtype=torch.int32, device="cuda")
    assert cache.resize(new, 64)[2].tolist() == [24, 4, 0, 1] and cache.lens.tolist() == [20, 3, 1]
    assert cache.resize([20, 40, 40], 64)[2].tolist() == [0] * 4 and cache.lens.tolist() == [20, 3, 1]      # 7 pages
    with pytest.raises(pp.PPError, match="more pages or slots"):
        pp.pp_get_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        counts = cache.resize(new, 64)[2]
    for lens, made in (([20, 17, 1], True), ([50, 50, 50], False), ([0, 17, 33], True), ([0, 0, 0], True)):
        was = cache.lens.tolist()
        new.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert counts[3].item() == made and cache.lens.tolist() == (lens if made else was) and new.tolist() == lens
    assert cache.n_free.item() == 6
    with pytest.raises(pp.PPError, match="more pages or slots"):
        pp.pp_get_status()


def test_rollout_from_lists_of_lengths():
    """A prefill and single steps with the lengths as lists: the rows are as many as the capacity, which by default is the
    sum of the lengths, and a step names it."""
    import shared_prefix_packed_b200 as pp
    hq, hkv = 8, 2
    cache = pp.PagedCache([2, 3], hq=hq, hkv=hkv, num_pages=40, max_tokens=256)
    wq, wk = (torch.ones(128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens = [100, 0, 0, 70, 0, 0, 0]

    def put(slots, pos):
        n = slots.numel()
        x = torch.randn(n, hq + 2 * hkv, 128, device="cuda").to(torch.bfloat16)
        q, k = torch.empty(n, hq, 128, dtype=x.dtype, device="cuda"), torch.empty(n, hkv, 128, dtype=x.dtype, device="cuda")
        pp.pp_qk_norm_rope(x[:, :hq], x[:, hq:hq + hkv], wq, wk, pos, q, k)
        cache.append(k, x[:, hq + hkv:], slots)
        return q

    slots, pos, counts = cache.resize(lens)
    assert slots.numel() == 170 and counts.tolist() == [170, 4, 0, 1]
    put(slots, pos)
    for _ in range(3):
        lens = [n + (i not in (0, 3)) for i, n in enumerate(lens)]
        slots, pos, counts = cache.resize(lens, capacity=5)
        q = put(slots, pos)
        o, lse = cache.decode(q)
        assert counts.tolist()[0] == 5 and torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
    assert pos.tolist() == [102, 102, 72, 72, 72]
    pp.pp_get_status()
