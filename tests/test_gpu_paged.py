"""The paged KV cache's kernels against plain 64-bit forms (tests/_paged_ref.py):
append, attention, gather and scatter, alone and as a program runs them."""
import math
import sys

import pytest
import torch

from tests import _paged_ref as ref
from tests._paged_ref import BF16, E5M2, RAW, TORCH, Setup

pytestmark = pytest.mark.gpu

DIMS = (64, 80, 96, 128, 256)
MARK = 0x5A   # bytes of outputs before a call


def say(*a):
    print("[gpu-case]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def paged():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from fp8_kv_cache_amd import paged
    return paged


def up(x):
    """To the GPU with the same strides."""
    if x.dim() == 4 and not x.is_contiguous():
        raw = x.view(torch.uint8 if x.element_size() == 1 else torch.int16)
        return raw.transpose(1, 2).cuda().transpose(1, 2).view(x.dtype)
    return x.cuda()


def down(x):
    return (x.view(torch.uint8) if x.dtype == torch.float8_e5m2 else x).cpu().view(x.dtype)


def bits(x):
    return x.view(RAW[BF16] if x.element_size() == 2 else RAW[E5M2])


def handles(paged, st, max_tokens=None, max_kv=None):
    cache = paged.PagedCache(up(st.k), up(st.v))
    batch = paged.PageBatch(st.table.cuda(), st.cu.cuda(), st.kv_lens.cuda(), st.total,
                            max(st.new) if max_tokens is None else max_tokens, max(st.kv) if max_kv is None else max_kv)
    return cache, batch, torch.zeros(1, dtype=torch.int32, device="cuda")


def marked(shape, dtype=torch.bfloat16):
    n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
    return torch.full((n,), MARK, dtype=torch.uint8, device="cuda").view(dtype).view(shape)


def check_attention(paged, st, heads, q=None, workspace=None, expect_status=0, handle=None, **kw):
    q = st.rows(heads) if q is None else q
    cache, batch, status = handle or handles(paged, st)
    out = marked(q.shape)
    got, lse = paged.attention(cache, batch, q.cuda() if not q.is_cuda else q, out=out, return_lse=True, status=status,
                               workspace=workspace, **kw)
    torch.cuda.synchronize()
    want, want_lse, spread, wide = ref.attention(st, q.cpu(), **kw)
    tol, tol_lse = ref.attention_tolerance(st, q.cpu(), want, spread, wide)
    used = int(st.cu[-1])
    assert (down(got)[used:].view(torch.uint8) == MARK).all(), "a row of padding was written"
    got, lse = down(got)[:used].double(), lse.cpu()[:used].double()
    assert torch.isfinite(got).all()
    worst = ((got - want[:used]).abs() / tol[:used].clamp(min=1e-300)).max() if used else 0
    assert worst <= 1, f"out: {float(worst):.3f} of the bound"
    empty = want_lse[:used] == -math.inf
    assert torch.equal(lse == -math.inf, empty) and (got[empty] == 0).all()
    off = (lse - want_lse[:used]).abs()[~empty]
    bound = (tol_lse[:used] + want_lse[:used].abs() * 2.0 ** -22)[~empty]
    assert (off <= bound).all(), f"lse: {float((off / bound).max()):.3f} of the bound"
    assert int(status) == expect_status
    return got


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("heads", [(8, 2), (3, 3), (40, 2)])
def test_single_tokens(paged, dim, dtype, heads):
    """One new token each, lengths on both sides of a block, a page and a split."""
    kv = [1, 2, 31, 32, 33, 127, 128, 129, 257, 600]
    say("single tokens", dim, dtype, heads)
    st = Setup([1] * len(kv), kv, heads[1], dim, dtype, seed=dim + dtype)
    check_attention(paged, st, heads[0])


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("new,kv", [([5, 3, 1, 8], [5, 40, 300, 90]), ([70, 1, 0, 33], [70, 515, 12, 200]),
                                    ([131], [260])])
def test_chunks(paged, dim, dtype, new, kv):
    say("chunks", dim, dtype, new, kv)
    check_attention(paged, Setup(new, kv, 2, dim, dtype, pad=3, seed=7 * dim + dtype), 8)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("page", [1, 2, 8, 32, 64, 256])
@pytest.mark.parametrize("head_major", [False, True])
def test_page_sizes_and_orders(paged, page, head_major, dtype):
    say("pages", page, head_major, dtype)
    st = Setup([1, 40, 3], [333, 150, 64], 2, 64, dtype, page=page, head_major=head_major, seed=page)
    check_attention(paged, st, 4)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("window", [1, 2, 16, 33, 64, 100, 1000])
def test_windows(paged, window, dtype):
    """The pages that a window has left behind may be gone from the table."""
    say("window", window, dtype)
    st = Setup([1, 50, 4, 140], [500, 300, 64, 140], 2, 64, dtype, seed=window)
    want = st.table.clone()
    for s, n in enumerate(st.kv):
        gone = max(0, n - st.new[s] + 1 - window) // st.page
        want[s, :gone] = -1
    full, st.table = st.table, want
    handle = handles(paged, st)
    st.table = full
    check_attention(paged, st, 8, handle=handle, window=window)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_not_causal(paged, dtype):
    say("not causal", dtype)
    check_attention(paged, Setup([1, 50, 7], [500, 130, 7], 2, 128, dtype), 8, causal=False)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 16, 17, 33, 64])
def test_groups(paged, group):
    say("group", group)
    check_attention(paged, Setup([1, 6, 2], [90, 130, 2], 3, 64, BF16, seed=group), 3 * group)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_rows_without_keys(paged, dtype):
    """No cached token at all, more new tokens than cached ones, and no new ones."""
    say("rows without keys", dtype)
    check_attention(paged, Setup([1, 3, 0, 2, 40], [0, 1, 9, 0, 30], 2, 64, dtype, pad=2), 4)
    check_attention(paged, Setup([1, 3, 0, 2, 40], [0, 1, 9, 0, 30], 2, 64, dtype, pad=2), 4, causal=False)


def test_one_key_gives_its_value(paged):
    say("one key")
    st = Setup([1, 1], [1, 1], 1, 64, BF16)
    got = check_attention(paged, st, 2)
    for s in range(2):
        assert torch.equal(got[s, 0], st.sequence(st.v, s)[0, 0])


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("seqs", [1, 70, 300])
def test_many_sequences(paged, seqs, dtype):
    say("sequences", seqs, dtype)
    g = torch.Generator().manual_seed(seqs)
    kv = torch.randint(0, 60, (seqs,), generator=g).tolist()
    new = [int(min(n, torch.randint(0, 4, (1,), generator=g))) for n in kv]
    check_attention(paged, Setup(new, kv, 1, 64, dtype, page=8, pad=5, seed=seqs), 2)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("new,kv", [([1], [9000]), ([1, 1], [40, 5000]), ([2], [4097])])
def test_long_lengths_are_split_and_joined(paged, new, kv, dtype):
    say("long", new, kv, dtype)
    st = Setup(new, kv, 2, 128, dtype, page=64, seed=3)
    cache, batch, _ = handles(paged, st)
    assert paged.workspace_bytes(cache, batch, 8) > 0
    check_attention(paged, st, 8)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -20, 1.0, 100.0])
def test_query_sizes(paged, size, dtype):
    """Queries far from 1, with a scale that makes up for it; one-sided scores."""
    say("query size", size, dtype)
    st = Setup([1, 9], [70, 130], 2, 64, dtype)
    q = (st.rows(4).float() * size).to(torch.bfloat16)
    q[0, 0] = 0
    check_attention(paged, st, 4, q=q, scale=0.2 / size)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_peaked_scores(paged, dtype):
    """Scores in the hundreds, their maximum in the last block, then in the first."""
    say("peaked", dtype)
    for order in (1, -1):
        st = Setup([1, 40], [700, 300], 1, 64, dtype, seed=5)
        for s in range(2):
            for p in range(st.kv[s]):
                page, slot = st.place(s, p)
                size = 8.0 * (p + 1) / st.kv[s] if order > 0 else 8.0 * (1 - p / st.kv[s])
                st.k[page, slot] = torch.full((1, 64), size).to(st.k.dtype)
        check_attention(paged, st, 2, q=torch.full((41, 2, 64), 1.0, dtype=torch.bfloat16), scale=1.0)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("window", [0, 5])
@pytest.mark.parametrize("new", [3, 20, 150])
def test_what_a_row_does_not_see_never_reaches_it(paged, new, window, dtype):
    """Inf and NaN in keys and values that some rows of a tile see and
    others do not."""
    say("not seen", new, window, dtype)
    kv = new + 40
    st = Setup([new], [kv], 1, 64, dtype, seed=new)
    q = st.rows(2)
    special = {kv - new + 1: math.inf, kv - new // 2: -math.inf, kv - 1: math.nan}
    for p, x in special.items():
        page, slot = st.place(0, p)
        st.v[page, slot, 0, 3] = torch.tensor(x).to(st.v.dtype)
    page, slot = st.place(0, kv - 1)
    st.k[page, slot, 0, 5] = torch.tensor(math.nan).to(st.k.dtype)
    cache, batch, status = handles(paged, st)
    got = down(paged.attention(cache, batch, q.cuda(), window=window)).double()
    want = ref.attention(st, q, window=window)[0]
    plain = Setup([new], [kv], 1, 64, dtype, seed=new)
    clean = ref.attention(plain, q, window=window)
    tol = ref.attention_tolerance(plain, q, clean[0], *clean[2:])[0]
    assert torch.equal(torch.isfinite(got), torch.isfinite(want))
    fine = torch.isfinite(want)
    assert ((got - want).abs()[fine] <= tol[fine]).all()
    bad = ~fine & ~torch.isnan(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got[bad], want[bad])
    assert fine.any() and bad.any() and torch.isnan(want).any()


def test_strided_rows(paged):
    """q a view into a packed projection, out a view into a wider buffer."""
    say("strided rows")
    st = Setup([3, 1], [50, 90], 2, 80, BF16)
    packed = torch.randn(st.total, 12, 80, generator=st.g).to(torch.bfloat16).cuda()
    q, wide = packed[:, 2:10], marked((st.total, 10, 80))
    cache, batch, status = handles(paged, st)
    paged.attention(cache, batch, q, out=wide[:, 1:9], status=status)
    want, _, spread, sizes = ref.attention(st, q.cpu())
    tol, _ = ref.attention_tolerance(st, q.cpu(), want, spread, sizes)
    assert ((down(wide)[:, 1:9].double() - want).abs() <= tol).all()
    assert (wide[:, 0].contiguous().view(torch.uint8) == MARK).all() and (wide[:, 9].contiguous().view(torch.uint8) == MARK).all()


# ------------------------------------------------------------------ append

def _append_reference(st, k, v, q, table, interleaved, q_norm, k_norm, eps):
    """{name: (low, high)} of each output in 64 bits, rounded ends, and the written slots."""
    def ends(x, w, p):
        y = ref.norm(x, w, eps)
        # the norm's sum, root and products: dim + 6 roundings of 32 bits
        slack = y.abs() * ((st.dim + 6) * 2.0 ** -23 if w is not None else 0)
        if table is None:
            return y, slack
        z, size = ref.rotate(y, table, p, interleaved)
        spread = ref.rotate(slack, table.abs(), p, interleaved)[1]
        return z, spread + size * 3 * 2.0 ** -24   # two products and a sum
    out = {}
    for row, s, p in st.tokens():
        if p < 0:
            continue
        out[row] = (st.place(s, p), ends(k[row], k_norm, p), ends(q[row], q_norm, p))
    return out


def _between(got, y, slack, dtype):
    low, high = ref.round_to(y - slack, dtype), ref.round_to(y + slack, dtype)
    return ((got >= low) & (got <= high)).all()


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("dim,rotary", [(64, 64), (64, 16), (80, 32), (80, 80), (96, 96), (128, 128), (128, 64), (256, 256)])
@pytest.mark.parametrize("norms", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(paged, dim, rotary, dtype, norms, interleaved):
    say("append", dim, rotary, dtype, norms, interleaved)
    st = Setup([3, 1, 0, 5], [20, 1, 7, 3], 2, dim, dtype, pad=2, seed=dim + rotary)   # the last: two tokens without a place
    k, v, q = st.rows(2), st.rows(2), st.rows(5)
    table = torch.randn(20, rotary, generator=st.g)
    w = [(1 + 0.3 * torch.randn(dim, generator=st.g)).to(torch.bfloat16) for _ in range(2)] if norms else (None, None)
    cache, batch, status = handles(paged, st)
    before_k, before_v = down(cache.k).clone(), down(cache.v).clone()
    q_out = marked(q.shape)
    paged.append(cache, batch, k.cuda(), v.cuda(), q=q.cuda(), q_out=q_out, rope=paged.Rope(table.cuda(), interleaved),
                 q_norm=w[0].cuda() if norms else None, k_norm=w[1].cuda() if norms else None, eps=1e-5, status=status)
    torch.cuda.synchronize()
    got_k, got_v, got_q = down(cache.k), down(cache.v), down(q_out)
    want = _append_reference(st, k, v, q, table, interleaved, *w, 1e-5)
    for row, ((page, slot), kk, qq) in want.items():
        assert _between(got_k[page, slot].double(), *kk, TORCH[dtype]), ("k", row)
        assert _between(got_q[row].double(), *qq, torch.bfloat16), ("q", row)
        assert torch.equal(bits(got_v[page, slot]), bits(v[row].to(TORCH[dtype]))), ("v", row)
        for x, y in ((got_k, before_k), (got_v, before_v)):
            bits(x)[page, slot] = bits(y)[page, slot]
    assert torch.equal(bits(got_k), bits(before_k)) and torch.equal(bits(got_v), bits(before_v)), "another slot was written"
    rest = [r for r in range(st.total) if r not in want]
    assert (got_q[rest].view(torch.uint8) == MARK).all(), "a row without a place was written"
    assert int(status) == 0


@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_append_without_rotation_copies_bits(paged, dtype):
    """Every BF16 pattern as keys and values: into a BF16 cache bit for bit,
    into an E5M2 one rounded as torch rounds."""
    say("append patterns", dtype)
    n = 65536 // 64
    st = Setup([n], [n + 5], 1, 64, dtype)
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(n, 1, 64).view(torch.bfloat16)
    cache, batch, status = handles(paged, st)
    assert paged.append(cache, batch, x.cuda(), x.flip(0).cuda(), status=status) is None
    for pool, src in ((down(cache.k), x), (down(cache.v), x.flip(0))):
        got = torch.stack([pool[st.place(0, 5 + i)] for i in range(n)])
        want = src.to(TORCH[dtype])
        nan = torch.isnan(want.float())
        if dtype == BF16:
            assert torch.equal(bits(got), bits(want))
        assert torch.equal(torch.isnan(got.float()), nan)
        assert torch.equal(bits(got)[~nan], bits(want)[~nan])


def test_append_queries_in_place_and_strided(paged):
    """q, k and v views of one packed projection; the queries rotated where they are."""
    say("append in place")
    st = Setup([4, 2], [9, 2], 2, 64, BF16)
    packed = torch.randn(st.total, 8, 64, generator=st.g).to(torch.bfloat16)
    table = torch.randn(9, 64, generator=st.g)
    dev = packed.cuda()
    cache, batch, status = handles(paged, st)
    got = paged.append(cache, batch, dev[:, 4:6], dev[:, 6:], q=dev[:, :4], q_out=dev[:, :4], rope=paged.Rope(table.cuda()))
    assert got.data_ptr() == dev.data_ptr()
    want = _append_reference(st, packed[:, 4:6], None, packed[:, :4], table, False, None, None, 0.0)
    for row, ((page, slot), kk, qq) in want.items():
        assert _between(down(cache.k)[page, slot].double(), *kk, torch.bfloat16)
        assert _between(down(dev)[row, :4].double(), *qq, torch.bfloat16)
    assert torch.equal(down(dev)[:, 4:], packed[:, 4:])


def test_rope_table_far_positions(paged):
    say("rope table")
    t = paged.rope_table(200000, 64, base=1e6, device="cuda").cpu().double()
    for p in (0, 1, 131071, 199999):
        for i in (0, 1, 31):
            angle = p * 1e6 ** (-i / 32)
            # the angle in 64 bits is off by a few 2^-53 of it, the table's value by its rounding
            assert abs(t[p, i] - math.cos(angle)) <= 2.0 ** -24 + angle * 2.0 ** -50
            assert abs(t[p, 32 + i] - math.sin(angle)) <= 2.0 ** -24 + angle * 2.0 ** -50


# --------------------------------------------------------- gather, scatter

@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("dim,heads,page", [(64, 1, 16), (80, 3, 8), (128, 8, 64), (256, 2, 1), (96, 4, 16)])
def test_gather_and_scatter(paged, dim, heads, page, head_major, dtype):
    say("gather, scatter", dim, heads, page, head_major, dtype)
    new, kv = [30, 0, 5, 7, 1], [30, 6, 90, 3, 1]     # the fourth: four rows without a place
    st = Setup(new, kv, heads, dim, dtype, page=page, head_major=head_major, pad=2)
    for pool in (st.k, st.v):   # any bit pattern
        flat = bits(pool)
        flat.copy_(torch.randint(-(1 << 15), 1 << 15, flat.shape, generator=st.g).to(flat.dtype))
    cache, batch, status = handles(paged, st)
    shape = (st.total, heads, dim)
    k, v = marked(shape, TORCH[dtype]), marked(shape, TORCH[dtype])
    paged.gather(cache, batch, k, v, status=status)
    other = Setup(new, kv, heads, dim, dtype, page=page, head_major=not head_major, pad=2, seed=9)
    target, its_batch, _ = handles(paged, other)
    free_k, free_v = down(target.k).clone(), down(target.v).clone()
    paged.scatter(target, its_batch, k, v, status=status)
    torch.cuda.synchronize()
    for x, pool, landed, free in ((down(k), st.k, down(target.k), free_k), (down(v), st.v, down(target.v), free_v)):
        for row, s, p in st.tokens():
            if p < 0:
                assert (bits(x)[row] == 0).all()
                continue
            assert torch.equal(bits(x)[row], bits(pool)[st.place(s, p)])
            assert torch.equal(bits(landed)[other.place(s, p)], bits(pool)[st.place(s, p)])
            bits(landed)[other.place(s, p)] = bits(free)[other.place(s, p)]
        assert torch.equal(bits(landed), bits(free)), "another slot was written"
        assert (x[sum(new):].view(torch.uint8) == MARK).all(), "a row of padding was written"
    assert int(status) == 0


def test_gather_into_wider_rows(paged):
    say("gather strided")
    st = Setup([9], [9], 2, 64, BF16)
    cache, batch, _ = handles(paged, st)
    both = marked((9, 4, 64))
    paged.gather(cache, batch, both[:, :2], both[:, 2:])
    assert torch.equal(down(both)[:, :2].double(), st.sequence(st.k, 0))
    assert torch.equal(down(both)[:, 2:].double(), st.sequence(st.v, 0))


# ------------------------------------------------- bad tables and lengths

def test_bad_pages_are_masked_and_reported(paged):
    """Ids outside the pool and positions past the table's width: those keys
    are as if masked, appends and gathers of them do nothing, the status says so."""
    say("bad pages")
    for bad in (-1, 10 ** 6, 2 ** 31 - 1):
        st = Setup([1, 3], [100, 64], 2, 64, BF16, page=16)
        q = st.rows(4)
        cache, batch, status = handles(paged, st)
        table = st.table.clone()
        table[0, 2] = bad
        batch = paged.PageBatch(table.cuda(), st.cu.cuda(), st.kv_lens.cuda(), st.total, 3, 100)
        got = down(paged.attention(cache, batch, q.cuda(), status=status)).double()
        assert int(status) == 1
        # the same sequence without those keys (attention without order: the mask is by position alone)
        keep = Setup([1, 3], [100, 64], 2, 64, BF16, page=16)
        whole = [keep.sequence(p, 0) for p in (keep.k, keep.v)]
        kk, vv = (torch.cat([x[:32], x[48:]]) for x in whole)
        for h in range(4):
            w = torch.softmax(kk[:, h // 2] @ q[0, h].double() / 8, 0)
            tol = 2.0 ** -7 * (w[:, None] * vv[:, h // 2].abs()).sum(0) + 1e-3
            assert ((got[0, h] - (w[:, None] * vv[:, h // 2]).sum(0)).abs() <= tol).all()
        status.zero_()
        batch = paged.PageBatch(table.cuda(), torch.tensor([0, 100, 164], dtype=torch.int32).cuda(), st.kv_lens.cuda(), 164, 100, 100)
        k, v = paged.gather(cache, batch, status=status)
        assert int(status) == 1 and (k[32:48].view(torch.int16) == 0).all() and (v[32:48].view(torch.int16) == 0).all()
        assert torch.equal(down(k)[48:100].double(), whole[0][48:])
        status.zero_()
        before = bits(cache.k).clone()
        x = torch.zeros(164, 2, 64, dtype=torch.bfloat16, device="cuda")
        x[:32], x[48:] = k[:32], k[48:]
        paged.scatter(cache, batch, x, v, status=status)
        assert int(status) == 1 and torch.equal(bits(cache.k), before)


def test_bad_lengths_are_reported_and_touch_nothing(paged):
    say("bad lengths")
    st = Setup([2, 3, 2], [50, 64, 40], 2, 64, BF16)
    k, v, q = (st.rows(h).cuda() for h in (2, 2, 4))
    cache, _, status = handles(paged, st)
    good = paged.attention(cache, handles(paged, st)[1], q)
    pools = [bits(x).clone() for x in (cache.k, cache.v)]
    for cu, lens in (([0, 2, 5, 7], [50, 65, 40]), ([0, 2, 5, 7], [50, -1, 40]), ([0, 2, 5, 7], [50, 2 ** 31 - 1, 40])):
        batch = paged.PageBatch(st.table.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(),
                                torch.tensor(lens, dtype=torch.int32).cuda(), 7, 3, 64)
        out = marked(q.shape)
        status.zero_()
        paged.attention(cache, batch, q, out=out, status=status)
        assert int(status) == 1
        assert torch.equal(out[:2], good[:2]) and torch.equal(out[5:], good[5:])
        assert (out[2:5].contiguous().view(torch.uint8) == MARK).all()
        status.zero_()
        a, b = (marked((7, 2, 64)) for _ in range(2))
        paged.gather(cache, batch, a, b, status=status)
        assert int(status) == 1 and (a[2:5].contiguous().view(torch.uint8) == MARK).all()
        status.zero_()
        x = k.clone()
        x[:2], x[5:] = a[:2], a[5:]
        y = v.clone()
        y[:2], y[5:] = b[:2], b[5:]
        paged.scatter(cache, batch, x, y, status=status)
        assert int(status) == 1
        assert torch.equal(bits(cache.k), pools[0]) and torch.equal(bits(cache.v), pools[1])
    # token ranges that run backwards, past the rows, or are longer than the batch allows
    for cu in ([0, 5, 2, 7], [0, 2, 9, 7], [0, 2, 2 ** 31 - 1, 7], [-2 ** 31, 2, 5, 7], [0, 0, 7, 7]):
        batch = paged.PageBatch(st.table.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), st.kv_lens.cuda(), 7, 3, 64)
        for call in (lambda: paged.attention(cache, batch, q, status=status), lambda: paged.gather(cache, batch, status=status)):
            status.zero_()
            call()
            assert int(status) == 1, cu


def test_positions_past_the_rotation_table(paged):
    say("short rotation table")
    st = Setup([4], [20], 2, 64, BF16)
    k, v, q = (st.rows(h).cuda() for h in (2, 2, 4))
    cache, batch, status = handles(paged, st)
    before = bits(cache.k).clone()
    q_out = marked(q.shape)
    paged.append(cache, batch, k, v, q=q, q_out=q_out, rope=paged.Rope(torch.randn(18, 64).cuda()), status=status)
    assert int(status) == 1
    changed = (bits(cache.k) != before).flatten(2).any(2)
    assert [bool(changed[st.place(0, p)]) for p in (16, 17, 18, 19)] == [True, True, False, False]
    assert (q_out[2:].contiguous().view(torch.uint8) == MARK).all() and not (q_out[:2].contiguous().view(torch.uint8) == MARK).all()


# --------------------------------------------------- as a program runs them

@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_prefill_then_decode_equals_one_pass(paged, dtype):
    """A prompt appended and attended in chunks, then token by token, gives
    what the whole sequence in one call gives (to the roundings of each)."""
    say("prefill, decode", dtype)
    n, hk, hq, dim = 150, 2, 8, 64
    g = torch.Generator().manual_seed(1)
    k, v, q = ((torch.randn(n, h, dim, generator=g)).to(torch.bfloat16).cuda() for h in (hk, hk, hq))
    rope = paged.Rope(paged.rope_table(n, dim))
    table = torch.randperm(20, generator=g)[:10].to(torch.int32)[None].cuda()

    def run(steps):
        cache = paged.PagedCache.empty(20, 16, hk, dim, dtype)
        for pool in (cache.k, cache.v):
            bits(pool).fill_(-1)
        out, at = [], 0
        for step in steps:
            cu = torch.tensor([0, step], dtype=torch.int32).cuda()
            batch = paged.PageBatch(table, cu, torch.tensor([at + step], dtype=torch.int32).cuda(), step, step, at + step)
            rows = slice(at, at + step)
            turned = paged.append(cache, batch, k[rows], v[rows], q=q[rows], rope=rope)
            out.append(paged.attention(cache, batch, turned))
            at += step
        return cache, torch.cat(out)

    cache, whole = run([n])
    again, parts = run([37, 64, 1, 1, 1, 20, 1, 25])
    assert torch.equal(bits(cache.k), bits(again.k)) and torch.equal(bits(cache.v), bits(again.v))
    spread = v.float().abs().max()
    assert (whole.float() - parts.float()).abs().max() <= 4 * 2.0 ** -8 * spread


@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_layers_through_the_codec_into_other_pages(paged, dtype):
    """Pages -> layer tensors -> compressed streams -> decoded -> another
    cache's pages: the attention there is the same to the bit."""
    import fp8_kv_cache_amd as sz
    from fp8_kv_cache_amd import codec
    say("through the codec", dtype)
    st = Setup([70, 33], [70, 33], 2, 128, dtype, page=16)
    q = torch.randn(2, 8, 128, generator=st.g).to(torch.bfloat16).cuda()
    cache, batch, _ = handles(paged, st)
    other = Setup([70, 33], [70, 33], 2, 128, dtype, page=32, head_major=True, seed=4)
    target, its_batch, _ = handles(paged, other)
    landed = []
    for x in paged.gather(cache, batch):
        stream, _, _ = codec.compress(x, dtype)
        y, status = codec.decompress(stream, x.numel(), dtype)
        assert status == sz.SZ_OK
        landed.append(y.view(x.shape))
    paged.scatter(target, its_batch, *landed)
    one = torch.arange(3, dtype=torch.int32).cuda()
    outs = [paged.attention(c, paged.PageBatch(s.table.cuda(), one, s.kv_lens.cuda(), 2, 1, 70), q)
            for c, s in ((cache, st), (target, other))]
    assert torch.equal(*outs)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_graph_replays_a_decode_step(paged, dtype):
    """Append and attention captured once and replayed as the lengths grow
    (in place, inside the batch's bounds), each replay against eager calls."""
    say("graph", dtype)
    hk, hq, dim, most = 2, 8, 128, 2100
    table = torch.randperm(400).to(torch.int32).cuda()[:2 * 132].view(2, 132)
    cache = paged.PagedCache.empty(400, 16, hk, dim, dtype)
    for pool in (cache.k, cache.v):
        pool.copy_(torch.randn(pool.shape, device="cuda").to(torch.bfloat16).to(pool.dtype))
    twin = paged.PagedCache(cache.k.clone(), cache.v.clone())
    lens = torch.tensor([1000, 2040], dtype=torch.int32, device="cuda")
    cu = torch.arange(3, dtype=torch.int32, device="cuda")
    batch = paged.PageBatch(table, cu, lens, 2, 1, most)
    rope = paged.Rope(paged.rope_table(most, dim))
    k, v, q = (torch.zeros(2, h, dim, dtype=torch.bfloat16, device="cuda") for h in (hk, hk, hq))
    turned, out = torch.empty_like(q), torch.empty_like(q)
    space = torch.empty(max(16, paged.workspace_bytes(cache, batch, hq)), dtype=torch.uint8, device="cuda")

    def step(c, to, turned_to):
        paged.append(c, batch, k, v, q=q, q_out=turned_to, rope=rope)
        paged.attention(c, batch, turned_to, out=to, workspace=space)

    step(twin, out, turned)     # warm
    twin = paged.PagedCache(cache.k.clone(), cache.v.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, out, turned)
    for i in range(4):
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, device="cuda"))
        lens += 1
        eager, eager_turned = torch.empty_like(q), torch.empty_like(q)
        step(twin, eager, eager_turned)
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(turned, eager_turned)
        assert torch.equal(bits(cache.k), bits(twin.k)) and torch.equal(bits(cache.v), bits(twin.v))


def test_another_stream(paged):
    """Calls on a stream that is not the current one, as a Stream and as a
    handle; what they allocate belongs to it."""
    say("stream")
    st = Setup([1, 1], [3000, 900], 2, 128, BF16, page=64)
    q = st.rows(8).cuda()
    cache, batch, status = handles(paged, st)
    want = paged.attention(cache, batch, q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        outs = [paged.attention(cache, batch, q, stream=stream) for _ in range(3)]
        k, v = paged.gather(cache, batch, stream=stream)
        side.synchronize()
        assert all(torch.equal(x, want) for x in outs)
        assert torch.equal(k, paged.gather(cache, batch)[0])


def test_repeats_are_the_same_bits(paged):
    say("repeat")
    st = Setup([1, 60], [5000, 400], 2, 128, BF16, page=64)
    q = st.rows(8).cuda()
    cache, batch, _ = handles(paged, st)
    first = paged.attention(cache, batch, q, return_lse=True)
    for _ in range(3):
        again = paged.attention(cache, batch, q, return_lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_empty_calls_do_nothing(paged):
    say("empty")
    cache = paged.PagedCache.empty(2, 16, 2, 64)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    for seqs in (0, 2):
        batch = paged.PageBatch(torch.zeros(seqs, 1, dtype=torch.int32).cuda(), torch.zeros(seqs + 1, dtype=torch.int32).cuda(),
                                torch.zeros(seqs, dtype=torch.int32).cuda(), 0, 0, 0)
        paged.append(cache, batch, none, none, q=none)
        assert paged.attention(cache, batch, none).shape == (0, 2, 64)
        k, v = paged.gather(cache, batch)
        paged.scatter(cache, batch, k, v)
    # rows that no sequence has
    batch = paged.PageBatch(torch.zeros(0, 1, dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda(),
                            torch.zeros(0, dtype=torch.int32).cuda(), 3, 1, 1)
    out = marked((3, 2, 64))
    paged.attention(cache, batch, torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda"), out=out)
    assert (out.view(torch.uint8) == MARK).all()


def test_pools_past_four_gigabytes(paged):
    """Pages whose offsets need more than 32 bits (in bytes and in elements)."""
    say("large pool")
    pages = (5 << 30) // (16 * 8 * 128 * 2) + 7      # 5 GiB + of BF16
    k = torch.empty(pages, 16, 8, 128, dtype=torch.bfloat16, device="cuda")
    cache = paged.PagedCache(k, torch.empty_like(k))
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    x = torch.randn(40, 8, 128, device="cuda").to(torch.bfloat16)
    y = torch.randn(40, 8, 128, device="cuda").to(torch.bfloat16)
    one = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    batch = paged.PageBatch(table, one, one[1:].clone(), 40, 40, 40)
    paged.append(cache, batch, x, y)
    assert torch.equal(cache.k[pages - 1], x[:16]) and torch.equal(cache.v[pages - 2, :8], y[32:])
    a, b = paged.gather(cache, batch)
    assert torch.equal(a, x) and torch.equal(b, y)
    q = torch.randn(1, 8, 128, device="cuda").to(torch.bfloat16)
    out = paged.attention(cache, paged.PageBatch(table, torch.tensor([0, 1], dtype=torch.int32).cuda(), one[1:].clone(), 1, 1, 40), q)
    small = paged.PagedCache(torch.stack([cache.k[pages - 1], cache.k[0], cache.k[pages - 2]]),
                             torch.stack([cache.v[pages - 1], cache.v[0], cache.v[pages - 2]]))
    same = paged.attention(small, paged.PageBatch(torch.arange(3, dtype=torch.int32)[None].cuda(),
                                                  torch.tensor([0, 1], dtype=torch.int32).cuda(), one[1:].clone(), 1, 1, 40), q)
    assert torch.equal(out, same)


@pytest.mark.parametrize("compressed", [True, False])
@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_transfer_between_paged_caches(paged, dtype, compressed):
    """Three layers of two sequences to another machine's pages, whose next
    token then attends to the same bits."""
    from fp8_kv_cache_amd.transfer import PagedLink
    say("paged link", dtype, compressed)
    # one page table serves every layer
    sets = [Setup([70, 33], [70, 33], 2, 128, dtype, page=16, seed=0) for _ in range(3)]
    for i, st in enumerate(sets):
        g = torch.Generator().manual_seed(i)
        st.k, st.v = (torch.randn(x.shape, generator=g).to(torch.bfloat16).to(x.dtype) for x in (st.k, st.v))
    caches = [paged.PagedCache(up(st.k), up(st.v)) for st in sets]
    batch = handles(paged, sets[0])[1]
    other = Setup([70, 33], [70, 33], 2, 128, dtype, page=32, head_major=True, seed=8)
    targets = [handles(paged, other)[0] for _ in range(3)]
    its_batch = handles(paged, other)[1]
    link = PagedLink(3, 103, 2, 128, dtype, group=2)
    for _ in range(2):
        link.ship(caches, batch, targets, its_batch, compressed)
    if compressed:
        assert all(s == 0 for s in link.link.statuses()) and all(s == 0 for s in link.link.compress_statuses())
    for a, b in zip(caches, targets):
        for x, y in zip(paged.gather(a, batch), paged.gather(b, its_batch)):
            assert torch.equal(bits(x), bits(y))
    with pytest.raises(ValueError):
        link.ship(caches[:2], batch, targets[:2], its_batch)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("new,kv,window", [([150, 90], [151, 400], 0), ([70, 129], [70, 777], 100), ([260], [64 * 5], 0)])
def test_long_chunks(paged, dim, dtype, new, kv, window):
    """More rows a sequence than the smaller tiles take; one key tile, two,
    and odd and even numbers of them."""
    say("long chunks", dim, dtype, new, kv, window)
    check_attention(paged, Setup(new, kv, 1, dim, dtype, pad=1, seed=dim), 4, window=window)


@pytest.mark.parametrize("keys", [1, 63, 64, 65, 127, 128, 129, 192, 193])
def test_key_tiles_at_their_edges(paged, keys):
    say("key tiles", keys)
    for new in (20, 40, 100):
        check_attention(paged, Setup([new], [keys], 1, 64, BF16, seed=keys), 8)
        check_attention(paged, Setup([new], [keys], 1, 64, E5M2, seed=keys), 8, causal=False)


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("dim,heads", [(64, 4), (80, 2), (96, 3), (128, 8), (128, 1), (256, 2)])
def test_bounds_far_above_the_lengths(paged, dim, heads, head_major, dtype):
    """max_kv_len and max_tokens bound the device's lengths and choose how
    the work is cut; whatever they are, the result is the lengths'."""
    say("bounds", dim, heads, head_major, dtype)
    new, kv = [1, 2, 1, 0, 1, 1], [700, 40, 1, 9, 0, 2100]
    st = Setup(new, kv, heads, dim, dtype, head_major=head_major, pad=2, seed=dim)
    q = st.rows(2 * heads)
    for max_tokens, max_kv in ((2, 2100), (2, 5000), (2, 300000), (3, 10 ** 9), (70, 2100), (70, 300000), (2000, 10 ** 9)):
        cache, batch, status = handles(paged, st, max_tokens, max_kv)
        check_attention(paged, st, 2 * heads, q=q, handle=(cache, batch, status))


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("max_kv", [8, 3000])
def test_thousands_of_sequences(paged, max_kv, dtype):
    """More sequences than two steps of the search tell apart."""
    say("thousands", max_kv, dtype)
    g = torch.Generator().manual_seed(7)
    kv = torch.randint(0, 9, (5000,), generator=g).tolist()
    new = [int(min(n, 1)) for n in kv]
    st = Setup(new, kv, 1, 64, dtype, page=8, pad=3, seed=1)
    check_attention(paged, st, 1, handle=handles(paged, st, 1, max_kv))
    cache, batch, status = handles(paged, st)
    k, _ = paged.gather(cache, batch, status=status)
    rows = [(row, st.place(s, p)) for row, s, p in st.tokens()]
    assert torch.equal(bits(down(k))[[r for r, _ in rows]],
                       torch.stack([bits(st.k)[page, slot] for _, (page, slot) in rows]))


def test_rows_before_the_first_sequence(paged):
    """cu_tokens may begin past 0: the rows before are padding too."""
    say("leading padding")
    st = Setup([3, 2], [40, 70], 2, 64, BF16)
    q, k, v = st.rows(4).cuda(), st.rows(2).cuda(), st.rows(2).cuda()
    cache, batch, status = handles(paged, st)
    want = paged.attention(cache, batch, q)
    moved = paged.PageBatch(st.table.cuda(), (st.cu + 4).cuda(), st.kv_lens.cuda(), 10, 3, 70)

    def pad(x):
        return torch.cat([torch.full_like(x[:4], math.nan), x, torch.full_like(x[:1], math.nan)])
    out = marked((10, 4, 64))
    paged.attention(cache, moved, pad(q), out=out, status=status)
    assert torch.equal(out[4:9], want) and (out[:4].contiguous().view(torch.uint8) == MARK).all()
    a, b = paged.gather(cache, batch)
    c, d = marked((10, 2, 64)), marked((10, 2, 64))
    paged.gather(cache, moved, c, d, status=status)
    assert torch.equal(c[4:9], a) and (c[:4].contiguous().view(torch.uint8) == MARK).all() and (d[9:].view(torch.uint8) == MARK).all()
    paged.append(cache, moved, pad(k), pad(v), status=status)
    assert torch.equal(paged.gather(cache, batch)[1], v) and int(status) == 0


def test_shared_pages_and_output_in_the_query(paged):
    """Two sequences with the same pages (a common prompt); out = q."""
    say("shared pages")
    st = Setup([1, 30], [90, 100], 2, 128, BF16)
    st.table[0] = st.table[1]
    q = st.rows(8)
    got = check_attention(paged, st, 8, q=q)
    cache, batch, _ = handles(paged, st)
    dev = q.cuda()
    paged.attention(cache, batch, dev, out=dev)
    assert torch.equal(down(dev).double(), got)


def test_null_stream_handle(paged):
    say("stream 0")
    st = Setup([1], [300], 2, 128, BF16)
    q = st.rows(8).cuda()
    cache, batch, _ = handles(paged, st)
    want = paged.attention(cache, batch, q)
    torch.cuda.synchronize()
    got = paged.attention(cache, batch, q, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_the_tensor_layer_refuses(paged):
    """Shapes, types, layouts, places and gradients that the calls do not take."""
    from fp8_kv_cache_amd import SzError
    say("refusals")
    st = Setup([2], [40], 2, 64, BF16)
    cache, batch, _ = handles(paged, st)
    k, q = st.rows(2).cuda(), st.rows(4).cuda()
    rope = paged.Rope(paged.rope_table(40, 64))
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    bad = [lambda: paged.attention(cache, batch, q[:1]), lambda: paged.attention(cache, batch, q.float()),
           lambda: paged.attention(cache, batch, q.cpu()), lambda: paged.attention(cache, batch, q[..., ::2]),
           lambda: paged.attention(cache, batch, q[:, :3]), lambda: paged.attention(cache, batch, q[:, 0]),
           lambda: paged.attention(cache, batch, q.transpose(0, 1).contiguous().transpose(0, 1)),
           lambda: paged.attention(cache, batch, q.clone().requires_grad_()),
           lambda: paged.attention(cache, batch, q, out=torch.empty_like(q[:, :2])),
           lambda: paged.attention(cache, batch, q, scale=0.0), lambda: paged.attention(cache, batch, q, scale=math.nan),
           lambda: paged.attention(cache, batch, q, window=-1), lambda: paged.attention(cache, batch, q, window=5, causal=False),
           lambda: paged.attention(cache, batch, q, status=torch.zeros(1, device="cuda")),
           lambda: paged.attention(cache, batch, q, workspace=torch.zeros(4, device="cuda")),
           lambda: paged.append(cache, batch, k, k[:1]), lambda: paged.append(cache, batch, k, k, q_out=q),
           lambda: paged.append(cache, batch, k, k, q_norm=w), lambda: paged.append(cache, batch, k, k, k_norm=w[:32]),
           lambda: paged.append(cache, batch, k, k, k_norm=w, eps=-1.0),
           lambda: paged.append(cache, batch, k, k, rope=paged.Rope(paged.rope_table(40, 96))),
           lambda: paged.append(cache, batch, k, k, rope=paged.Rope(paged.rope_table(40, 24))),
           lambda: paged.gather(cache, batch, k, k.to(torch.float8_e5m2)), lambda: paged.scatter(cache, batch, k, k[:, :1]),
           lambda: paged.scatter(cache, batch, k, k.float()),
           lambda: paged.PagedCache(cache.k[..., :48], cache.v[..., :48]) and paged.gather(
               paged.PagedCache(cache.k[..., :48], cache.v[..., :48]), batch),
           lambda: paged.PagedCache(cache.k, cache.v.transpose(1, 2)), lambda: paged.PagedCache(cache.k.half(), cache.v.half()),
           lambda: paged.PagedCache(cache.k, cache.v.contiguous()[:, :8]),
           lambda: paged.PageBatch(st.table.cuda().long(), st.cu.cuda(), st.kv_lens.cuda()),
           lambda: paged.PageBatch(st.table.cuda(), st.cu.cuda()[:1], st.kv_lens.cuda()),
           lambda: paged.PageBatch(st.table.cuda(), st.cu.cuda(), st.kv_lens.cuda(), -1),
           lambda: paged.Rope(torch.zeros(4, 64, device="cuda").half())]
    for i, call in enumerate(bad):
        with pytest.raises(SzError):
            call()
            pytest.fail(f"call {i} was not refused")
    assert paged.append(cache, batch, k, k, q=q, rope=rope, q_norm=w, k_norm=w).shape == q.shape


def test_lengths_read_from_the_device(paged):
    say("read lengths")
    st = Setup([2, 5], [40, 9], 2, 64, BF16)
    cache = paged.PagedCache(up(st.k), up(st.v))
    batch = paged.PageBatch(st.table.cuda(), st.cu.cuda(), st.kv_lens.cuda())
    assert (batch.total_tokens, batch.raw.max_tokens, batch.raw.max_kv_len) == (7, 5, 40)
    check_attention(paged, st, 4, handle=(cache, batch, torch.zeros(1, dtype=torch.int32, device="cuda")))


def test_two_graphs_and_eager_work_side_by_side(paged):
    """Two captured attentions with workspaces of their own, replayed on two
    streams at once, with eager calls between."""
    say("two graphs")
    st = Setup([1, 1], [3000, 2500], 2, 128, BF16, page=64)
    cache, batch, _ = handles(paged, st)
    qs = [st.rows(8).cuda() for _ in range(2)]
    want = [paged.attention(cache, batch, q) for q in qs]
    outs = [torch.empty_like(q) for q in qs]
    graphs = [torch.cuda.CUDAGraph() for _ in qs]
    for graph, q, out in zip(graphs, qs, outs):
        space = torch.empty(paged.workspace_bytes(cache, batch, 8), dtype=torch.uint8, device="cuda")
        with torch.cuda.graph(graph):
            paged.attention(cache, batch, q, out=out, workspace=space)
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(4):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        eager = paged.attention(cache, batch, qs[0])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(eager, want[0])


@pytest.mark.parametrize("new", [1, 40])
def test_small_weights_of_a_long_row_are_not_lost(paged, new):
    """E5M2: one key at weight 1 and all others at 2^-25.3, values 0 and 1, so
    that the result is the small weights' sum n w / (1 + n w).  Lifted by 2^7
    a weight is 2^-18.3 and FP16's step there 2^-24: half a step is 2^-6.7 of
    it.  The output's rounding adds 2^-8, the score's 32-bit roundings (a
    product of 25.3 and a difference of that size) less than 2^-18, and the
    sum's n 2^-24 of it 2^-9."""
    say("small weights", new)
    kv = 30000
    st = Setup([new], [kv], 1, 64, E5M2)
    for pool, fill in ((st.k, 0.0), (st.v, 1.0)):
        pool[st.table[0].long()] = torch.tensor(fill).to(st.k.dtype)
    page, slot = st.place(0, 5)
    st.k[page, slot, 0, 0] = torch.tensor(16.0).to(st.k.dtype)
    st.v[page, slot] = torch.zeros(1, 64).to(st.v.dtype)
    q = torch.zeros(new, 2, 64, dtype=torch.bfloat16)
    q[:, :, 0] = 1
    cache, batch, status = handles(paged, st)
    out, lse = paged.attention(cache, batch, q.cuda(), scale=25.3 * math.log(2) / 16, return_lse=True, status=status)
    n = kv - new + torch.arange(new, dtype=torch.float64)[:, None, None]   # keys beside the one
    tail = n * 2.0 ** -25.3
    want = tail / (1 + tail)
    off = (out.cpu().double() - want).abs() / want
    assert float(off.max()) <= 2.0 ** -6.7 + 2.0 ** -8 + 2.0 ** -9 + 2.0 ** -17
    want_lse = 25.3 * math.log(2) + torch.log1p(tail[..., 0])
    # n 2^-24 of the sum, and the score's and the logarithm's roundings near 17.5
    assert ((lse.cpu().double() - want_lse).abs() <= kv * 2.0 ** -24 + 17.6 * 2.0 ** -22).all() and int(status) == 0


@pytest.mark.parametrize("dtype", [BF16, E5M2])
@pytest.mark.parametrize("new", [1, 40])
def test_the_largest_scale(paged, new, dtype):
    """Scores of 0 stay 0 at any scale: every row is the mean of its values,
    and keys that a row does not see stay out."""
    say("largest scale", new, dtype)
    st = Setup([new], [new + 30], 1, 64, dtype)
    st.k[st.table[0].long()] = torch.tensor(0.0).to(st.k.dtype)
    check_attention(paged, st, 2, scale=3.4e38)


@pytest.mark.parametrize("kv", [40, 3000])
def test_a_step_without_new_tokens(paged, kv):
    """Sequences without new tokens, and rows of padding: nothing is written."""
    say("no new tokens", kv)
    st = Setup([0, 0], [kv, 7], 2, 64, BF16, pad=3)
    cache = paged.PagedCache(up(st.k), up(st.v))
    batch = paged.PageBatch(st.table.cuda(), st.cu.cuda(), st.kv_lens.cuda(), 3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, x = marked((3, 4, 64)), st.rows(2).cuda()
    paged.attention(cache, batch, st.rows(4).cuda(), out=out, status=status)
    k, v = paged.gather(cache, batch, marked((3, 2, 64)), marked((3, 2, 64)), status=status)
    paged.append(cache, batch, x, x, status=status)
    paged.scatter(cache, batch, x, x, status=status)
    for y in (out, k, v):
        assert (y.view(torch.uint8) == MARK).all()
    assert torch.equal(bits(down(cache.k)), bits(st.k)) and torch.equal(bits(down(cache.v)), bits(st.v))
    assert int(status) == 0
