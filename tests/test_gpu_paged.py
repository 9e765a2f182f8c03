"""The paged cache's operators against their definition in float64.

Written rows are compared byte for byte.  Attention is held to what its
roundings allow, element by element: with A = sum_j p_j |v_j|, each weight is
rounded once to bf16 (half a step, 2^-8 of the weight; fp16 weights of E4M3
caches are finer) and the result once more, so
    |out - exact| <= 2^-8 (A + |exact|) (1 + 2^-7) + 3 dz A + 2^-126
where dz bounds the error of a logit: 128 fp32 additions, |dz| <= 130 * 2^-24
* max_j scale * sum_i |q_i k_ji| (+ one part in 2^22 for exp2 and its
argument), each weight and their sum moving by at most exp(dz) - 1 < 1.5 dz.
The log-sum-exp moves by dz, by the fp32 sum of n terms (n * 2^-24) and by its
own rounding."""
import numpy as np
import pytest
import torch

from gen import counter_hash as ch
from oracle import paged as P
from oracle import reference as R
import shared_top_routing_b200 as sa
from shared_top_routing_b200 import sa as S
from tests.gpu_util import bits_of, dev, i32, to_dev

pytestmark = pytest.mark.gpu

TYPES = [P.BF16, P.E4M3]


def _normal(seed, tid, shape):
    return ch.normal_bf16(seed, tid, count=int(np.prod(shape))).reshape(shape)


def _rng(seed):
    return np.random.default_rng(seed)


def _table(lens, page_size, rng, spare=2, extra_cols=1):
    """A block table whose pages lie in random order, unused entries bad."""
    need = [-(-n // page_size) for n in lens]
    pages = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(need + [1]) + extra_cols), -7, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = pages[at:at + n]
        at += n
    return table, sum(need) + spare


def _random_pool(seed, num_pages, page_size, hkv, kv_type, gain=1.0):
    """A pool of made rows (every row written)."""
    n = num_pages * page_size
    x = R.bf16_bits_to_f64(_normal(seed, 1, (n, hkv, 128))) * gain
    x[:, :, ::29] *= 4
    bits = ch.f32_to_bf16_bits(x.astype(np.float32).reshape(-1)).reshape(x.shape)
    row = P.row_bytes(kv_type, hkv)
    if kv_type == P.BF16:
        rows = np.concatenate([bits.reshape(n, -1).view(np.uint8), np.zeros((n, 16), np.uint8)], 1)
    else:
        rows = np.stack([P.make_row(b, kv_type) for b in bits]) if n <= 64 else _fast_rows(bits)
    return rows.reshape(num_pages, page_size, row)


def _fast_rows(bits):
    """make_row for many rows (the same definition, vectorised)."""
    n, hkv, _ = bits.shape
    x = R.bf16_bits_to_f64(bits)
    e = P.scale_exponent(x)
    codes = P.e4m3_nearest(x / np.exp2(e.astype(float))[..., None]).reshape(n, -1)
    tail = np.zeros((n, 16), np.uint8)
    tail[:, :hkv] = e + 127
    return np.concatenate([codes, tail], 1)


def _dev_pool(pool, kv_type):
    t = torch.from_numpy(pool.copy()).to(dev())
    return t.view(torch.bfloat16) if kv_type == P.BF16 else t


def _host_pool(t):
    return t.view(torch.uint8).cpu().numpy()


def _check_attn(out, lse, ref, n_keys):
    o_ref, l_ref, mag, zabs = ref
    live = ~np.isnan(l_ref)
    got = out.float().cpu().numpy().astype(np.float64)
    dz = (130 * 2.0 ** -24 * zabs + 2.0 ** -22 * (1 + zabs))[..., None]
    tol = 2.0 ** -8 * (mag + np.abs(o_ref)) * (1 + 2.0 ** -7) + 3 * dz * mag + 2.0 ** -126
    err = np.abs(got - o_ref)
    assert np.isfinite(got[live]).all()
    assert (err[live] <= tol[live]).all(), (err[live] / tol[live]).max()
    if lse is not None:
        l = lse.cpu().numpy().astype(np.float64)
        none = np.isneginf(l_ref)
        assert np.array_equal(np.isneginf(l) & live, none)
        fin = live & ~none
        ltol = dz[..., 0] + n_keys * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(fin, l_ref, 0)) + 2.0 ** -22
        assert (np.abs(l[fin] - l_ref[fin]) <= ltol[fin]).all(), np.abs(l[fin] - l_ref[fin]).max()


# ------------------------------------------------------------------- write

@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("hkv,page", [(1, 16), (2, 64), (3, 16), (5, 32), (8, 256), (8, 64)])
def test_write(kv_type, hkv, page):
    """Ragged chunks of a fused projection, a sequence with nothing new, tokens
    in front of and behind the sequences, a chunk longer than its length and a
    bad page; every other byte of the pools stays."""
    rng = _rng(hkv * 1000 + page)
    q_len, kv = [3, 0, 1, 40, 5], [3, 9, 65, 70, 2]
    table, num_pages = _table(kv, page, rng)
    table[2, 64 // page] = num_pages          # the only new token of sequence 2 has no page
    first = 2
    q_start = np.cumsum([first] + q_len).astype(np.int32)
    N = int(q_start[-1]) + 3
    hq = 2 * hkv
    fused = torch.from_numpy(R.bf16_bits_to_f64(_normal(3, hkv, (N, hq + 2 * hkv, 128)))).to(dev()).bfloat16()
    new = [fused[:, hq:hq + hkv], fused[:, hq + hkv:]]
    before = [rng.integers(0, 256, (num_pages, page, P.row_bytes(kv_type, hkv)), dtype=np.uint8) for _ in range(2)]
    pools = [_dev_pool(p, kv_type) for p in before]
    res = sa.sa_paged_kv_write(*new, *pools, i32(table), i32(q_start), i32(kv))
    assert res[0] is pools[0] and res[1] is pools[1]
    for x, p, old in zip(new, pools, before):
        ref = P.paged_write(bits_of(x.contiguous()), old, table, q_start, kv, kv_type)
        assert np.array_equal(_host_pool(p), ref)
        assert not np.array_equal(ref, old)


@pytest.mark.parametrize("kv_type", TYPES)
def test_a_write_beyond_the_table_is_dropped(kv_type):
    """Lengths past the table's last position, far past it and below zero: the
    rows that have a place are written, every other byte stays."""
    hkv, page, cols = 2, 16, 3
    table = np.arange(4 * cols, dtype=np.int32)[::-1].reshape(4, cols).copy()
    q_start, kv = [0, 5, 9, 12, 20], [page * cols + 2, 2 ** 31 - 1, -2 ** 31, page * cols]
    x = _normal(40, 1, (20, hkv, 128))
    old = _rng(41).integers(0, 256, (4 * cols, page, P.row_bytes(kv_type, hkv)), dtype=np.uint8)
    pools = [_dev_pool(old, kv_type) for _ in range(2)]
    sa.sa_paged_kv_write(to_dev(x), to_dev(x), *pools, i32(table), i32(q_start), i32(kv))
    ref = P.paged_write(x, old, table, q_start, kv, kv_type)
    assert (ref != old).reshape(4 * cols * page, -1).any(1).sum() == 3 + 8
    for p in pools:
        assert np.array_equal(_host_pool(p), ref)


def test_write_values_at_the_ends_of_the_range():
    """Zeros, subnormals, the largest values, infinities, NaN, borders of the
    scale, ties of the codes."""
    hkv, page = 8, 16
    rows = np.zeros((12, hkv, 128))
    base = R.bf16_bits_to_f64(_normal(4, 1, (hkv, 128)))
    for t, f in enumerate([0.0, 2.0 ** -133, 2.0 ** -126, 2.0 ** -110, 2.0 ** 100, 2.0 ** 119, 2.0 ** 124, 1.0]):
        rows[t] = base * f
    rows[8, :, 0], rows[8, :, 1] = 448.0, 450.0 * (np.arange(hkv) % 2)
    rows[9] = np.resize((R.e4m3_bits_to_f64(np.arange(126)) + R.e4m3_bits_to_f64(np.arange(1, 127))) / 2, (hkv, 128))
    rows[10], rows[11] = base, base
    with np.errstate(over="ignore"):
        bits = ch.f32_to_bf16_bits(np.clip(rows, -3.38e38, 3.38e38).astype(np.float32).reshape(-1)).reshape(rows.shape)
    bits[10, 0, 3], bits[10, 1, 4], bits[10, 2, 5] = 0x7F80, 0xFF80, 0x7FC0     # inf, -inf, NaN
    bits[11, :, :] = 0x7FC0                                                     # nothing finite
    table, num_pages = _table([12], page, _rng(1))
    zero = np.zeros((num_pages, page, P.row_bytes(P.E4M3, hkv)), np.uint8)
    pools = [_dev_pool(zero, P.E4M3) for _ in range(2)]
    sa.sa_paged_kv_write(to_dev(bits), to_dev(bits), *pools, i32(table), i32([0, 12]), i32([12]))
    ref = P.paged_write(bits, zero, table, [0, 12], [12], P.E4M3)
    got = _host_pool(pools[0])
    nan = (ref & 0x7F) == 0x7F          # the sign of a NaN code is not defined
    nan[..., hkv * 128:] = False
    off = np.argwhere(np.where(nan, 0x7F, ref) != np.where(nan, got & 0x7F, got))
    assert not len(off), [(tuple(i), int(ref[tuple(i)]), int(got[tuple(i)])) for i in off[:8]]
    assert np.array_equal(got, _host_pool(pools[1]))


# ------------------------------------------------------------------ gather

@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("hkv,page,k", [(1, 16, 5), (3, 64, 130), (8, 32, 64), (5, 256, 17)])
def test_gather(kv_type, hkv, page, k):
    """Counts of 0, k, more than k and below 0; positions outside the table;
    codes and scales that are NaN; repeated positions."""
    rng = _rng(k)
    lens = [300, 40, 77, 5]
    table, num_pages = _table(lens, page, rng, extra_cols=0)
    table[table < 0] = num_pages + 3
    pools = [_random_pool(k + i, num_pages, page, hkv, kv_type) for i in range(2)]
    if kv_type == P.E4M3:
        pools[0][:, 1, 0] = 0x7F
        pools[0][:, 2, hkv * 128] = 255
        pools[1][:, 3, hkv * 128:hkv * 128 + hkv] = 0
    idx = rng.integers(0, 300, (4, k), dtype=np.int32)
    idx[1:] %= 40
    idx[0, 0], idx[0, 1], idx[0, 2], idx[0, 3] = -4, table.shape[1] * page + 9, 1, 1
    count = [k, k + 5, 0, -2]
    kr, vr = sa.sa_paged_kv_gather(*[_dev_pool(p, kv_type) for p in pools], i32(table), i32(idx), i32(count))
    for got, p in zip((kr, vr), pools):
        ref = P.paged_gather(p, table, idx, count, kv_type).reshape(4, k, hkv * 128)
        g = got.float().cpu().numpy().astype(np.float64)
        assert not g[..., hkv * 128:].any()
        with np.errstate(over="ignore"):
            want = R.bf16_bits_to_f64(ch.f32_to_bf16_bits(np.nan_to_num(ref).astype(np.float32)))
        assert np.array_equal(np.isnan(g[..., :hkv * 128]), np.isnan(ref))
        assert np.array_equal(np.nan_to_num(g[..., :hkv * 128]), want)


# --------------------------------------------------------------- attention

def _attn_case(seed, kv_type, hkv, G, page, q_len, kv, max_q=None, scale=0.0, lead=0, tail=0, gain=1.0,
               pools=None, strided=False):
    rng = _rng(seed)
    table, num_pages = _table(kv, page, rng)
    if pools is None:
        pools = [_random_pool(seed + i, num_pages, page, hkv, kv_type, gain) for i in range(2)]
    else:
        pools = pools(num_pages)
    q_start = np.cumsum([lead] + q_len).astype(np.int32)
    N, hq = int(q_start[-1]) + tail, hkv * G
    q = _normal(seed, 9, (N, hq, 128))
    tq = to_dev(q)
    if strided:
        wide = torch.full((N, hq + 3, 128), float("nan"), dtype=torch.bfloat16, device=dev())
        wide[:, :hq] = tq
        tq = wide[:, :hq]
    out = torch.full((N, hq, 128), 7.0, dtype=torch.bfloat16, device=dev())
    got, lse = sa.sa_paged_attn(tq, *[_dev_pool(p, kv_type) for p in pools], i32(table), i32(q_start), i32(kv),
                                max(q_len) if max_q is None else max_q, scale=scale, out=out, with_lse=True)
    assert got is out
    ref = P.paged_attention(q, *pools, table, q_start, kv, kv_type, scale)
    return got, lse, ref, max(kv)


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("hkv,G", [(8, 4), (1, 16), (2, 8), (3, 5), (5, 3), (7, 1), (4, 7), (6, 2)])
def test_one_token_per_sequence(kv_type, hkv, G):
    got = _attn_case(hkv * 17 + G, kv_type, hkv, G, 16, [1] * 6, [1, 16, 17, 131, 640, 15])
    _check_attn(*got)


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("hkv,G,q_len,kv", [
    (2, 4, [3, 1, 5, 0, 2], [200, 1, 5, 33, 129]),          # drafts; a whole prompt; a sequence with nothing new
    (1, 3, [130, 20, 1], [130, 257, 300]),                  # chunks past a tile of rows and of keys
    (2, 1, [70, 300], [301, 300]),
])
def test_chunks(kv_type, page, hkv, G, q_len, kv):
    _check_attn(*_attn_case(page + G, kv_type, hkv, G, page, q_len, kv, strided=True))


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8, 11, 16])
def test_every_group_size(kv_type, G):
    _check_attn(*_attn_case(G, kv_type, 1, G, 32, [150, 9], [333, 140]))


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("q_len,kv", [([5, 40], [3, 0]), ([1], [0]), ([200], [130])])
def test_tokens_with_nothing_to_attend_to(kv_type, q_len, kv):
    """kv_len below the chunk's length: the first tokens see no key."""
    got, lse, ref, n = _attn_case(3, kv_type, 2, 4, 16, q_len, kv)
    _check_attn(got, lse, ref, n)
    none = np.isneginf(ref[1])
    assert none.any() and not got.float().cpu().numpy()[none].any()


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("q_len", [[2, 1, 3], [40, 1, 90]])
def test_tokens_of_no_sequence_and_beyond_the_bound_stay(kv_type, q_len):
    got, lse, ref, n = _attn_case(5, kv_type, 2, 4, 16, q_len, [70, 33, 95], lead=2, tail=3)
    _check_attn(got, lse, ref, n)
    dead = np.isnan(ref[1][:, 0])
    assert dead.sum() == 5 and (got.float().cpu().numpy()[dead] == 7.0).all()
    # a bound below a sequence's length: its later tokens are left alone
    bound = max(q_len) - 1
    got, _, ref, _ = _attn_case(5, kv_type, 2, 4, 16, q_len, [70, 33, 95], max_q=bound)
    at = sum(q_len[:q_len.index(max(q_len))])
    assert (got.float().cpu().numpy()[at + bound] == 7.0).all()
    ref[1][at + bound] = np.nan
    _check_attn(got, None, ref, n)


@pytest.mark.parametrize("kv_type", TYPES)
def test_scale_and_large_logits(kv_type):
    """A given scale, and logits in the hundreds: one key takes nearly all."""
    _check_attn(*_attn_case(21, kv_type, 2, 4, 16, [1, 33], [300, 200], scale=0.31))
    _check_attn(*_attn_case(22, kv_type, 2, 4, 16, [1, 140], [300, 200], gain=24.0))


def test_scales_far_apart():
    """E4M3 rows whose scales differ by up to 2^60: weights and scales are kept
    apart from one another's range."""
    def pools(num_pages):
        out = []
        for i in range(2):
            p = _random_pool(40 + i, num_pages, 16, 2, P.E4M3)
            rng = _rng(50 + i)
            spread = rng.integers(-6, 3, (num_pages, 16, 2)) if i == 0 else rng.integers(-40, 20, (num_pages, 16, 2))
            p[..., 256:258] = np.clip(p[..., 256:258].astype(int) + spread, 1, 254)
            out.append(p)
        return out

    for q_len, kv in (([1, 1, 3], [300, 17, 90]), ([150, 40], [300, 290])):
        _check_attn(*_attn_case(41, P.E4M3, 2, 4, 16, q_len, kv, pools=pools))


def _poison(rows, kv_type, hkv, what):
    """Makes cache rows hold infinities or NaN everywhere."""
    if kv_type == P.BF16:
        rows[..., :hkv * 256].view(np.uint16)[...] = what
    else:
        rows[..., :hkv * 128] = 0x7F
        rows[..., hkv * 128:] = 0xFF


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("what", [0x7F80, 0xFFC0])
@pytest.mark.parametrize("q_len,kv", [([1, 1, 1], [1, 77, 130]), ([4, 2], [90, 18]), ([130, 50], [300, 51])])
def test_what_rows_beyond_hold_has_no_effect(kv_type, what, q_len, kv):
    """Every row behind a sequence's last, every page of no sequence, and every
    table entry behind the last page hold infinities, NaN and bad pages."""
    rng = _rng(7)
    page, hkv, G = 16, 2, 4
    table, num_pages = _table(kv, page, rng)

    def pools(n):
        assert n == num_pages
        out = []
        for i in range(2):
            p = _random_pool(60 + i, n, page, hkv, kv_type)
            used = np.zeros((n, page), bool)
            for b, s in enumerate(kv):
                j = np.arange(s)
                used[table[b, j // page], j % page] = True
            dead = p[~used]
            _poison(dead, kv_type, hkv, what)
            p[~used] = dead
            out.append(p)
        return out

    _check_attn(*_attn_case(7, kv_type, hkv, G, page, q_len, kv, pools=pools))


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("q_len,kv,bad", [([6], [40], 36), ([150], [290], 200), ([300], [300], 299), ([4], [130], 127)])
def test_a_later_tokens_infinities_reach_only_those_that_see_them(kv_type, q_len, kv, bad):
    """K and V of one position of the chunk are not finite: tokens before it
    are exact, tokens from it on show it."""
    page, hkv, G = 16, 2, 4
    table, num_pages = _table(kv, page, _rng(9))

    def pools(n):
        out = []
        for i in range(2):
            p = _random_pool(70 + i, n, page, hkv, kv_type)
            if i == 1:   # V: one infinite and one NaN element; K stays finite
                row = p[table[0, bad // page], bad % page]
                if kv_type == P.BF16:
                    row[:hkv * 256].view(np.uint16)[5], row[:hkv * 256].view(np.uint16)[128 + 9] = 0x7F80, 0x7FC0
                else:
                    row[5], row[128 + 9] = 0x7F, 0xFF
            out.append(p)
        return out

    got, lse, ref, n = _attn_case(9, kv_type, hkv, G, page, q_len, kv, pools=pools)
    g = got.float().cpu().numpy()
    first = bad - (kv[0] - q_len[0])          # the first token that sees it
    assert np.isfinite(g[:first]).all()
    assert not np.isfinite(g[first:, :G, 5]).any() and np.isnan(g[first:, G:, 9]).all()
    if kv_type == P.BF16:
        assert np.isposinf(g[first:, :G, 5]).all()
    hit = np.zeros(g.shape, bool)
    hit[first:, :G, 5] = hit[first:, G:, 9] = True
    ref_o = np.where(hit, 0.0, np.nan_to_num(ref[0], nan=0.0, posinf=0.0))
    got0 = torch.from_numpy(np.where(hit, 0.0, g)).to(dev())
    mag = np.where(hit, 0.0, np.nan_to_num(ref[2], nan=0.0, posinf=0.0))
    _check_attn(got0, lse, [ref_o, ref[1], mag, ref[3]], n)


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("q_len,kv", [([1], [100]), ([140], [200])])
def test_a_bad_key_makes_nan_of_the_tokens_that_see_it(kv_type, q_len, kv):
    page, hkv, G, bad = 16, 1, 4, kv[0] - 1
    table, _ = _table(kv, page, _rng(11))

    def pools(n):
        out = [_random_pool(80 + i, n, page, hkv, kv_type) for i in range(2)]
        row = out[0][table[0, bad // page], bad % page]
        if kv_type == P.BF16:
            row[:256].view(np.uint16)[3] = 0x7FC0
        else:
            row[3] = 0x7F
        return out

    got, lse, ref, _ = _attn_case(11, kv_type, hkv, G, page, q_len, kv, pools=pools)
    assert torch.isnan(got[-1]).all() and torch.isnan(lse[-1]).all()
    assert torch.isfinite(got[:-1]).all()


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("hkv,G,k", [(8, 4, 40), (1, 16, 300), (2, 8, 1), (3, 5, 129), (7, 2, 64)])
def test_sparse_decode(kv_type, hkv, G, k):
    """Counts from 0 to k, unsorted and repeated positions, positions outside
    the table, bad pages where no position goes."""
    rng = _rng(hkv * 31 + k)
    page, lens = 32, [400, 64, 33, 1, 90]
    table, num_pages = _table(lens, page, rng)
    pools = [_random_pool(90 + i, num_pages, page, hkv, kv_type) for i in range(2)]
    B = len(lens)
    idx = np.stack([rng.integers(0, n, k) for n in lens]).astype(np.int32)
    count = np.minimum([k, k + 3, k // 2, 0, 1], [k + 3] * B)
    idx[2, k // 2:] = -1
    q = _normal(hkv, 77, (B, hkv * G, 128))
    got, lse = sa.sa_paged_sparse_attn_decode(to_dev(q), *[_dev_pool(p, kv_type) for p in pools], i32(table),
                                              i32(idx), i32(count), with_lse=True)
    ref = P.paged_sparse_attention(q, *pools, table, idx, count, kv_type)
    _check_attn(got, lse, ref, k)
    # a used position outside the table is clamped, a bad page too: a wrong row, no fault
    idx[0, 0], idx[1, 0] = -3, 1 << 30
    got, lse = sa.sa_paged_sparse_attn_decode(to_dev(q), *[_dev_pool(p, kv_type) for p in pools], i32(table),
                                              i32(idx), i32(count), with_lse=True)
    _check_attn(got, lse, P.paged_sparse_attention(q, *pools, table, idx, count, kv_type), k)


@pytest.mark.parametrize("kv_type", TYPES)
def test_a_long_chunk_is_the_same_every_time(kv_type):
    """Many items per SM, thousands of key tiles: every run gives the same bits,
    and the log-sum-exp is that of fp32 products (error: 130 * 2^-24 * the sum
    of magnitudes, below 60 for these inputs, twice; and the sums')."""
    hkv, G, page, T, S = 8, 4, 64, 1536, 12000
    g = torch.Generator(device=dev()).manual_seed(3)
    num_pages = -(-S // page)
    pools = sa.sa_paged_kv_alloc(num_pages, page, hkv, kv_type, device=dev())
    k, v = (torch.randn(S, hkv, 128, device=dev(), generator=g).bfloat16() for _ in range(2))
    table = torch.randperm(num_pages, device=dev(), generator=g).int()[None]
    sa.sa_paged_kv_write(k, v, *pools, table, i32([0, S]), i32([S]))
    rows = sa.sa_paged_kv_gather(*pools, table, torch.arange(S, device=dev(), dtype=torch.int32)[None], i32([S]))
    kr, vr = (r[0, :, :hkv * 128].float().view(S, hkv, 128).transpose(0, 1) for r in rows)
    q = torch.randn(T, hkv * G, 128, device=dev(), generator=g).bfloat16()
    args = (q, *pools, table, i32([0, T]), i32([S]), T)
    out, lse = sa.sa_paged_attn(*args, with_lse=True)
    for _ in range(8):
        o2, l2 = sa.sa_paged_attn(*args, with_lse=True)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    seen = torch.arange(S, device=dev()) <= (S - T + torch.arange(T, device=dev()))[:, None]
    for h in range(hkv):
        z = torch.matmul(q[:, h * G:h * G + G].float().transpose(0, 1), kr[h].T) * 128 ** -0.5
        z.masked_fill_(~seen, float("-inf"))
        ref = torch.logsumexp(z, -1)
        assert (lse[:, h * G:h * G + G].T - ref).abs().max() < 2 * 130 * 2.0 ** -24 * 60 + 2.0 ** -15
        p = torch.exp(z - ref[..., None])
        o, mag = torch.matmul(p, vr[h]), torch.matmul(p, vr[h].abs())
        err = (out[:, h * G:h * G + G].transpose(0, 1).float() - o).abs()
        assert (err <= 2.0 ** -8 * (mag + o.abs()) * 1.01 + 2.0 ** -10 * mag).all()


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("hkv,G,top", [(1, 1, 32), (2, 4, 8), (1, 8, 16), (3, 16, 8), (8, 5, 6)])
def test_short_chunks_of_every_length(kv_type, hkv, G, top):
    """Chunks that take one block of rows up to those that take many."""
    q_len = [1 + (7 * i) % top for i in range(9)] + [top]
    _check_attn(*_attn_case(G, kv_type, hkv, G, 16, q_len, [n + 37 * i for i, n in enumerate(q_len)]))


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("B,hkv,G", [
    (5, 2, 4),       # a few items per SM at most
    (70, 3, 16),     # more items per kv head than threads of a block
    (130, 1, 16),    # more than are sorted: the list is cut
])
def test_ragged_batches_of_many_items(kv_type, B, hkv, G):
    q_len = [1 + 13 * i % 11 for i in range(B)]
    q_len[B // 2] = 130
    kv = [n + (29 * i) % 150 for i, n in enumerate(q_len)]
    _check_attn(*_attn_case(B, kv_type, hkv, G, 32, q_len, kv))


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("hkv,G", [(2, 1), (8, 4), (3, 5), (1, 16)])
def test_decoding_sequences_beside_a_long_chunk(kv_type, hkv, G):
    """Chunks of every length around a block of 16 rows, beside one of many;
    tokens of no sequence around them, a sequence with nothing new."""
    few = 16 // G
    q_len = [1, few, 129 // G + 30, few + 1, 0, max(1, few - 1), 1]
    kv = [70, few + 3, 250, 400, 5, 0, 1]
    got, lse, ref, n = _attn_case(G, kv_type, hkv, G, 16, q_len, kv, lead=3, tail=40)
    _check_attn(got, lse, ref, n)
    dead = np.isnan(ref[1][:, 0])
    assert dead.sum() == 43 and (got.float().cpu().numpy()[dead] == 7.0).all()


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("lens", [[1000] * 4, [2000, 300, 77, 900]])
def test_whole_prompts(kv_type, lens):
    """Items dealt to the CTAs whole, of one length and of many; every run the
    same bits."""
    hkv, G, page = 8, 2, 64
    g = torch.Generator(device=dev()).manual_seed(4)
    pages = [-(-n // page) for n in lens]
    pools = sa.sa_paged_kv_alloc(sum(pages), page, hkv, kv_type, device=dev())
    table, at = np.zeros((len(lens), max(pages)), np.int32), 0
    for b, n in enumerate(pages):
        table[b, :n] = np.arange(at, at + n)[::-1]
        at += n
    N = sum(lens)
    start = np.cumsum([0] + lens)
    k, v = (torch.randn(N, hkv, 128, device=dev(), generator=g).bfloat16() for _ in range(2))
    args = (i32(table), i32(start), i32(lens))
    sa.sa_paged_kv_write(k, v, *pools, *args)
    q = torch.randn(N, hkv * G, 128, device=dev(), generator=g).bfloat16()
    out, lse = sa.sa_paged_attn(q, *pools, *args, max(lens), with_lse=True)
    for _ in range(4):
        o2, l2 = sa.sa_paged_attn(q, *pools, *args, max(lens), with_lse=True)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    for b, n in enumerate(lens):
        idx = torch.arange(n, device=dev(), dtype=torch.int32)[None]
        rows = sa.sa_paged_kv_gather(*pools, i32(table[b:b + 1]), idx, i32([n]))
        kr, vr = (r[0, :, :hkv * 128].double().view(n, hkv, 128).transpose(0, 1) for r in rows)
        part = slice(start[b], start[b + 1])
        qb = q[part].double().view(n, hkv, G, 128).permute(1, 2, 0, 3)
        z = torch.matmul(qb, kr.transpose(1, 2)[:, None]) * 128 ** -0.5
        seen = torch.ones(n, n, dtype=torch.bool, device=dev()).tril()
        zabs = (torch.matmul(qb.abs(), kr.abs().transpose(1, 2)[:, None]) * seen).amax(-1) * 128 ** -0.5
        z.masked_fill_(~seen, float("-inf"))
        ref = torch.logsumexp(z, -1)
        p = torch.exp(z - ref[..., None])
        o, mag = torch.matmul(p, vr[:, None]), torch.matmul(p, vr.abs()[:, None])

        def flat(t):   # [hkv, G, n, ...] as [n, hkv * G, ...]
            return t.movedim(2, 0).reshape(n, hkv * G, *t.shape[3:]).cpu().numpy()

        _check_attn(out[part], lse[part], tuple(flat(t) for t in (o, ref, mag, zabs)), n)


@pytest.mark.parametrize("B,hkv,max_pages", [(3, 8, 5000), (2, 8, 30000), (2, 1, 140000)])
def test_codes_written_out_in_rounds(B, hkv, max_pages):
    """A block table so wide that the rows of all sequences, or of all heads of
    one, do not fit the space for rows in bf16: a few at a time."""
    G, page, q_len, kv = 16, 16, [40, 9, 150][:B], [333, 140, 170][:B]
    table, num_pages = _table(kv, page, _rng(B))
    wide = np.full((B, max_pages), -3, np.int32)
    wide[:, :table.shape[1]] = table
    pools = [_random_pool(140 + i, num_pages, page, hkv, P.E4M3) for i in range(2)]
    q_start = np.cumsum([0] + q_len).astype(np.int32)
    q = _normal(30, 1, (int(q_start[-1]), hkv * G, 128))
    out, lse = sa.sa_paged_attn(to_dev(q), *[_dev_pool(p, P.E4M3) for p in pools], i32(wide), i32(q_start), i32(kv),
                                max(q_len), with_lse=True)
    _check_attn(out, lse, P.paged_attention(q, *pools, table, q_start, kv, P.E4M3), max(kv))


# ---------------------------------------------------------- in use together

@pytest.mark.parametrize("kv_type", TYPES)
def test_prefill_then_decode_steps(kv_type):
    """A prompt in two chunks, then decode steps: each call writes its rows and
    attends; a layer of selected rows straight from the pages, and through
    gathered rows, gives what the dense form over those rows gives."""
    hkv, G, page, k = 2, 4, 16, 24
    hq, lens = hkv * G, [90, 41]
    table, num_pages = _table([n + 4 for n in lens], page, _rng(13))
    pools = sa.sa_paged_kv_alloc(num_pages, page, hkv, kv_type, device=dev())
    host = [np.zeros((num_pages, page, P.row_bytes(kv_type, hkv)), np.uint8) for _ in range(2)]
    kv = [0, 0]
    step = 0
    for q_len in ([50, 41], [40, 0], [1, 1], [1, 1], [2, 1]):
        step += 1
        kv = [a + n for a, n in zip(kv, q_len)]
        q_start = np.cumsum([0] + q_len)
        N = int(q_start[-1])
        q, kn, vn = (_normal(100 + step, i, (N, h, 128)) for i, h in ((1, hq), (2, hkv), (3, hkv)))
        sa.sa_paged_kv_write(to_dev(kn), to_dev(vn), *pools, i32(table), i32(q_start), i32(kv))
        host = [P.paged_write(x, p, table, q_start, kv, kv_type) for x, p in zip((kn, vn), host)]
        out, lse = sa.sa_paged_attn(to_dev(q), *pools, i32(table), i32(q_start), i32(kv), max(q_len), with_lse=True)
        assert all(np.array_equal(_host_pool(p), h) for p, h in zip(pools, host))
        _check_attn(out, lse, P.paged_attention(q, *host, table, q_start, kv, kv_type), max(kv))
    # sparse layers: the indexer's selection over the same positions
    d = 64
    q_idx, k_idx = ch.int_bf16(5, 1, count=2 * d).reshape(2, d), ch.int_bf16(5, 2, count=2 * 128 * d).reshape(2, 128, d)
    idx, cnt = sa.sa_index_score_topk(to_dev(q_idx), to_dev(k_idx), k, Tk=128, kv_len=i32(kv))
    q = _normal(200, 1, (2, hq, 128))
    out, lse = sa.sa_paged_sparse_attn_decode(to_dev(q), *pools, i32(table), idx, cnt, with_lse=True)
    ref = P.paged_sparse_attention(q, *host, table, idx.cpu().numpy(), cnt.cpu().numpy(), kv_type)
    _check_attn(out, lse, ref, k)
    rows = sa.sa_paged_kv_gather(*pools, i32(table), idx, cnt)
    out2, lse2 = sa.sa_sparse_attn_decode_rows(to_dev(q), *rows, cnt, with_lse=True)
    _check_attn(out2, lse2, ref, k)


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("q_len", [[1, 1], [60, 3]])
def test_graphs_streams_and_two_calls_at_once(kv_type, q_len):
    """Two graphs captured on one stream and replayed on two, next to an eager
    call on a third: each has a workspace of its own, all give one answer."""
    hkv, G, page, kv = 2, 4, 16, [900, 333]
    table, num_pages = _table(kv, page, _rng(15))
    pools = [_dev_pool(_random_pool(120 + i, num_pages, page, hkv, kv_type), kv_type) for i in range(2)]
    q_start = i32(np.cumsum([0] + q_len))
    N = sum(q_len)
    qs = [to_dev(_normal(16 + i, 1, (N, hkv * G, 128))) for i in range(2)]
    args = (*pools, i32(table), q_start, i32(kv), max(q_len))
    want = [sa.sa_paged_attn(q, *args, with_lse=True) for q in qs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sa.sa_paged_attn(q, *args, with_lse=True))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = sa.sa_paged_attn(qs[0], *args, with_lse=True, stream=streams[2])
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(outs + [eager], want + want[:1]):
        assert torch.equal(o, wo) and torch.equal(l, wl)


def test_a_captured_step_reads_lengths_at_replay():
    """Lengths, tables and rows are device data: one captured decode step
    (write, then attend) serves every later step."""
    hkv, G, page = 2, 4, 16
    table, num_pages = _table([40, 40], page, _rng(17))
    pools = sa.sa_paged_kv_alloc(num_pages, page, hkv, S.SA_KV_E4M3, device=dev())
    host = [np.zeros((num_pages, page, P.row_bytes(P.E4M3, hkv)), np.uint8) for _ in range(2)]
    kv_len, q_start, tab = i32([1, 1]), i32([0, 1, 2]), i32(table)
    q, k, v = (torch.zeros(2, h, 128, dtype=torch.bfloat16, device=dev()) for h in (hkv * G, hkv, hkv))

    def step():
        sa.sa_paged_kv_write(k, v, *pools, tab, q_start, kv_len)
        return sa.sa_paged_attn(q, *pools, tab, q_start, kv_len, 1, with_lse=True)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = step()
    for n in range(1, 38, 4):
        for t in range(4):
            kv = [n + t, max(1, n + t - 3)]
            new = [_normal(300 + n + t, i, (2, h, 128)) for i, h in ((1, hkv * G), (2, hkv), (3, hkv))]
            for dst, src in zip((q, k, v), new):
                dst.copy_(to_dev(src))
            kv_len.copy_(i32(kv))
            g.replay()
            host = [P.paged_write(x, p, table, [0, 1, 2], kv, P.E4M3) for x, p in zip(new[1:], host)]
        _check_attn(out, lse, P.paged_attention(new[0], *host, table, [0, 1, 2], kv, P.E4M3), 40)


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("q_len", [[1, 1], [100, 7]])
def test_error_word_gives_nan(kv_type, q_len):
    """A workspace whose error word is set (as a wait that gave up leaves it)
    makes every output NaN; sa_workspace_status reports it."""
    hkv, G, page, kv = 2, 4, 16, [200, 60]
    table, num_pages = _table(kv, page, _rng(19))
    pools = [_dev_pool(_random_pool(130 + i, num_pages, page, hkv, kv_type), kv_type) for i in range(2)]
    N = sum(q_len)
    q = to_dev(_normal(20, 1, (N, hkv * G, 128)))
    need = S.lib().sa_paged_attn_workspace(2, N, max(q_len), table.shape[1], page, hkv * G, hkv, 128, kv_type)
    ws = torch.zeros(need, dtype=torch.uint8, device=dev())
    args = (*pools, i32(table), i32(np.cumsum([0] + q_len)), i32(kv), max(q_len))
    good = sa.sa_paged_attn(q, *args, ws=ws)
    assert S.sa_workspace_status(ws) == S.SA_OK
    ws[:4].view(torch.int32)[0] = 21
    bad, lse = sa.sa_paged_attn(q, *args, ws=ws, with_lse=True)
    assert torch.isnan(bad).all() and torch.isnan(lse).all()
    assert S.sa_workspace_status(ws) == S.SA_ERR_TIMEOUT
    ws.zero_()
    assert torch.equal(sa.sa_paged_attn(q, *args, ws=ws), good)


def test_nothing_to_do():
    pools = sa.sa_paged_kv_alloc(2, 16, 2, device=dev())
    none = torch.empty(0, 8, 128, dtype=torch.bfloat16, device=dev())
    table, zero = i32(np.zeros((1, 2))), i32([0, 0])
    assert sa.sa_paged_attn(none, *pools, table, zero, i32([5])).shape == (0, 8, 128)
    sa.sa_paged_kv_write(none[:, :2], none[:, :2], *pools, table, zero, i32([5]))
    empty = sa.sa_paged_kv_gather(*pools, i32(np.zeros((0, 2))), i32(np.zeros((0, 3))), i32(np.zeros(0)))
    assert empty[0].shape == (0, 3, 264)


def test_debug_build_records_bad_pages_and_positions(monkeypatch):
    """The debug library notes a used bad page and position and the canary of
    each workspace stays; results equal the release library's."""
    LD = S.lib_debug()
    S.debug_read(LD, reset=True)
    hkv, G, page, kv = 2, 4, 16, [70, 40]
    table, num_pages = _table(kv, page, _rng(23))
    pools = [_dev_pool(_random_pool(140 + i, num_pages, page, hkv, P.E4M3), P.E4M3) for i in range(2)]
    q = to_dev(_normal(24, 1, (2, hkv * G, 128)))
    qc = to_dev(_normal(24, 2, (42, hkv * G, 128)))
    idx, cnt = i32(np.tile(np.arange(9), (2, 1))), i32([9, 5])

    def calls(tab, idx):
        ws = [torch.zeros(1 << 26, dtype=torch.uint8, device=dev()) for _ in range(3)]
        return [sa.sa_paged_attn(q, *pools, tab, i32([0, 1, 2]), i32(kv), 1, ws=ws[0]),
                sa.sa_paged_attn(qc, *pools, tab, i32([0, 40, 42]), i32(kv), 40, ws=ws[1]),
                sa.sa_paged_sparse_attn_decode(q, *pools, tab, idx, cnt, ws=ws[2]),
                *sa.sa_paged_kv_gather(*pools, tab, idx, cnt)]

    bad_tab, bad_idx = table.copy(), idx.clone()
    bad_tab[1, 1] = num_pages + 40
    bad_idx[0, 4] = 1 << 20
    want = [calls(i32(table), idx), calls(i32(bad_tab), idx), calls(i32(table), bad_idx)]
    torch.cuda.synchronize()
    monkeypatch.setattr(S, "_lib", LD)
    got = [calls(i32(table), idx)]
    torch.cuda.synchronize()
    assert S.debug_read(LD) == [0, 0, 0, 0]
    got.append(calls(i32(bad_tab), idx))
    torch.cuda.synchronize()
    rec = S.debug_read(LD)
    assert rec[:3] == [5, num_pages + 40, num_pages] and rec[3] >= 1
    got.append(calls(i32(table), bad_idx))
    torch.cuda.synchronize()
    assert S.debug_read(LD)[:3] == [6, 1 << 20, table.shape[1] * page]
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_the_binding_refuses_on_the_gpu():
    pools = sa.sa_paged_kv_alloc(4, 16, 2, device=dev())
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device=dev())
    table, qs, kl = i32(np.zeros((2, 2))), i32([0, 1, 2]), i32([3, 4])
    with pytest.raises(ValueError, match="side by side"):
        sa.sa_paged_attn(q.transpose(0, 1).contiguous().transpose(0, 1), *pools, table, qs, kl)
    with pytest.raises(ValueError, match="kv_len"):
        sa.sa_paged_attn(q, *pools, table, qs, kl.long())
    with pytest.raises(ValueError, match="q_start"):
        sa.sa_paged_attn(q, *pools, table, qs[:2], kl)
    with pytest.raises(ValueError, match="bfloat16"):
        sa.sa_paged_attn(q.float(), *pools, table, qs, kl)
    with pytest.raises(ValueError, match="out"):
        sa.sa_paged_attn(q, *pools, table, qs, kl, out=torch.empty(2, 8, 64, dtype=torch.bfloat16, device=dev()))
    with pytest.raises(sa.SAError, match="multiple"):
        sa.sa_paged_attn(q[:, :7].contiguous(), *pools, table, qs, kl)
    with pytest.raises(ValueError, match="k_new"):
        sa.sa_paged_kv_write(q, q, *pools, table, qs, kl)
    with pytest.raises(ValueError, match="idx"):
        sa.sa_paged_kv_gather(*pools, table, kl, kl)


# ------------------------------------- batches with few tokens for their slots

def _slots_case(kind, slots, G):
    """q_len of a batch whose packed tokens (two more belong to no sequence)
    are at most slots * (16 // G), with a chunk of more than 128 rows per kv
    head, or a bound that allows one."""
    few = 16 // G
    room = slots * few - 2
    if kind == "drafts":          # drafts too long for a block of rows beside single tokens, the bound left out
        long = max(5, few + 1)
        n = min(slots // 2, (room - slots) // (long - 1)) if few > 1 else 3
        ones = slots - n if few > 1 else 8
        q_len = [long] * n + [1] * ones
    elif kind == "single tokens":
        q_len = [128 // G + 8] + [1] * (slots - 1 if few > 1 else 8)
    else:
        q_len = [128 // G + 8]
    q_len += [0] * (slots - len(q_len))
    q_len = q_len[slots // 3:] + q_len[:slots // 3]
    assert sum(q_len) <= room and max(q_len) > few
    return q_len


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("hkv", [1, 8])        # rows to fold: fewer than a warp each is used for, or more
@pytest.mark.parametrize("slots", [28, 40])    # sequences planned by a warp, or by a block
@pytest.mark.parametrize("G", [1, 4, 8, 16])
@pytest.mark.parametrize("kind", ["single tokens", "idle slots", "drafts"])
def test_a_long_chunk_in_a_batch_with_few_tokens(kv_type, hkv, slots, G, kind):
    """A chunk for the tensor cores beside decoding or idle sequences, fewer
    tokens in all than the blocks of the short ones could hold."""
    q_len = _slots_case(kind, slots, G)
    rng = _rng(slots + G)
    kv = [n + (29 * i) % 150 + 60 * (n > 16 // G) for i, n in enumerate(q_len)]
    table, num_pages = _table(kv, 16, rng)
    pools = [_random_pool(G + i, num_pages, 16, hkv, kv_type) for i in range(2)]
    q_start = np.cumsum([1] + q_len).astype(np.int32)
    N = int(q_start[-1]) + 1
    q = _normal(slots, 9, (N, hkv * G, 128))
    bound = {} if kind == "drafts" else {"max_q": max(q_len)}
    assert (N if kind == "drafts" else max(q_len)) * G > 128
    out = torch.full((N, hkv * G, 128), 7.0, dtype=torch.bfloat16, device=dev())
    _, lse = sa.sa_paged_attn(to_dev(q), *[_dev_pool(p, kv_type) for p in pools], i32(table), i32(q_start), i32(kv),
                              out=out, with_lse=True, **bound)
    ref = P.paged_attention(q, *pools, table, q_start, kv, kv_type)
    _check_attn(out, lse, ref, max(kv))
    assert (out[0] == 7.0).all() and (out[-1] == 7.0).all()


# ------------------------------------------------ what the joins have to keep

@pytest.mark.parametrize("kv_type,kv", [(P.BF16, 97), (P.BF16, 129), (P.E4M3, 33), (P.E4M3, 257)])
@pytest.mark.parametrize("B", [3, 64])         # rows to fold: a block each, or a warp
@pytest.mark.parametrize("sparse", [False, True])
def test_a_bad_key_alone_in_its_part_makes_nan(kv_type, kv, B, sparse):
    """The last key, which no other shares a warp's slice (97, 33) or a tile
    (129, 257) with, is NaN: so are the output and the log-sum-exp."""
    hkv, G, page = 1, 16, 16
    table, num_pages = _table([kv] * B, page, _rng(kv))
    pools = [_random_pool(150 + i, num_pages, page, hkv, kv_type) for i in range(2)]
    row = pools[0][table[1, (kv - 1) // page], (kv - 1) % page]
    if kv_type == P.BF16:
        row[:256].view(np.uint16)[3] = 0x7FC0
    else:
        row[3] = 0x7F
    q = _normal(31, 1, (B, G, 128))
    dp = [_dev_pool(p, kv_type) for p in pools]
    if sparse:
        idx, count = np.tile(np.arange(kv, dtype=np.int32), (B, 1)), [kv] * B
        out, lse = sa.sa_paged_sparse_attn_decode(to_dev(q), *dp, i32(table), i32(idx), i32(count), with_lse=True)
    else:
        out, lse = sa.sa_paged_attn(to_dev(q), *dp, i32(table), i32(np.arange(B + 1)), i32([kv] * B), 1, with_lse=True)
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    ref = P.paged_attention(q, *pools, table, np.arange(B + 1), [kv] * B, kv_type)
    for r in ref:
        r[1] = np.nan                          # (not compared)
    _check_attn(out, lse, ref, kv)


def _faint_case(kv_type, G, q_len, kv, faint, bad):
    """One sequence, one kv head, every query row the same vector u; the keys
    that `faint` names are -40 u, so that their weights are far below fp32's
    least (2^-600 or so of the others'), and V of position `bad`, one of them,
    holds NaN in element 5: NaN by the definition."""
    page = 16
    u = _normal(32, 1, (1, 1, 128))
    q = np.tile(u, (q_len, G, 1))
    table, num_pages = _table([kv], page, _rng(33))
    pools = [_random_pool(160 + i, num_pages, page, 1, kv_type) for i in range(2)]
    far = ch.f32_to_bf16_bits((-40 * R.bf16_bits_to_f64(u).reshape(-1)).astype(np.float32)).reshape(1, 128)
    for j in np.flatnonzero(faint(np.arange(kv))):
        pools[0][table[0, j // page], j % page] = P.make_row(far, kv_type)
    row = pools[1][table[0, bad // page], bad % page]
    if kv_type == P.BF16:
        row[:256].view(np.uint16)[5] = 0x7FC0
    else:
        row[5] = 0x7F
    args = (to_dev(q), *[_dev_pool(p, kv_type) for p in pools], i32(table))
    ref = P.paged_attention(q, *pools, table, [0, q_len], [kv], kv_type)
    return args, ref, faint(np.arange(kv))


def _check_faint(out, lse, ref, kv):
    o, l, mag, zabs = ref
    assert np.isnan(o[..., 5]).all() and not np.isnan(np.delete(o, 5, -1)).any()
    assert torch.isnan(out[..., 5]).all(), "a NaN value's weight was taken for nothing"
    clean = out.clone()
    clean[..., 5] = 0
    o[..., 5] = mag[..., 5] = 0
    _check_attn(clean, lse, (o, l, mag, zabs), kv)


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("G,q_len", [(16, 1), (1, 3)])
@pytest.mark.parametrize("sparse", [False, True])
def test_a_value_that_is_nan_shows_however_little_its_weight(kv_type, G, q_len, sparse):
    """All keys of a warp's slice (and of a tile) have weights that are nothing
    beside the others'."""
    if sparse and q_len > 1:
        q_len = 1
    kv = 900
    args, ref, _ = _faint_case(kv_type, G, q_len, kv, lambda j: j < 256, 7)
    if sparse:
        out, lse = sa.sa_paged_sparse_attn_decode(*args, i32(np.arange(kv)[None]), i32([kv]), with_lse=True)
    else:
        out, lse = sa.sa_paged_attn(*args, i32([0, q_len]), i32([kv]), q_len, with_lse=True)
    _check_faint(out, lse, ref, kv)


def test_a_value_that_is_nan_shows_when_a_warp_folds_a_row():
    """As above with enough rows that a warp folds each."""
    kv, B, G = 900, 64, 16
    (q, kp, vp, table), ref, _ = _faint_case(P.BF16, G, 1, kv, lambda j: j < 256, 7)
    out, lse = sa.sa_paged_attn(q.expand(B, G, 128).contiguous(), kp, vp, table.expand(B, -1).contiguous(),
                                i32(np.arange(B + 1)), i32([kv] * B), 1, with_lse=True)
    ref = [np.repeat(r, B, 0) for r in ref]
    _check_faint(out, lse, ref, kv)


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("q_len,kv,faint", [
    (290, 900, lambda j: j < 128),                    # pieces of an item folded by the merge
    (290, 420, lambda j: j // 128 % 2 == 0),          # a block's even key tiles beside its odd ones
])
def test_a_value_that_is_nan_shows_in_a_chunk(kv_type, q_len, kv, faint):
    """The weights of one part of a row's keys are nothing beside those of the
    part it is joined with; NaN in that part's values stays."""
    args, ref, _ = _faint_case(kv_type, 1, q_len, kv, faint, 7)
    out, lse = sa.sa_paged_attn(*args, i32([0, q_len]), i32([kv]), q_len, with_lse=True)
    _check_faint(out, lse, ref, kv)


@pytest.mark.parametrize("kv_type", TYPES)
@pytest.mark.parametrize("q_len,kv", [([300], [400]), ([300], [1500]), ([200, 140], [230, 900])])
def test_values_that_are_not_finite_all_over_a_chunk(kv_type, q_len, kv):
    """Every new position has an element of V that is infinite or NaN, another
    one each: a token shows those of the positions it sees, in rows finished at
    once and in rows folded from pieces, and the same bits every time."""
    page, hkv, G = 16, 2, 2
    table, _ = _table(kv, page, _rng(35))

    def pools(n):
        out = [_random_pool(170 + i, n, page, hkv, kv_type) for i in range(2)]
        for b, (T, S) in enumerate(zip(q_len, kv)):
            for j in range(S - T, S):
                row, d = out[1][table[b, j // page], j % page], (7 * j) % 256
                if kv_type == P.BF16:
                    row[:hkv * 256].view(np.uint16)[d] = 0x7F80
                else:
                    row[d] = 0x7F
        return out

    runs = [_attn_case(35, kv_type, hkv, G, page, q_len, kv, pools=pools) for _ in range(4)]
    (got, lse, ref, n), bits = runs[0], [bits_of(r[0]) for r in runs]
    assert all(np.array_equal(b, bits[0]) for b in bits)
    odd = ~np.isfinite(ref[0])
    g = got.float().cpu().numpy()
    assert np.array_equal(~np.isfinite(g), odd)
    o, mag = (np.where(odd, 0.0, x) for x in (ref[0], ref[2]))
    _check_attn(torch.from_numpy(np.where(odd, 0.0, g)).to(dev()), lse, (o, ref[1], mag, ref[3]), n)


@pytest.mark.parametrize("kv_type", TYPES)
def test_host_threads_on_one_stream(kv_type):
    """Four threads call at once on the default stream, short and long chunks
    and selected rows, and share its workspace: each gets what it gets alone."""
    import threading

    hkv, G, page, kv = 2, 4, 16, [1900, 333, 60]
    table, num_pages = _table(kv, page, _rng(36))
    pools = [_dev_pool(_random_pool(180 + i, num_pages, page, hkv, kv_type), kv_type) for i in range(2)]
    tab, lens, work = i32(table), i32(kv), []
    for i, q_len in enumerate(([1, 1, 1], [90, 3, 1], [4, 40, 2])):
        q, start = to_dev(_normal(37 + i, 1, (sum(q_len), hkv * G, 128))), i32(np.cumsum([0] + q_len))
        work.append(lambda q=q, start=start, m=max(q_len): sa.sa_paged_attn(q, *pools, tab, start, lens, m, with_lse=True))
    qs, idx, cnt = to_dev(_normal(40, 1, (3, hkv * G, 128))), i32(np.tile(np.arange(50), (3, 1))), i32([50, 50, 7])
    work.append(lambda: sa.sa_paged_sparse_attn_decode(qs, *pools, tab, idx, cnt, with_lse=True))
    want = [w() for w in work]
    got, errors, gate = [[] for _ in work], [], threading.Barrier(len(work))

    def run(i):
        try:
            gate.wait()
            for _ in range(60):
                got[i].append(work[i]())
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for res, (o, l) in zip(got, want):
        assert len(res) == 60 and all(torch.equal(a, o) and torch.equal(b, l) for a, b in res)


@pytest.mark.parametrize("kv_type", TYPES)
def test_pools_past_four_gibibytes(kv_type):
    """Pages at the far end of pools of more than 2^32 bytes: rows written there
    are read back, and attended to, as from a small pool."""
    hkv, G, page = 8, 2, 64
    num_pages = (2 ** 32 + 2 ** 28) // (page * P.row_bytes(kv_type, hkv))
    dtype, row = (torch.bfloat16, hkv * 128 + 8) if kv_type == P.BF16 else (torch.uint8, hkv * 128 + 16)
    big = [torch.empty(num_pages, page, row, dtype=dtype, device=dev()) for _ in range(2)]
    assert big[0].numel() * big[0].element_size() > 2 ** 32
    q_len, kv = [200, 1, 3], [300, 129, 70]
    small_table, n = _table(kv, page, _rng(41))
    far = np.where(small_table >= 0, num_pages - 1 - small_table, small_table).astype(np.int32)
    small = sa.sa_paged_kv_alloc(n, page, hkv, kv_type, device=dev())
    lens, whole = i32(kv), np.cumsum([0] + kv)
    kn, vn = (to_dev(_normal(42 + i, 1, (sum(kv), hkv, 128))) for i in range(2))
    q, start = to_dev(_normal(44, 1, (sum(q_len), hkv * G, 128))), i32(np.cumsum([0] + q_len))
    idx, cnt = i32(np.stack([_rng(45 + b).integers(0, m, 48) for b, m in enumerate(kv)])), i32([48, 48, 20])
    res = []
    for pools, table in ((small, i32(small_table)), (big, i32(far))):
        sa.sa_paged_kv_write(kn, vn, *pools, table, i32(whole), lens)
        res.append([*sa.sa_paged_kv_gather(*pools, table, idx, cnt),
                    *sa.sa_paged_attn(q, *pools, table, start, lens, max(q_len), with_lse=True),
                    *sa.sa_paged_attn(q[-3:], *pools, table, i32([0, 1, 2, 3]), lens, 1, with_lse=True),
                    *sa.sa_paged_sparse_attn_decode(q[:3], *pools, table, idx, cnt, with_lse=True)])
    for a, b in zip(*res):
        assert torch.equal(a, b)
