"""The serving operators against plain float64 forms: kv_append,
attention_packed, attention_decode.

Tolerances, from the kernels' arithmetic.  Attention: scores, softmax and
sums are fp32 (errors near 2^-20 relative, growing with the scores: a score of
size z is off by at most (d + 2) 2^-24 |q| |k| scale, which moves its weight by
as much relative); the weights are rounded to the operand type before the
second product (half a step e relative each), the output once more:
    |o - o*| <= (e + 2^-14) * (p* |v|) + e * |o*| + tiny,
e = 2^-8 for bf16 and 2^-11 for fp16 (half a step is eps / 2), 2^-14 covers the
fp32 part for the sizes here, tiny = 2^-24 the subnormal steps of fp16 (a
weight below 2^-14 is rounded to a multiple of 2^-24, so 2^-25 each, times the
keys).  The logsumexp is fp32: 1e-5 (1 + |lse|).
Append: the rotation is two fp32 products and a sum of values that are at most
sqrt(2) max(|a|, |b|) with angles off by 2^-24 of a turn's half; rounded once:
    |y - y*| <= e |y*| + 2^-20 (|a| + |b|).
"""
import numpy as np
import pytest

import row_wise_softmax_gb300 as rws
from row_wise_softmax_gb300.serving import _packed_workspace
from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rws.build()
    rws.lib()
    rws.device_status(clear=True)


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype, by=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * by).to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def close(o, lse, want, dtype, n_keys, what=""):
    w, wl, mag = want
    e = HALF_STEP[dtype]
    got = f64(o)
    assert np.array_equal(np.isnan(got), np.isnan(w)), what
    fine = ~np.isnan(w)
    tiny = 2.0 ** -24 * max(1.0, n_keys * 2.0 ** -3)
    bound = (e + 2.0 ** -14) * mag + e * np.abs(w) + tiny
    err = np.abs(got - w)
    assert np.all(err[fine] <= bound[fine]), "%s: off by %.3g more than %.3g" % (
        what, float(np.max(np.where(fine, err - bound, -1))), float(bound[fine].min()))
    if lse is not None:
        got = f64(lse)
        fin = np.isfinite(wl)
        assert np.array_equal(got[~fin], wl[~fin]), what
        assert np.all(np.abs(got[fin] - wl[fin]) <= 1e-5 * (1 + np.abs(wl[fin]))), what


# ---------------------------------------------------------------- decode
def paged(g, lengths, page, hk, d, dtype, fill=None, spare=3, heads_first=False, width=None):
    """Caches with pages in no order; rows in no sequence hold `fill`."""
    need = [-(-n // page) for n in lengths]
    total = sum(need) + spare
    shape = (total, hk, page, d) if heads_first else (total, page, hk, d)
    k, v = (normal(g, *shape, dtype=dtype) for _ in range(2))
    if heads_first:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    order = torch.randperm(total, generator=g, device="cuda").tolist()
    table = np.full((len(lengths), width or max(1, max(need))), -7, np.int32)
    used = np.zeros((total, page), bool)
    for s, n in enumerate(lengths):
        for i in range(need[s]):
            table[s, i] = order.pop()
            used[table[s, i], :min(page, n - i * page)] = True
    if fill is not None:
        free = torch.from_numpy(~used).cuda()
        k[free] = fill
        v[free] = fill
    return k, v, table


def decode_case(lengths, h, hk, d, page, dtype, seed, fill=float("nan"), by=1.5, **kw):
    g = rng(seed)
    k, v, table = paged(g, lengths, page, hk, d, dtype, fill, **kw)
    q = normal(g, len(lengths), h, d, dtype=dtype, by=by)
    o, lse = rws.attention_decode(q, k, v, torch.from_numpy(table).cuda(), ints(lengths),
                                  return_lse=True)
    want = ref.decode(f64(q), f64(k), f64(v), table, lengths, d ** -0.5)
    close(o, lse, want, dtype, max(lengths), "lengths %s" % (lengths[:8],))
    assert rws.device_status() == rws.OK


DECODE = [  # lengths, heads, kv_heads, head_dim, page
    ([1], 1, 1, 64, 1),
    ([1, 2, 15, 16, 17], 8, 2, 128, 16),
    ([63, 64, 65, 127, 128, 129], 4, 4, 64, 16),
    ([700], 32, 8, 128, 16),
    ([0, 5, 0, 200, 0], 6, 2, 128, 8),              # empty sequences: NaN, -inf
    ([333, 1, 40], 5, 1, 64, 24),                   # pages that are no power of two
    ([1000, 900], 16, 1, 128, 7),                   # sixteen heads to one
    ([257, 130], 40, 2, 64, 32),                    # twenty: two blocks of heads
    ([100, 65], 33, 1, 128, 128),                   # thirty-three: three, one head in the last
    ([2000, 3, 1999, 64], 12, 4, 128, 64),
    ([20000], 8, 2, 128, 16),                       # one sequence over every CTA
    ([37] * 70, 4, 2, 64, 16),                      # many short ones
    ([5, 0, 300, 64, 65, 1000, 0, 33] * 12, 8, 4, 64, 16),           # four heads abreast
    ([5, 0, 300, 64, 65, 1000, 0, 33] * 22, 18, 2, 64, 16),          # two, and two blocks of heads
]


@pytest.mark.parametrize("dtype", list(TYPES.values()), ids=list(TYPES))
@pytest.mark.parametrize("i", range(len(DECODE)))
def test_decode(i, dtype):
    decode_case(*DECODE[i], dtype, 100 + i)


@pytest.mark.parametrize("i", range(len(DECODE)))
def test_decode_behind_a_wide_table(i):
    """The same through the kernels of long calls: a table with room for far
    more tokens than there are decides the launch."""
    lengths, h, hk, d, page = DECODE[i]
    decode_case(lengths, h, hk, d, page, torch.bfloat16, 130 + i, width=400000 // page + 1)


@pytest.mark.parametrize("width", [None, 40000])
def test_decode_different_strides_of_k_and_v(width):
    g = rng(9)
    lengths, page, hk, d = [90, 200, 7], 16, 2, 128
    k, _, table = paged(g, lengths, page, hk, d, torch.bfloat16, width=width)
    _, v, _ = paged(g, lengths, page, hk, d, torch.bfloat16, heads_first=True)
    v = v[:k.shape[0]]
    q = normal(g, 3, 8, d, dtype=torch.bfloat16)
    o = rws.attention_decode(q, k, v, torch.from_numpy(table).cuda(), ints(lengths))
    close(o, None, ref.decode(f64(q), f64(k), f64(v), table, lengths, d ** -0.5), q.dtype, 200)


@pytest.mark.parametrize("group", [48, 128])
@pytest.mark.parametrize("width", [None, 40000])
def test_decode_many_heads_to_one(group, width):
    decode_case([300, 5], group, 1, 64, 16, torch.bfloat16, 10, width=width)


def test_decode_strided_in_place_and_lse_only_rows():
    """q a part of a projection's output, out = q, and a scale."""
    g = rng(11)
    lengths, page, h, hk, d = [100, 0, 33], 16, 4, 2, 128
    k, v, table = paged(g, lengths, page, hk, d, torch.float16)
    wide = normal(g, 3, h + 2, d, dtype=torch.float16)
    q, rest = wide[:, :h], wide[:, h:].clone()
    want = ref.decode(f64(q), f64(k), f64(v), table, lengths, 0.3)
    o, lse = rws.attention_decode(q, k, v, torch.from_numpy(table).cuda(), ints(lengths), scale=0.3,
                                  out=q, return_lse=True)
    assert o is q and torch.equal(wide[:, h:], rest)
    close(o, lse, want, torch.float16, 100)


@pytest.mark.parametrize("width", [16, 40000])
def test_decode_bad_pages_and_lengths(width):
    """A sequence with a bad page or length gives NaN and a status; the others
    are as ever, and a bad page past a sequence's length is not looked at."""
    g = rng(12)
    lengths, page, h, hk, d = [200, 64, 130, 50, 9], 16, 8, 2, 128
    k, v, table = paged(g, lengths, page, hk, d, torch.bfloat16, width=width)
    q = normal(g, 5, h, d, dtype=torch.bfloat16)
    want = ref.decode(f64(q), f64(k), f64(v), table, lengths, d ** -0.5)
    table[1, 3] = k.shape[0]                        # the first page that is not there
    table[2, 0] = -1
    table[4, 1] = 1 << 30                           # past the length
    n = list(lengths)
    n[3] = width * page + 1
    for bad in (n[3], -1):
        n[3] = bad
        o, lse = rws.attention_decode(q, k, v, torch.from_numpy(table).cuda(), ints(n),
                                      return_lse=True)
        assert bool(torch.isnan(o[1:4]).all()) and bool(torch.isnan(lse[1:3]).all())
        ok = [0, 4]
        close(o[ok], lse[ok], [w[ok] for w in want], torch.bfloat16, 200)
        assert rws.device_status(clear=False) == rws.ERR_DEVICE_INDEX
        assert rws.device_status() == rws.ERR_DEVICE_INDEX
        assert rws.device_status() == rws.OK


def test_decode_far_pages():
    """Rows more than 2^31 elements into the caches."""
    page, hk, d = 16, 8, 128
    pages = (1 << 31) // (page * hk * d) + 40
    k = torch.empty(pages, page, hk, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    g = rng(13)
    for c in (k, v):
        c[-30:] = normal(g, 30, page, hk, d, dtype=torch.bfloat16)
    table = (pages - 30 + np.random.default_rng(1).permutation(30)).astype(np.int32).reshape(2, 15)
    q = normal(g, 2, 16, d, dtype=torch.bfloat16)
    lengths = [240, 177]
    got = rws.attention_decode(q, k, v, torch.from_numpy(table).cuda(), ints(lengths))
    near = table - (pages - 30)
    close(got, None, ref.decode(f64(q), f64(k[-30:]), f64(v[-30:]), near, lengths, d ** -0.5),
          q.dtype, 240)
    pos = ints([241, 180])
    k2, v2 = (normal(g, 2, hk, d, dtype=torch.bfloat16) for _ in range(2))
    table = np.concatenate([table, [[pages - 1], [pages - 2]]], 1).astype(np.int32)
    rws.kv_append(k2, v2, k, v, torch.from_numpy(table).cuda(), pos)
    assert torch.equal(k[pages - 1, 1], k2[0]) and torch.equal(v[table[1, 11], 4], v2[1])
    assert rws.device_status() == rws.OK


def test_decode_heads_first_pages_and_wide_table():
    decode_case([130, 77, 1], 8, 2, 128, 16, torch.bfloat16, 7, heads_first=True, width=40)


def test_decode_large_scores():
    decode_case([300, 1000], 8, 2, 64, 16, torch.float16, 8, by=24.0)


# ---------------------------------------------------------------- packed
def packed_case(n_q, n_k, h, hk, d, causal, dtype, seed, fused=False, scale=None, by=1.5):
    g = rng(seed)
    t, m = sum(n_q), sum(n_k)
    if fused:
        qkv = normal(g, t, (h + 2 * hk), d, dtype=dtype)
        q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
    else:
        q = normal(g, t, h, d, dtype=dtype, by=by)
        k, v = (normal(g, m, hk, d, dtype=dtype) for _ in range(2))
    cu_q, cu_k = np.cumsum([0] + n_q), np.cumsum([0] + n_k)
    o, lse = rws.attention_packed(q, k, v, ints(cu_q), ints(cu_k), scale=scale, causal=causal,
                                  return_lse=True)
    want = ref.packed(f64(q), f64(k), f64(v), cu_q, cu_k, scale or d ** -0.5, causal)
    close(o, lse, want, dtype, max(n_k), "n_q %s n_k %s" % (n_q, n_k))
    assert rws.device_status() == rws.OK


PACKED = [  # n_q, n_k, heads, kv_heads, head_dim, causal, fused
    ([1], [1], 1, 1, 64, True, False),
    ([90], [90], 8, 2, 128, True, False),
    ([1, 2, 127, 128, 129], [1, 2, 127, 128, 129], 4, 2, 64, True, True),
    ([255, 0, 256, 257, 3], [255, 0, 256, 257, 3], 6, 3, 128, True, True),
    ([5, 130, 0, 60], [500, 131, 9, 60], 8, 1, 128, True, False),    # behind a context
    ([70, 5], [30, 0], 4, 4, 64, True, False),      # queries that see nothing: NaN
    ([33, 200, 1], [1, 77, 300], 5, 5, 64, False, False),
    ([100, 300], [100, 300], 12, 12, 64, False, True),
    ([40, 600], [40, 600], 10, 2, 128, True, False),                 # five heads to one
    ([64] * 20, [64] * 20, 3, 1, 128, True, True),                   # three heads to one
    ([700], [1500], 16, 1, 64, True, False),                         # sixteen heads to one
]


@pytest.mark.parametrize("dtype", list(TYPES.values()), ids=list(TYPES))
@pytest.mark.parametrize("i", range(len(PACKED)))
def test_packed(i, dtype):
    n_q, n_k, h, hk, d, causal, fused = PACKED[i]
    packed_case(n_q, n_k, h, hk, d, causal, dtype, 200 + i, fused)


def test_packed_many_sequences():
    """More sequences than the kernel ranks by length, and units that see no key."""
    r = np.random.default_rng(3)
    n_q = [int(x) for x in r.integers(0, 40, 300)]
    n_k = [max(0, n + int(r.integers(-8, 30))) for n in n_q]
    packed_case(n_q, n_k, 4, 2, 64, True, torch.bfloat16, 81)
    packed_case(n_q, n_k, 2, 1, 128, False, torch.float16, 82)


@pytest.mark.parametrize("group", [32, 48, 128])
def test_packed_many_heads_to_one(group):
    packed_case([70, 3], [70, 100], group, 1, 128, True, torch.bfloat16, 83)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("in_place", [False, True])
def test_packed_unseen_values_have_no_influence(d, bad, in_place):
    """Keys and values of other sequences, behind the last one, and past the
    diagonal hold NaN or infinity: a query that does not see them is as if
    they were not there; one that does has them in its output."""
    g = rng(84)
    lens, h, hk, dtype = [150, 70, 200], 4, 2, torch.bfloat16
    cu = np.cumsum([0] + lens)
    t = cu[-1]
    q = normal(g, t + 9, h, d, dtype=dtype)
    k, v = (normal(g, t + 9, hk, d, dtype=dtype) for _ in range(2))
    k[cu[1]:cu[2]] = bad                            # the sequence between
    v[cu[1]:cu[2]] = bad
    k[t:], v[t:] = bad, bad
    v[cu[2] + 130] = bad                            # a later token of the last
    v[90, 0, 3] = bad                               # one value of a token of the first
    want, _, mag = ref.packed(f64(q), f64(k), np.where(np.isfinite(f64(v)), f64(v), 0.0), cu, cu,
                              d ** -0.5, True)
    out = q.clone() if in_place else torch.full_like(q, 3.0)
    o = rws.attention_packed(out if in_place else q, k, v, ints(cu), causal=True, out=out)
    got = f64(o)
    assert np.array_equal(got[t:], f64(q)[t:] if in_place else np.full(got[t:].shape, 3.0))
    seen = np.zeros(got.shape, bool)                # outputs that such a value reaches
    seen[90:cu[1], :h // hk, 3] = True
    seen[cu[1]:cu[2]] = True
    seen[cu[2] + 130:t] = True
    seen[t:] = True
    assert np.all(np.isfinite(got[~seen]))
    bound = (2.0 ** -8 + 2.0 ** -14) * mag + 2.0 ** -8 * np.abs(want) + 2.0 ** -24
    assert np.all(np.abs(got - want)[~seen] <= bound[~seen])
    seen[t:] = False
    assert not np.any(np.isfinite(got[seen]))
    assert rws.device_status() == rws.OK


def test_packed_rows_in_no_sequence_stay():
    g = rng(85)
    h, hk, d, dtype = 2, 1, 128, torch.float16
    q = normal(g, 400, h, d, dtype=dtype)
    k, v = (normal(g, 400, hk, d, dtype=dtype) for _ in range(2))
    cu = np.array([17, 100, 100, 333])
    out = torch.full_like(q, -5.0)
    o, lse = rws.attention_packed(q, k, v, ints(cu), out=out, return_lse=True)
    want = ref.packed(f64(q), f64(k), f64(v), cu, cu, d ** -0.5, True)
    close(o[17:333], lse[17:333], [w[17:333] for w in want], dtype, 233)
    assert bool((out[:17] == -5).all()) and bool((out[333:] == -5).all())


def test_packed_bad_bounds():
    g = rng(86)
    h, d, dtype = 2, 64, torch.bfloat16
    q, k, v = (normal(g, 300, h, d, dtype=dtype) for _ in range(3))
    good = np.array([0, 50, 120, 200, 300])
    want, _, mag = ref.packed(f64(q), f64(k), f64(v), good, good, d ** -0.5, True)
    # (Rows 40 to 49 of the first lie in two sequences: either's.)
    for cu, ok in ((np.array([0, 50, 40, 200, 300]), [(0, 40), (200, 300)]),
                   (np.array([0, 50, 120, 301, 1 << 30]), [(0, 50), (50, 120)]),
                   (np.array([-3, 50, 120, 200, 300]), [(50, 120), (120, 200), (200, 300)])):
        out = torch.full_like(q, 9.0)
        rws.attention_packed(q, k, v, ints(cu), out=out)
        assert rws.device_status() == rws.ERR_DEVICE_INDEX
        got = f64(out)
        for a, b in ok:
            bound = 2.0 ** -7 * (mag + np.abs(want)) + 1e-6
            assert np.all(np.abs(got - want)[a:b] <= bound[a:b])
    assert rws.device_status() == rws.OK


def test_packed_repeated_and_missing_keys():
    """Heads of K and V that are one in memory (stride 0), and no key at all."""
    g = rng(87)
    n, h, d, dtype = 60, 4, 64, torch.bfloat16
    q = normal(g, n, h, d, dtype=dtype)
    k1, v1 = (normal(g, n, 1, d, dtype=dtype) for _ in range(2))
    cu = np.array([0, 25, 60])
    o, lse = rws.attention_packed(q, k1.expand(n, 2, d), v1.expand(n, 2, d), ints(cu),
                                  return_lse=True)
    two = [np.repeat(f64(x), 2, 1) for x in (k1, v1)]
    close(o, lse, ref.packed(f64(q), *two, cu, cu, d ** -0.5, True), dtype, 35)
    none = torch.empty(0, 2, d, dtype=dtype, device="cuda")
    o, lse = rws.attention_packed(q, none, none, ints([0, 25, 60]), ints([0, 0, 0]), causal=False,
                                  return_lse=True)
    assert bool(torch.isnan(o).all()) and bool((lse == float("-inf")).all())
    assert rws.device_status() == rws.OK


FEW = [  # few query rows over long sequences, whose keys are cut into parts
    ([1], [3000], 8, 2, 128, True),
    ([4, 0, 37], [2500, 600, 1100], 8, 2, 64, True),
    ([130], [5000], 4, 4, 128, False),
    ([300], [1300], 2, 1, 64, True),
    ([70, 9], [40, 6000], 6, 3, 128, True),         # sees nothing; fewer tiles than parts
    ([513], [1281], 1, 1, 128, True),
    ([2, 3, 5], [1500, 1409, 4097], 10, 2, 128, False),
    ([700], [1500], 3, 1, 64, True),
]


@pytest.mark.parametrize("dtype", list(TYPES.values()), ids=list(TYPES))
@pytest.mark.parametrize("i", range(len(FEW)))
def test_packed_few_queries(i, dtype):
    n_q, n_k, h, hk, d, causal = FEW[i]
    assert _packed_workspace(0, len(n_q), sum(n_q), sum(n_k), h, hk, d) > 0
    packed_case(n_q, n_k, h, hk, d, causal, dtype, 400 + i, False)
    packed_case(n_q, n_k, h, hk, d, causal, dtype, 400 + i, False, by=3.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
def test_packed_few_queries_unseen_values(d, bad):
    """Such values in parts of a sequence, one of them seen by late queries
    only; out in the place of q; rows behind the last sequence."""
    g = rng(88)
    n_q, n_k, h, hk, dtype = 200, 2600, 4, 2, torch.float16
    q = normal(g, n_q + 5, h, d, dtype=dtype)
    k, v = (normal(g, n_k + 300, hk, d, dtype=dtype) for _ in range(2))
    k[n_k:], v[n_k:] = bad, bad                     # behind the sequence
    v[n_k - 50, 1, 5] = bad                         # seen by its last 50 queries, heads 2 and 3
    cu_q, cu_k = np.array([0, n_q]), np.array([0, n_k])
    assert _packed_workspace(0, 1, n_q + 5, n_k + 300, h, hk, d) > 0
    want, _, mag = ref.packed(f64(q), f64(k), np.where(np.isfinite(f64(v)), f64(v), 0.0), cu_q,
                              cu_k, d ** -0.5, True)
    before = f64(q)
    got = f64(rws.attention_packed(q, k, v, ints(cu_q), ints(cu_k), out=q))
    assert np.array_equal(got[n_q:], before[n_q:])
    seen = np.zeros(got.shape, bool)
    seen[n_q - 50:n_q, 2:, 5] = True
    seen[n_q:] = True
    bound = (2.0 ** -11 + 2.0 ** -14) * mag + 2.0 ** -11 * np.abs(want) + 2.0 ** -24 * n_k
    assert np.all(np.abs(got - want)[~seen] <= bound[~seen])
    assert not np.any(np.isfinite(got[n_q - 50:n_q, 2:, 5]))
    assert rws.device_status() == rws.OK


def test_packed_few_queries_bad_bounds_and_graph():
    g = rng(89)
    h, hk, d, dtype = 8, 2, 128, torch.bfloat16
    q = normal(g, 12, h, d, dtype=dtype)
    k, v = (normal(g, 4000, hk, d, dtype=dtype) for _ in range(2))
    cu_q, cu_k = ints([0, 5, 12]), ints([0, 1900, 4000])
    want, wl, mag = ref.packed(f64(q), f64(k), f64(v), [0, 5, 12], [0, 1900, 4000], d ** -0.5, True)
    out = torch.full_like(q, 4.0)
    rws.attention_packed(q, k, v, cu_q, ints([0, 1900, 4001]), out=out)
    assert rws.device_status(clear=True) == rws.ERR_DEVICE_INDEX
    assert bool((out[5:] == 4).all())
    close(out[:5], None, [w[:5] for w in (want, wl, mag)], dtype, 4000)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        rws.attention_packed(q, k, v, cu_q, cu_k)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            o, lse = rws.attention_packed(q, k, v, cu_q, cu_k, return_lse=True)
    first = None
    for _ in range(3):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        first = o.clone() if first is None else first
        assert torch.equal(o, first)                # the join's order is fixed
    close(o, lse, (want, wl, mag), dtype, 4000)
    assert rws.device_status() == rws.OK


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_packed_many_units_per_cta(d, causal):
    """Several times more units of work than fit on the device, with query
    tiles that end at different key tiles (or have no rows), checked head by
    head against float64 on the device."""
    r = np.random.default_rng(17)
    n_q = [int(x) for x in r.integers(1, 900, 40)] + [0, 1, 513, 257]
    n_k = [n + int(r.integers(-60, 300)) if n > 100 else n for n in n_q]
    h, hk, dtype = 16, 16, torch.bfloat16
    g = rng(61)
    q = normal(g, sum(n_q), h, d, dtype=dtype, by=1.5)
    k, v = (normal(g, sum(n_k), hk, d, dtype=dtype) for _ in range(2))
    cu_q, cu_k = np.cumsum([0] + n_q), np.cumsum([0] + n_k)
    for _ in range(3):
        o = rws.attention_packed(q, k, v, ints(cu_q), ints(cu_k), causal=causal)
    assert rws.device_status() == rws.OK
    for s in range(len(n_q)):
        a, b, c, e = cu_q[s], cu_q[s + 1], cu_k[s], cu_k[s + 1]
        qs, ks, vs = (x.double().transpose(0, 1) for x in (q[a:b], k[c:e], v[c:e]))
        z = qs @ ks.transpose(1, 2) * d ** -0.5
        if causal:
            i, j = torch.arange(b - a, device="cuda"), torch.arange(e - c, device="cuda")
            z.masked_fill_(j[None] > i[:, None] + (e - c) - (b - a), float("-inf"))
        w = torch.softmax(z, -1)
        want, mag = ((w @ x).transpose(0, 1) for x in (vs, vs.abs()))
        got = o[a:b].double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        bound = (2.0 ** -8 + 2.0 ** -14) * mag + 2.0 ** -8 * want.abs() + 2.0 ** -24
        fine = ~torch.isnan(want)
        assert bool(((got - want).abs()[fine] <= bound[fine]).all()), (s, n_q[s], n_k[s])


# ---------------------------------------------------------------- append
def append_case(n, h, hk, d, rot, interleaved, page, dtype, seed, far=5000, positions=None,
                seq_ids=None, n_seqs=None, in_place=False):
    g = rng(seed)
    qkv = normal(g, n, h + 2 * hk, d, dtype=dtype)
    q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
    pos = np.random.default_rng(seed).integers(0, far, n) if positions is None else positions
    seqs = n if seq_ids is None else n_seqs
    row = np.arange(n) if seq_ids is None else seq_ids
    width = max(int(max(pos)), 0) // page + 1
    # One page for each (sequence, page) that is written; the rest of the table is bad.
    table = np.full((seqs, width), -1, np.int32)
    want_page = sorted({(int(r), int(p) // page) for r, p in zip(row, pos) if p >= 0})
    order = np.random.default_rng(seed + 1).permutation(len(want_page) + 2)
    for i, (r, c) in enumerate(want_page):
        table[r, c] = order[i]
    kc, vc = (normal(g, len(order), page, hk, d, dtype=dtype) for _ in range(2))
    inv = 10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    want_k, want_v = f64(kc), f64(vc)
    before = f64(q), f64(k), f64(v)
    q0 = f64(torch.full_like(q, 7.0))
    out = q if in_place else torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    got = rws.kv_append(k, v, kc, vc, torch.from_numpy(table).cuda(), ints(pos),
                        None if seq_ids is None else ints(seq_ids), q=q, q_out=out,
                        inv_freq=torch.tensor(inv, device="cuda") if rot else None,
                        interleaved=interleaved)
    assert got is out
    e = HALF_STEP[dtype]

    def tolerance(x, y):
        size = np.abs(x)
        half = rot // 2
        pair = size.copy()
        if interleaved:
            pair[..., 0:rot:2] += size[..., 1:rot:2]
            pair[..., 1:rot:2] += size[..., 0:rot:2]
        else:
            pair[..., :half] += size[..., half:rot]
            pair[..., half:rot] += size[..., :half]
        return e * np.abs(y) + 2.0 ** -20 * pair + 2.0 ** -25

    keep = np.asarray(pos) >= 0
    turned_q = ref.rotate(before[0], pos, inv[:rot // 2], interleaved)
    turned_k = ref.rotate(before[1], pos, inv[:rot // 2], interleaved)
    tol_k = np.zeros(want_k.shape)
    for t in np.nonzero(keep)[0]:
        at = table[row[t], pos[t] // page], pos[t] % page
        want_k[at], want_v[at] = turned_k[t], before[2][t]
        tol_k[at] = tolerance(before[1][t], turned_k[t])
    assert np.all(np.abs(f64(kc) - want_k) <= tol_k)
    assert np.array_equal(f64(vc), want_v)
    have = f64(out)
    assert np.all(np.abs(have - turned_q)[keep] <= tolerance(before[0], turned_q)[keep])
    if not in_place:
        assert np.array_equal(have[~keep], q0[~keep])
    assert np.array_equal(f64(k), before[1]) and np.array_equal(f64(v), before[2])
    assert rws.device_status() == rws.OK


APPEND = [  # tokens, heads, kv_heads, head_dim, rot_dim, interleaved, page
    (1, 1, 1, 64, 64, False, 1),
    (8, 32, 8, 128, 128, False, 16),
    (77, 6, 2, 128, 64, True, 24),
    (33, 5, 1, 64, 32, False, 7),
    (9, 4, 4, 64, 16, True, 64),
    (12, 4, 4, 128, 16, False, 64),
    (5, 3, 3, 128, 0, False, 16),
    (1500, 8, 2, 64, 64, True, 16),
    (1201, 3, 1, 128, 96, False, 32),
    (5003, 3, 1, 128, 64, True, 16),
    (4098, 4, 2, 64, 64, False, 8),
]


@pytest.mark.parametrize("dtype", list(TYPES.values()), ids=list(TYPES))
@pytest.mark.parametrize("i", range(len(APPEND)))
def test_append(i, dtype):
    append_case(*APPEND[i], dtype, 300 + i)


def test_append_far_positions():
    """Positions near 2^30: the angle modulo a turn keeps its precision.  A
    float64 product of such a position and a frequency is off by 2^-53 * 2^30
    radians, far below the tolerance."""
    n = 64
    pos = (1 << 20) - 1 - np.arange(n) * 777
    append_case(n, 4, 2, 128, 128, False, 1 << 14, torch.float16, 31, positions=pos,
                seq_ids=np.zeros(n, np.int64), n_seqs=1)


def test_append_packed_prompts_padding_and_in_place():
    ids = np.repeat([0, 1, 2], [40, 1, 30])
    pos = np.concatenate([np.arange(40) + 100, [0], np.arange(30)])
    pos[[3, 50]] = -1                               # padding
    append_case(len(ids), 4, 2, 64, 64, False, 16, torch.bfloat16, 32, positions=pos,
                seq_ids=ids, n_seqs=3, in_place=True)


def test_append_bad_indexes_write_nothing():
    """Bad sequences, positions and pages: a status, and no cache row but the
    good token's changes; queries are turned all the same."""
    g = rng(40)
    page, hk, d, dtype = 8, 2, 64, torch.bfloat16
    kc, vc = (normal(g, 4, page, hk, d, dtype=dtype) for _ in range(2))
    k, v = (normal(g, 6, hk, d, dtype=dtype) for _ in range(2))
    q = normal(g, 6, 3, d, dtype=dtype)
    table = ints([[0, 1], [2, 4], [-1, 3]])
    ids, pos = ints([0, 7, -1, 1, 2, 0]), ints([3, 0, 0, 8, 1, 16])
    before_k, before_v = kc.clone(), vc.clone()
    inv = torch.ones(8, dtype=torch.float64, device="cuda")
    out = rws.kv_append(k, v, kc, vc, table, pos, ids, q=q, inv_freq=inv)
    assert rws.device_status() == rws.ERR_DEVICE_INDEX and rws.device_status() == rws.OK
    want = ref.rotate(f64(k), [3] * 6, np.ones(8), False)[0]
    assert np.all(np.abs(f64(kc[0, 3]) - want) <= 2.0 ** -8 * np.abs(want) + 1e-5)
    assert torch.equal(vc[0, 3], v[0])
    kc[0, 3], vc[0, 3] = before_k[0, 3], before_v[0, 3]
    assert torch.equal(kc, before_k) and torch.equal(vc, before_v)
    want = ref.rotate(f64(q), pos.tolist(), np.ones(8), False)
    assert np.all(np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + 1e-5)


def test_append_into_one_interleaved_cache_tensor():
    g = rng(41)
    cache = torch.zeros(5, 2, 16, 2, 128, dtype=torch.float16, device="cuda")
    k, v = (normal(g, 20, 2, 128, dtype=torch.float16) for _ in range(2))
    rws.kv_append(k, v, cache[:, 0], cache[:, 1], ints([[3, 1]]), ints(list(range(20))),
                  ints([0] * 20))
    assert torch.equal(cache[3, 0], k[:16]) and torch.equal(cache[3, 1], v[:16])
    assert torch.equal(cache[1, 0, :4], k[16:]) and torch.equal(cache[1, 1, :4], v[16:])
    assert not cache[1, :, 4:].any() and not cache[[0, 2, 4]].any()


# ------------------------------------------------------------- together
def test_prompt_then_steps():
    """Prompts through kv_append and attention_packed, then three decoding
    steps, against one attention over everything in float64."""
    g = rng(50)
    lens, steps, h, hk, d, page = [37, 1, 130], 3, 8, 2, 128, 16
    dtype, e = torch.bfloat16, HALF_STEP[torch.bfloat16]
    b, cu = len(lens), np.cumsum([0] + lens)
    inv = 10000.0 ** (-np.arange(d // 2) / (d // 2))
    freq = torch.tensor(inv, device="cuda")
    width = -(-(max(lens) + steps) // page)
    table = torch.randperm(b * width, generator=g, device="cuda").int().view(b, width)
    kc = torch.full((b * width, page, hk, d), float("nan"), dtype=dtype, device="cuda")
    vc = kc.clone()
    qkv = normal(g, int(cu[-1]), h + 2 * hk, d, dtype=dtype)
    ids = np.repeat(np.arange(b), lens)
    pos = np.concatenate([np.arange(n) for n in lens])
    q = rws.kv_append(qkv[:, h:h + hk], qkv[:, h + hk:], kc, vc, table, ints(pos), ints(ids),
                      q=qkv[:, :h], inv_freq=freq)
    keys = torch.stack([kc[table[s, p // page], p % page] for s, p in zip(ids, pos)])
    values = torch.stack([vc[table[s, p // page], p % page] for s, p in zip(ids, pos)])
    assert torch.equal(values, qkv[:, h + hk:])
    out = rws.attention_packed(q, keys, values, ints(cu))
    close(out, None, ref.packed(f64(q), f64(keys), f64(values), cu, cu, d ** -0.5, True), dtype, 130)
    now = list(lens)
    for _ in range(steps):
        qkv = normal(g, b, h + 2 * hk, d, dtype=dtype)
        q = rws.kv_append(qkv[:, h:h + hk], qkv[:, h + hk:], kc, vc, table, ints(now), q=qkv[:, :h],
                          inv_freq=freq)
        turned = ref.rotate(f64(qkv[:, :h]), now, inv, False)
        assert np.all(np.abs(f64(q) - turned) <= e * np.abs(turned) + 1e-5)
        now = [n + 1 for n in now]
        out = rws.attention_decode(q, kc, vc, table, ints(now))
        close(out, None, ref.decode(f64(q), f64(kc), f64(vc), table.cpu().numpy(), now, d ** -0.5),
              dtype, max(now))
    assert rws.device_status() == rws.OK


def everything(g, dtype=torch.bfloat16):
    """Inputs of one call of each operator, and the call."""
    lens = [70, 300, 5]
    k, v, table = paged(g, [4000, 90, 0, 700], 16, 2, 128, dtype, width=20000)
    s = dict(k=k, v=v, table=torch.from_numpy(table).cuda(), lengths=ints([4000, 90, 0, 700]),
             q=normal(g, 4, 8, 128, dtype=dtype), pq=normal(g, 375, 8, 128, dtype=dtype),
             pk=normal(g, 375, 2, 128, dtype=dtype), pv=normal(g, 375, 2, 128, dtype=dtype),
             cu=ints(np.cumsum([0] + lens)), kc=torch.zeros_like(k), vc=torch.zeros_like(v),
             pos=ints([7, 30, -1, 16]), freq=torch.rand(64, dtype=torch.float64, device="cuda"))

    def call(stream=None):
        return (rws.attention_decode(s["q"], s["k"], s["v"], s["table"], s["lengths"],
                                     stream=stream),
                rws.attention_decode(s["q"], s["k"], s["v"], s["table"][:, :250].contiguous(),
                                     s["lengths"], stream=stream),
                rws.attention_packed(s["pq"], s["pk"], s["pv"], s["cu"], stream=stream),
                rws.kv_append(s["pk"][:4], s["pv"][:4], s["kc"], s["vc"], s["table"], s["pos"],
                              q=s["q"], inv_freq=s["freq"], stream=stream)[:2],
                s["kc"], s["vc"])
    return s, call


def test_same_bits_on_every_run_and_stream():
    s, call = everything(rng(51))
    want = [x.clone() for x in call()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        got = [call(st) for st in streams] + [call(st.cuda_stream) for st in streams]
        torch.cuda.synchronize()
        for outs in got:
            for a, b in zip(outs, want):
                assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_graph_replay_reads_new_lengths():
    """Two graphs that hold the same calls, replayed side by side with other
    lengths, bounds and inputs than were captured."""
    s, call = everything(rng(52))
    call()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = call()[:3]
        graphs.append((graph, outs, torch.cuda.Stream()))
    s["lengths"].copy_(ints([100, 3999, 64, 0]))
    s["table"].copy_(torch.where(s["table"] < 0, 0, s["table"]))
    s["cu"].copy_(ints([10, 11, 200, 375]))
    s["q"].mul_(0.5)
    want = [x.clone() for x in call()[:3]]
    torch.cuda.synchronize()
    for _ in range(4):
        for graph, _, st in graphs:
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
    for _, outs, _ in graphs:
        for n, (a, b) in enumerate(zip(outs, want)):
            if n == 2:                              # rows before cu[0] are nobody's
                a, b = a[10:], b[10:]
            assert torch.equal(a.view(torch.int16), b.view(torch.int16)), n


def test_binding_checks():
    s, _ = everything(rng(53))
    cpu = s["q"].cpu()
    with pytest.raises(ValueError):
        rws.attention_decode(cpu, s["k"], s["v"], s["table"], s["lengths"])
    with pytest.raises(ValueError):
        rws.attention_decode(s["q"], s["k"].cpu(), s["v"], s["table"], s["lengths"])
    with pytest.raises(TypeError):
        rws.attention_decode(s["q"].float(), s["k"], s["v"], s["table"], s["lengths"])
    with pytest.raises(ValueError):
        rws.attention_decode(s["q"], s["k"], s["v"], s["table"].long(), s["lengths"])
    with pytest.raises(ValueError):
        rws.attention_decode(s["q"], s["k"], s["v"], s["table"], s["lengths"][:3])
    with pytest.raises(ValueError):
        rws.attention_packed(s["pq"][:, :3], s["pk"], s["pv"], s["cu"])
    with pytest.raises(ValueError):
        rws.attention_packed(s["pq"], s["pk"], s["pv"], s["cu"].long())
    with pytest.raises(rws.SoftmaxError):           # a head_dim that is not offered
        rws.attention_packed(*(s[x][..., :96].contiguous() for x in ("pq", "pk", "pv")), s["cu"])
    with pytest.raises(rws.SoftmaxError):           # out over k
        rws.attention_packed(s["pk"], s["pk"], s["pv"], s["cu"], out=s["pv"])
    with pytest.raises(ValueError):
        rws.kv_append(s["pk"][:5], s["pv"][:5], s["kc"], s["vc"], s["table"], ints([0] * 5))
    with pytest.raises(rws.SoftmaxError):           # rot_dim past head_dim
        rws.kv_append(s["pk"][:4], s["pv"][:4], s["kc"], s["vc"], s["table"], s["pos"],
                      inv_freq=torch.ones(72, dtype=torch.float64, device="cuda"))
    before = rws.launch_count()
    rws.attention_packed(s["pq"][:0], s["pk"], s["pv"], ints([0, 0]), ints([0, 375]))
    rws.attention_decode(s["q"][:0], s["k"], s["v"], s["table"][:0], s["lengths"][:0])
    rws.kv_append(s["pk"][:0], s["pv"][:0], s["kc"], s["vc"], s["table"], s["pos"][:0])
    assert rws.launch_count() == before             # nothing to do
    assert rws.device_status() == rws.OK


def test_decode_outputs_in_the_workspace_are_refused():
    from row_wise_softmax_gb300 import serving as sv
    lib = sv._lib()
    b, h, d, pages, size = 2, 4, 128, 256, 64
    need = lib.softmax_attention_decode_workspace(b, h, 1, d, 1 << 19)
    assert need >= 4096                               # not the form that needs none
    kc = torch.zeros(pages, size, 1, d, device="cuda", dtype=torch.bfloat16)
    vc, q = torch.zeros_like(kc), torch.zeros(b, h, d, device="cuda", dtype=torch.bfloat16)
    table = torch.zeros(b, (1 << 19) // size, device="cuda", dtype=torch.int32)
    lengths, ws = ints([5, 70]), torch.zeros(need + 1024, device="cuda", dtype=torch.uint8)
    c = sv._cache("t", kc, vc, table, kc.shape, kc.dtype, 0)
    x, o = sv._heads("t", "q", q, q.dtype, 0), torch.empty_like(q)

    def call(out, lse):
        return lib.softmax_attention_decode(c, x, out, lse, h, lengths.data_ptr(), 1.0, rws.BF16,
                                            ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    y = sv._heads("t", "o", o, o.dtype, 0)
    inside = sv._HEADS(ws.data_ptr() + 512, h * d, d)
    assert call(y, ws.data_ptr() + 256) == rws.ERR_INVALID_ARG
    assert call(inside, None) == rws.ERR_INVALID_ARG
    assert call(y, ws.data_ptr() + need) == rws.OK    # just behind it
    torch.cuda.synchronize()
    assert torch.equal(o, torch.zeros_like(o))
