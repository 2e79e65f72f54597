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
]


@pytest.mark.parametrize("dtype", list(TYPES.values()), ids=list(TYPES))
@pytest.mark.parametrize("i", range(len(DECODE)))
def test_decode(i, dtype):
    decode_case(*DECODE[i], dtype, 100 + i)


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
