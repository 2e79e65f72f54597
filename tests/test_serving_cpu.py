"""Refusals of the serving entry points: every check of arguments happens on
the host, before any device is looked for (fake addresses; nothing runs)."""
import numpy as np
import pytest

import row_wise_softmax_gb300 as rws
from tests import serving_ref as ref

torch = pytest.importorskip("torch")

from row_wise_softmax_gb300 import serving as sv  # noqa: E402

MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    rws.build()
    return sv._lib()


def heads(at=MB, row=1024, head=128):
    return sv._HEADS(at, row, head)


CACHE = dict(k=64 * MB, v=128 * MB, n_pages=10, page_size=16, n_kv_heads=2, head_dim=128,
             kp=4096, kr=256, kh=128, vp=4096, vr=256, vh=128, table=MB, n_seqs=3, width=4, step=4)


def cache(**kw):
    return sv._CACHE(*{**CACHE, **kw}.values())


# Without a device a call whose arguments are good answers UNSUPPORTED; with
# one these fake addresses are not to be launched on.
def good():
    return rws.ERR_UNSUPPORTED


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses")

BAD_CACHES = [
    dict(n_pages=-1), dict(page_size=0), dict(n_kv_heads=0), dict(n_seqs=-1), dict(width=-1),
    dict(step=3), dict(k=0), dict(v=0), dict(k=64 * MB + 8), dict(v=128 * MB + 2), dict(kp=-8),
    dict(kr=257), dict(vh=4), dict(vp=1 << 60), dict(table=0), dict(table=MB + 2),
    dict(page_size=1 << 20, width=1 << 20), dict(n_pages=1 << 31),
]


def decode(lib, c=None, q=None, o=None, lse=None, h=4, lengths=32 * MB, scale=1.0, dtype=rws.BF16,
           ws=None, size=0):
    return lib.softmax_attention_decode(
        cache() if c is None else c, heads() if q is None else q,
        heads(2 * MB) if o is None else o, lse, h, lengths, scale, dtype, ws, size, None)


@no_gpu
def test_decode_refusals(lib):
    bad = rws.ERR_INVALID_ARG
    assert decode(lib) == good()
    for kw in BAD_CACHES:
        assert decode(lib, cache(**kw)) == bad, kw
    assert decode(lib, cache(head_dim=96)) == rws.ERR_UNSUPPORTED
    assert decode(lib, dtype=rws.F32) == rws.ERR_UNSUPPORTED
    assert decode(lib, dtype=9) == bad
    for h in (0, -2, 3):
        assert decode(lib, h=h) == bad
    for s in (0.0, -1.0, float("nan"), 3e38):
        assert decode(lib, scale=s) == bad
    assert decode(lib, lengths=None) == bad and decode(lib, lengths=32 * MB + 1) == bad
    assert decode(lib, q=heads(MB + 8)) == bad and decode(lib, q=heads(0)) == bad
    assert decode(lib, q=heads(row=-8)) == bad and decode(lib, q=heads(head=100)) == bad
    assert decode(lib, o=heads(2 * MB, head=64)) == bad       # heads of out overlap
    assert decode(lib, o=heads(2 * MB, row=256)) == bad       # and rows
    assert decode(lib, o=heads(MB)) == good()                 # out is q
    assert decode(lib, o=heads(MB + 256)) == bad              # out over q
    assert decode(lib, o=heads(64 * MB)) == bad               # out over the cache
    assert decode(lib, lse=2 * MB + 64) == bad and decode(lib, lse=3) == bad
    assert decode(lib, cache(n_seqs=0)) == rws.OK
    # An empty table is fine (every length must then be 0).
    assert decode(lib, cache(width=0, step=0, table=0, n_pages=0, k=0, v=0)) == good()


@no_gpu
def test_decode_workspace_of_bad_sizes(lib):
    f = lib.softmax_attention_decode_workspace
    assert f(0, 8, 2, 128, 100) == 0
    for args in ((-1, 8, 2, 128, 100), (4, 8, 3, 128, 100), (4, 8, 2, 96, 100), (4, 0, 2, 128, 100),
                 (4, 8, 2, 128, -1), (4, 8, 2, 128, (1 << 30) + 1), (4, 8, 0, 128, 100)):
        assert f(*args) == -1
    assert f(4, 8, 2, 128, 100) == -1                         # no device


def packed(lib, q=None, k=None, v=None, o=None, lse=None, cu=32 * MB, ck=33 * MB, seqs=2, tq=100,
           tk=100, h=4, hk=2, d=128, scale=1.0, causal=1, dtype=rws.BF16):
    return lib.softmax_attention_packed(
        heads() if q is None else q, heads(4 * MB) if k is None else k,
        heads(5 * MB) if v is None else v, heads(2 * MB) if o is None else o, lse, cu, ck, seqs, tq,
        tk, h, hk, d, scale, causal, dtype, None, 0, None)


@no_gpu
def test_packed_refusals(lib):
    bad = rws.ERR_INVALID_ARG
    assert packed(lib) == good()
    for kw in (dict(seqs=-1), dict(tq=-1), dict(tk=-1), dict(h=0), dict(hk=0), dict(h=5),
               dict(scale=0.0), dict(scale=float("nan")), dict(causal=2), dict(dtype=7),
               dict(cu=None), dict(ck=None), dict(cu=32 * MB + 2), dict(tq=1 << 31),
               dict(q=heads(0)), dict(k=heads(4 * MB + 4)), dict(v=heads(5 * MB, head=-8)),
               dict(o=heads(2 * MB, row=128)), dict(o=heads(4 * MB)), dict(o=heads(5 * MB + 256)),
               dict(o=heads(MB + 512)), dict(lse=MB), dict(lse=5 * MB)):
        assert packed(lib, **kw) == bad, kw
    assert packed(lib, d=80) == rws.ERR_UNSUPPORTED
    assert packed(lib, dtype=rws.F32) == rws.ERR_UNSUPPORTED
    assert packed(lib, seqs=0) == rws.OK and packed(lib, tq=0) == rws.OK
    assert packed(lib, tk=0, k=heads(0), v=heads(0)) == good()
    # Parts of one projection's output, out in the place of q: fine.
    row = 8 * 128
    assert packed(lib, q=heads(MB, row), k=heads(MB + 1024, row), v=heads(MB + 1536, row),
                  o=heads(MB, row)) == good()
    assert packed(lib, q=heads(MB, row), k=heads(MB + 1024, row), v=heads(MB + 1536, row),
                  o=heads(MB + 1024, row)) == bad


@no_gpu
def test_packed_workspace_of_bad_sizes(lib):
    f = lib.softmax_attention_packed_workspace
    assert f(0, 10, 10, 8, 2, 128) == 0 and f(1, 0, 10, 8, 2, 128) == 0
    for args in ((-1, 10, 10, 8, 2, 128), (1, -1, 10, 8, 2, 128), (1, 10, -1, 8, 2, 128),
                 (1, 10, 10, 8, 3, 128), (1, 10, 10, 0, 2, 128), (1, 10, 10, 8, 0, 128),
                 (1, 10, 10, 8, 2, 96), (1, 1 << 31, 10, 8, 2, 128), (1, 10, 1 << 31, 8, 2, 64)):
        assert f(*args) == -1
    assert f(1, 10, 10000, 8, 2, 128) == -1                   # no device


@no_gpu
@pytest.mark.parametrize("key", ["tq", "tk"])
def test_packed_rows_that_a_tile_could_pass(lib, key):
    """A tile that begins at the last row ends past it, still below 2^31."""
    most = (1 << 31) - (1 << 16)
    far = dict(q=heads(1 << 50), o=heads(1 << 54), k=heads(1 << 56), v=heads(1 << 57))
    assert packed(lib, **far, **{key: most}) == good()
    assert packed(lib, **far, **{key: most + 1}) == rws.ERR_INVALID_ARG


def append(lib, c=None, k=None, v=None, q=None, o=None, h=4, pos=32 * MB, ids=33 * MB, n=5,
           freq=34 * MB, rot=128, inter=0, dtype=rws.F16):
    return lib.softmax_kv_append(
        cache() if c is None else c, heads(4 * MB) if k is None else k,
        heads(5 * MB) if v is None else v, q, o, h, pos, ids, n, freq, rot, inter, dtype, None)


@no_gpu
def test_append_refusals(lib):
    bad = rws.ERR_INVALID_ARG
    assert append(lib) == good()
    assert append(lib, q=heads(), o=heads(2 * MB)) == good()
    assert append(lib, q=heads(), o=heads()) == good()        # in place
    for kw in BAD_CACHES:
        assert append(lib, cache(**kw)) == bad, kw
    for kw in (dict(n=-1), dict(rot=8), dict(rot=144), dict(rot=-16), dict(inter=2), dict(pos=None),
               dict(pos=32 * MB + 3), dict(ids=33 * MB + 1), dict(freq=None), dict(freq=34 * MB + 4),
               dict(k=heads(0)), dict(v=heads(5 * MB + 2)), dict(dtype=5), dict(q=heads()),
               dict(o=heads()), dict(q=heads(), o=heads(2 * MB), h=0),
               dict(q=heads(), o=heads(2 * MB, head=120)), dict(q=heads(), o=heads(MB + 256)),
               dict(q=heads(), o=heads(4 * MB)), dict(q=heads(), o=heads(64 * MB)),
               dict(k=heads(64 * MB)), dict(v=heads(128 * MB))):
        assert append(lib, **kw) == bad, kw
    assert append(lib, cache(kr=128)) == bad                  # a page's rows overlap
    assert append(lib, cache(kh=64)) == bad                   # its heads do
    assert append(lib, rot=0, freq=None) == good()
    assert append(lib, n=0, pos=None) == rws.OK
    assert append(lib, cache(head_dim=32)) == rws.ERR_UNSUPPORTED
    assert append(lib, dtype=rws.F32) == rws.ERR_UNSUPPORTED


def test_status_string_of_a_bad_index(lib):
    assert "index" in rws.status_string(rws.ERR_DEVICE_INDEX)


def test_binding_refuses_host_tensors(lib):
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    c = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        rws.attention_decode(q, c, c, torch.zeros(2, 4, dtype=torch.int32), n)
    with pytest.raises(ValueError):
        rws.attention_packed(q, q, q, n)
    with pytest.raises(ValueError):
        rws.kv_append(c[0], c[0], c, c, torch.zeros(2, 4, dtype=torch.int32), n)


def test_the_plain_forms_agree_with_each_other():
    """The tests' own float64 forms: rotation against complex arithmetic, and a
    decoding step against the last row of a causal prompt."""
    r = np.random.default_rng(4)
    x, pos, inv = r.normal(size=(5, 2, 64)), r.integers(0, 99, 5), r.random(16)
    turn = np.exp(1j * pos[:, None, None] * inv)
    y = (x[..., :16] + 1j * x[..., 16:32]) * turn
    got = ref.rotate(x, pos, inv, False)
    assert np.allclose(got[..., :16], y.real) and np.allclose(got[..., 16:32], y.imag)
    assert np.array_equal(got[..., 32:], x[..., 32:])
    y = (x[..., 0:32:2] + 1j * x[..., 1:32:2]) * turn
    got = ref.rotate(x, pos, inv, True)
    assert np.allclose(got[..., 0:32:2], y.real) and np.allclose(got[..., 1:32:2], y.imag)
    q, k, v = r.normal(size=(9, 4, 64)), r.normal(size=(9, 2, 64)), r.normal(size=(9, 2, 64))
    o, lse, _ = ref.packed(q, k, v, [0, 9], [0, 9], 0.2, True)
    kc, vc = (np.zeros((3, 4, 2, 64)) for _ in range(2))
    table = np.array([[2, 0, 1]])
    for t in range(9):
        kc[table[0, t // 4], t % 4], vc[table[0, t // 4], t % 4] = k[t], v[t]
    o1, lse1, _ = ref.decode(q[8:], kc, vc, table, [9], 0.2)
    assert np.allclose(o1[0], o[8]) and np.allclose(lse1[0], lse[8])
