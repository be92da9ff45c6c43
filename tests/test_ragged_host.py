"""The calls of a ragged step without a GPU: arguments that the library and its binding refuse before
anything is enqueued (fake addresses are never touched)."""
import ctypes
import inspect

import pytest
import torch

FAKE = 0x100000


@pytest.fixture(scope="module")
def K():
    from persistent_kv_cache_gb300 import build
    build.build()
    from persistent_kv_cache_gb300 import kvc
    return kvc


def lengths(K, at=FAKE):
    return K.KvcLengths(at, at, at, at, at)


def caller(fn, **base):
    """fn(**changes) with named arguments in the order of `base`"""
    def call(**kw):
        assert set(kw) <= set(base), set(kw) - set(base)
        return fn(*{**base, **kw}.values())
    return call


def test_page_release(K):
    f = caller(K.library().kvc_page_release, released=FAKE, table=FAKE, max_pages=4, page=16, free=FAKE, pool=64, count=FAKE,
               left=FAKE + 64, batch=0, status=None, stream=None)
    assert f(max_pages=0) == 2 and f(page=0) == 2 and f(pool=0) == 2 and f(batch=-1) == 2
    assert f(batch=16385) == 5
    assert f(max_pages=1 << 20, page=2048) == 6 and f(pool=1 << 27) == 6 and f(pool=1 << 40) == 6
    assert f(free=None) == 1 and f(count=None) == 1 and f(left=None) == 1
    assert f(batch=1, released=None) == 1 and f(batch=1, table=None) == 1
    assert f(left=FAKE) == 2  # the same word as the count


def test_ragged_plan(K):
    f = caller(K.library().kvc_ragged_plan, cached=FAKE, new=FAKE, table=FAKE, max_pages=4, page=16, free=FAKE, pool=64, count=FAKE,
               left=FAKE + 64, batch=1, tokens=8, offsets=FAKE, len=lengths(K), positions=FAKE, slots=FAKE, status=None, stream=None)
    assert f(max_pages=0) == 2 and f(page=0) == 2 and f(pool=0) == 2 and f(batch=-1) == 2 and f(tokens=-1) == 2
    assert f(batch=16385) == 5
    assert f(max_pages=1 << 20, page=2048) == 6 and f(pool=1 << 27) == 6
    for name in ("cached", "new", "table", "free", "count", "left", "offsets", "positions", "slots"):
        assert f(**{name: None}) == 1, name
    assert f(len=lengths(K, None)) == 1
    assert f(positions=FAKE + 4) == 4 and f(slots=FAKE + 8) == 4
    assert f(left=FAKE) == 2


def test_rope_tables(K):
    f = caller(K.library().kvc_rope_tables, cos=FAKE, sin=FAKE * 8, first=0, positions=8, dim=64, base=1e4, scaling=0, factor=0.0,
               trained=0, low=0.0, high=0.0, magnitude=1.0, stream=None)
    inf, nan = float("inf"), float("nan")
    assert f(positions=-1) == 2 and f(first=-1) == 2 and f(first=(1 << 63) - 4) == 2 and f(dim=0) == 2 and f(dim=7) == 2
    assert f(dim=258) == 5 and f(scaling=-1) == 5 and f(scaling=4) == 5
    assert f(base=0.0) == 2 and f(base=-1.0) == 2 and f(base=nan) == 2 and f(base=inf) == 2 and f(magnitude=nan) == 2
    assert f(scaling=1) == 2 and f(scaling=1, factor=-2.0) == 2 and f(scaling=2, factor=inf) == 2 and f(scaling=2, factor=2.0, dim=2) == 2
    parts = dict(scaling=3, factor=4.0, trained=64, low=1.0, high=4.0)
    assert f(**{**parts, "trained": 0}) == 2 and f(**{**parts, "high": 1.0}) == 2 and f(**{**parts, "low": nan}) == 2
    assert f(cos=None) == 1 and f(sin=None) == 1 and f(cos=FAKE + 2) == 4 and f(sin=FAKE * 8 + 1) == 4
    assert f(sin=FAKE + 512) == 2  # overlapping tables
    assert f(positions=0, cos=None, sin=None) == 0
    assert f(base=1e-300, dim=256, scaling=1, factor=1e-300) == 2  # a speed that is no number


def test_ragged_append(K):
    f = caller(K.library().kvc_ragged_append, q_out=FAKE, k_pool=1 << 30, v_pool=1 << 31, q=1 << 32, k=(1 << 32) + 1024,
               v=(1 << 32) + 1536, qs=1024, ks=1024, vs=1024, qw=None, kw=None, eps=1e-6, positions=FAKE, slots=FAKE, tokens=4,
               q_heads=4, kv_heads=2, pool=8, page=16, dim=128, dtype=1, turned=128, inter=0, cos=FAKE, sin=FAKE, rmax=64,
               status=None, stream=None)
    assert f(dtype=7) == 3 and f(dtype=0) == 5
    assert f(tokens=-1) == 2 and f(q_heads=0) == 2 and f(kv_heads=0) == 2 and f(pool=0) == 2 and f(page=0) == 2 and f(dim=0) == 2
    assert f(dim=72) == 5 and f(dim=272) == 5 and f(q_heads=40000) == 5
    assert f(pool=1 << 28) == 6
    assert f(sin=None) == 1 and f(cos=None) == 1
    assert f(rmax=0) == 2 and f(turned=0) == 2 and f(turned=144) == 2 and f(turned=24) == 5
    assert f(qw=FAKE, eps=-1.0) == 2 and f(kw=FAKE, eps=float("nan")) == 2
    assert f(qs=256) == 2 and f(ks=128) == 2 and f(vs=128) == 2
    for name in ("q_out", "k_pool", "v_pool", "q", "k", "v", "positions", "slots"):
        assert f(**{name: None}) == 1, name
    for name in ("q_out", "k_pool", "v_pool", "q", "k", "v"):
        assert f(**{name: (1 << 33) + 8}) == 4, name
    for name in ("qw", "kw", "cos", "sin"):
        assert f(**{name: FAKE + 4}) == 4, name
    assert f(qs=1028) == 4 and f(ks=1026) == 4 and f(vs=1025) == 4
    # what is written over what is read or written
    assert f(v_pool=(1 << 30) + 64) == 2 and f(q_out=1 << 30) == 2 and f(q_out=1 << 32) == 2 and f(k_pool=1 << 32) == 2
    assert f(v_pool=(1 << 32) - 16) == 2 and f(q_out=(1 << 32) + 2048) == 2
    assert f(tokens=0, q_out=None) == 0


def test_gqa_ragged(K):
    lib = K.library()
    f = caller(lib.kvc_gqa_ragged, out=FAKE, q=1 << 24, k=1 << 30, v=1 << 31, offsets=FAKE, table=FAKE, max_pages=4, pool=8, page=16,
               len=lengths(K), batch=2, tokens=4, q_heads=4, kv_heads=2, dim=128, dtype=1, window=0, scale=0.0, ws=FAKE, bytes=1 << 40,
               status=None, stream=None)
    assert f(dtype=9) == 3 and f(dtype=0) == 5
    assert f(batch=-1) == 2 and f(tokens=-1) == 2 and f(q_heads=0) == 2 and f(kv_heads=0) == 2 and f(q_heads=5) == 2
    assert f(max_pages=0) == 2 and f(pool=0) == 2 and f(page=0) == 2 and f(page=24) == 2 and f(page=8) == 2
    assert f(dim=96) == 5 and f(q_heads=34) == 5 and f(batch=65536) == 5
    assert f(max_pages=1 << 28) == 6 and f(pool=1 << 27) == 6 and f(pool=1 << 26, kv_heads=4) == 6 and f(tokens=1 << 30) == 6
    for name in ("out", "q", "k", "v", "offsets", "table"):
        assert f(**{name: None}) == 1, name
    assert f(len=lengths(K, None)) == 1
    for name in ("out", "q", "k", "v"):
        assert f(**{name: (1 << 33) + 8}) == 4, name
    assert f(out=1 << 24) == 2 and f(out=(1 << 24) + 64) == 2 and f(out=1 << 30) == 2 and f(out=1 << 31) == 2
    assert f(ws=None) == 8 and f(bytes=0) == 8 and f(ws=FAKE + 16) == 4
    assert f(batch=0, out=None) == 0 and f(tokens=0, out=None) == 0
    size = lib.kvc_gqa_ragged_workspace_size
    assert size(0, 1, 4, 2, 64) == 0 and size(1, 0, 4, 2, 64) == 0 and size(1, 1, 5, 2, 64) == 0 and size(1, 1, 4, 2, 0) == 0
    assert size(1, 1, 4, 2, 64) > 0


def test_binding_refuses_other_shapes(K, monkeypatch):
    """The library gets sizes from one tensor of each kind: the binding compares the others.  (Tensors of
    the meta device stand in for the GPU's.)"""
    monkeypatch.setattr(K, "_get_device", lambda: -1)
    monkeypatch.setattr(K, "_addresses", lambda *a: (_ for _ in ()).throw(AssertionError("got as far as the addresses")))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    f32 = lambda *s: torch.zeros(s)  # noqa: E731
    table, free, one = i32(3, 4), i32(64), i32(1)
    for kw in (dict(released=i32(2)), dict(released=i32(3).long()), dict(block_table=i32(3, 4).long()), dict(free_count=i32(2)),
               dict(free_left=one.long()), dict(free_pages=free.long())):
        args = {**dict(released=i32(3), block_table=table, page_size=16, free_pages=free, free_count=one, free_left=i32(1)), **kw}
        with pytest.raises(ValueError, match="expected"):
            K.kvc_page_release(**args)
    plan = K.RaggedPlan(3, 8, "cpu")
    for kw in (dict(cached=i32(2)), dict(new_tokens=i32(4)), dict(new_tokens=i32(3).long()), dict(block_table=i32(3, 4).short()),
               dict(plan=K.RaggedPlan(2, 8, "cpu"))):
        args = {**dict(cached=i32(3), new_tokens=i32(3), block_table=table, page_size=16, free_pages=free, free_count=one,
                       free_left=i32(1), plan=plan), **kw}
        with pytest.raises(ValueError, match="expected"):
            K.kvc_ragged_plan(**args)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    good = dict(out=bf(5, 4, 64), q=bf(5, 4, 64), k_pool=bf(8, 2, 16, 64), v_pool=bf(8, 2, 16, 64), block_table=table,
                offsets=i32(4), lengths=K.Lengths(3, "cpu"), workspace=i32(64))
    for kw in (dict(out=bf(4, 4, 64)), dict(q=bf(5, 4, 64).half()), dict(q=bf(5, 4, 32)), dict(v_pool=bf(8, 2, 32, 64)),
               dict(offsets=i32(3)), dict(offsets=i32(4).long()), dict(block_table=table.long()), dict(out=bf(5, 4, 64).float())):
        with pytest.raises(ValueError, match="expected"):
            K.kvc_gqa_ragged(**{**good, **kw})
    for a, b in ((f32(4, 8), f32(5, 8)), (f32(4, 8).double(), f32(4, 8)), (f32(4, 8), f32(4, 8).half())):
        with pytest.raises(ValueError, match="expected"):
            K.kvc_rope_tables(a, b)


def test_append_binding_refuses(K):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        K.kvc_ragged_append(bf(4, 4, 64), bf(8, 2, 16, 64), bf(8, 2, 16, 64), bf(4, 4, 64), bf(4, 2, 64), bf(4, 2, 64),
                            torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    x = bf(4, 8, 64)
    assert "stride" in inspect.getsource(K._token_rows)
    with pytest.raises(ValueError):
        K._token_rows("q", x[:, ::2], (4, 4, 64), torch.bfloat16)   # heads that are not dense
    with pytest.raises(ValueError):
        K._token_rows("q", x, (4, 4, 64), torch.bfloat16)           # another number of heads
    with pytest.raises(ValueError):
        K._token_rows("q", x, (4, 8, 64), torch.float16)


def test_struct_of_lengths_is_five_addresses(K):
    assert ctypes.sizeof(K.KvcLengths) == 5 * ctypes.sizeof(ctypes.c_void_p)


def test_release_and_plan_write_apart_from_what_they_read(K):
    A = [i << 20 for i in range(1, 20)]
    f = caller(K.library().kvc_page_release, released=A[0], table=A[1], max_pages=4, page=16, free=A[2], pool=64, count=A[3],
               left=A[4], batch=8, status=None, stream=None)
    for kw in (dict(released=A[2] + 252), dict(table=A[2] - 124), dict(count=A[2]), dict(left=A[2] + 128), dict(left=A[0] + 28),
               dict(left=A[1])):
        assert f(**kw) == 2, kw
    L = lambda at: K.KvcLengths(*at)  # noqa: E731
    lens = A[10:15]
    f = caller(K.library().kvc_ragged_plan, cached=A[0], new=A[1], table=A[2], max_pages=4, page=16, free=A[3], pool=64, count=A[4],
               left=A[5], batch=8, tokens=100, offsets=A[6], len=L(lens), positions=A[7], slots=A[8], status=None, stream=None)
    for i, at in enumerate(lens):
        # the lengths of the step before as what is cached now
        assert f(cached=at) == 2 and f(new=at + 28) == 2, i
        for over in (A[2] + 124, A[3] + 252, A[4], A[5], A[6] + 32, A[7] + 384, A[8]):
            assert f(len=L(lens[:i] + [over] + lens[i + 1:])) == 2, (i, over)
    for kw in (dict(cached=A[6]), dict(new=A[7]), dict(cached=A[8] + 396), dict(table=A[3]), dict(table=A[0] - 124), dict(offsets=A[7]),
               dict(left=A[0]), dict(left=A[6] + 32), dict(slots=A[7] + 384), dict(free=A[2])):
        assert f(**kw) == 2, kw
    assert f(tokens=(1 << 31) - 1023) == 6


def test_append_writes_apart_from_lists_tables_and_weights(K):
    G = 1 << 30
    f = caller(K.library().kvc_ragged_append, q_out=G, k_pool=2 * G, v_pool=3 * G, q=4 * G, k=5 * G, v=6 * G, qs=512, ks=256, vs=256,
               qw=7 * G, kw=7 * G + 256, eps=1e-6, positions=8 * G, slots=8 * G + 16, tokens=4, q_heads=4, kv_heads=2, pool=8, page=16,
               dim=128, dtype=1, turned=64, inter=0, cos=9 * G, sin=10 * G, rmax=64, status=None, stream=None)
    for at, size in ((G, 4 * 4 * 128 * 2), (2 * G, 8 * 16 * 2 * 128 * 2), (3 * G, 8 * 16 * 2 * 128 * 2)):
        for name, own in (("qw", 256), ("kw", 256), ("positions", 16), ("slots", 16), ("cos", 64 * 32 * 4), ("sin", 64 * 32 * 4)):
            assert f(**{name: at + size - 16}) == 2 and f(**{name: at - own + 16}) == 2, (name, at)
    assert f(cos=1 << 40, rmax=1 << 62, sin=G // 2) == 2  # (tables past 2^31 positions)
    assert f(tokens=(1 << 31) - 1023) == 6


def test_attention_writes_apart_from_what_it_reads(K):
    G = 1 << 30
    size = K.library().kvc_gqa_ragged_workspace_size(2, 4, 4, 2, 128)
    assert size < G
    f = caller(K.library().kvc_gqa_ragged, out=G, q=2 * G, k=3 * G, v=4 * G, offsets=5 * G, table=6 * G, max_pages=4, pool=8, page=16,
               len=K.KvcLengths(7 * G, 8 * G, 9 * G, 10 * G, 11 * G), batch=2, tokens=4, q_heads=4, kv_heads=2, dim=128, dtype=1,
               window=0, scale=0.0, ws=12 * G, bytes=size, status=None, stream=None)
    for at, span in ((G, 4 * 4 * 128 * 2), (12 * G, size)):
        last = at + span - 4
        assert f(offsets=last) == 2 and f(offsets=at - 8) == 2 and f(table=last) == 2 and f(table=at - 28) == 2
        for i in (0, 1, 3):  # those that are read
            lens = [7 * G, 8 * G, 9 * G, 10 * G, 11 * G]
            lens[i] = last
            assert f(len=K.KvcLengths(*lens)) == 2, i
    for name in ("out", "q", "k", "v"):
        assert f(**{name: 12 * G}) == 2, name
    assert f(out=12 * G + (size - 16) // 16 * 16) == 2


def test_magnitude_beyond_float32(K):
    f = caller(K.library().kvc_rope_tables, cos=FAKE, sin=FAKE * 8, first=0, positions=8, dim=64, base=1e4, scaling=0, factor=0.0,
               trained=0, low=0.0, high=0.0, magnitude=1e39, stream=None)
    assert f() == 2
