"""Entry points of the serving operators: what they refuse before anything is enqueued, and
their sizes (no GPU needed)."""
import ctypes

import pytest
import torch

from clustered_softmax_attention_b200 import muse as m

FAKE = 1 << 20  # aligned, never dereferenced: validation fails first
ST = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    return m.load_library()


def _d(B=2, H=4, N=8, D=64, Dv=64, dtype=m.MUSE_BF16, scale=1.0):
    return m.MuseDims(B, H, N, D, Dv, dtype, scale)


def _r(p=FAKE, sb=4096, sh=1024, sn=128):
    return m.MuseRows(p, sb, sh, sn)


def _c(tiles=FAKE, table=FAKE, pages=8, Hkv=4, page=64, max_pages=4):
    return m.MuseCache(tiles, table, pages, Hkv, page, max_pages)


def _rope(sections=(8, 12, 12), base=1e4, flags=0, axes=None):
    return m.MuseRope(len(sections) if axes is None else axes,
                      (ctypes.c_int * 4)(*list(sections)[:4]), base, flags)


BAD_ROWS = [_r(p=None), _r(p=FAKE + 4), _r(sb=4097), _r(sh=4), _r(sn=-128)]


def test_new_entry_points_are_declared_and_exported(lib):
    names = m.declared_entry_points()
    for n in ("muse_rope_axes", "muse_cache_tile_bytes", "muse_cache_write", "muse_cache_read",
              "muse_cache_attend"):
        assert n in names and hasattr(lib, n)


def test_sizes(lib):
    assert [m.muse_cache_tile_bytes(a, b) for a, b in ((64, 64), (64, 128), (128, 64), (128, 128))] \
        == [2304, 3456, 3456, 4608]
    assert m.muse_cache_tile_bytes(96, 64) == 0
    assert m.muse_cache_shape(10, 4, 128, 64, 64) == (10, 4, 4, 2304)
    with pytest.raises(m.MuseError):
        m.muse_cache_shape(10, 4, 48, 64, 64)
    ws = lambda d, Hkv: m.muse_workspace_size("muse_cache_attend", d, Hkv)
    assert ws(_d(N=1), 4) > 0 and ws(_d(N=128, H=8), 2) > 0
    assert ws(_d(N=129), 4) == 0 and ws(_d(N=1), 3) == 0 and ws(_d(N=1), 0) == 0
    assert ws(_d(N=1, D=96), 4) == 0


def test_rope_refusals(lib):
    f = lambda Q=_r(), K=m.MuseRows(), Hk=0, d=_d(), pos=FAKE, nb=2, r=_rope(), Qo=_r(), Ko=m.MuseRows(): \
        lib.muse_rope_axes(Q, K, Hk, d, pos, nb, r, Qo, Ko, ST)
    assert f(d=_d(dtype=5)) == 3
    assert f(d=_d(D=96)) == 2 and f(d=_d(N=0)) == 2 and f(d=_d(B=70000, H=1)) == 2
    for bad in BAD_ROWS:
        assert f(Q=bad) == 1 and f(Qo=bad) == 1
        assert f(K=_r(), Hk=2, Ko=bad) == 1
    assert f(K=_r(sn=4), Hk=2, Ko=_r()) == 1
    assert f(K=_r(), Hk=0, Ko=_r()) == 2
    assert f(pos=None) == 1 and f(nb=3) == 2
    for bad in (_rope((33,)), _rope((16, 17)), _rope((0, 4)), _rope((4,), axes=0), _rope((4,), axes=5),
                _rope((-1, 4)), _rope(flags=8), _rope(base=0.5), _rope(base=float("nan")),
                _rope(base=float("inf")), _rope((2 ** 31 - 1, 2 ** 31 - 1))):
        assert f(r=bad) == 1


def test_cache_refusals(lib):
    def write(K=_r(), V=_r(), d=_d(), c=_c(), start=FAKE):
        a = lib.muse_cache_write(K, V, d, c, start, None, ST)
        assert a == lib.muse_cache_read(d, c, start, None, K, V, ST)
        return a
    assert write(d=_d(dtype=2)) == 3
    assert write(d=_d(Dv=32)) == 2 and write(d=_d(H=2)) == 2
    for bad in BAD_ROWS:
        assert write(K=bad) == 1 and write(V=bad) == 1
    assert write(start=None) == 1
    assert write(c=_c(tiles=None)) == 1 and write(c=_c(tiles=FAKE + 8)) == 1
    assert write(c=_c(table=None)) == 1
    for bad in (_c(page=16), _c(page=96), _c(page=2048), _c(page=0), _c(pages=0), _c(max_pages=0),
                _c(max_pages=2 ** 25), _c(pages=2 ** 30), _c(pages=2 ** 28, page=64)):
        assert write(c=bad) == 2


def test_attend_refusals(lib):
    big = 1 << 40
    f = lambda Q=_r(), d=_d(), c=_c(), lens=FAKE, O=_r(), lse=FAKE, ws=FAKE, n=big: \
        lib.muse_cache_attend(Q, d, c, lens, None, O, lse, ws, n, ST)
    assert f(d=_d(dtype=9)) == 3
    assert f(d=_d(N=129)) == 2 and f(d=_d(N=0)) == 2 and f(d=_d(H=6)) == 2 and f(c=_c(Hkv=3)) == 2
    assert f(c=_c(Hkv=0)) == 2 and f(d=_d(H=2)) == 2
    assert f(d=_d(scale=float("inf"))) == 1
    for bad in BAD_ROWS:
        assert f(Q=bad) == 1 and f(O=bad) == 1
    assert f(lens=None) == 1 and f(c=_c(table=None)) == 1
    assert f(ws=None) == 4 and f(n=0) == 4 and f(ws=FAKE + 8) == 4
    need = m.muse_workspace_size("muse_cache_attend", _d(), 4)
    assert f(n=need - 1) == 4


def test_binding_refuses_what_the_library_cannot_see():
    x = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)
    pos = torch.zeros(2, 1, 8, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        m.muse_rope_axes(x, pos, [32])
    with pytest.raises(ValueError, match="positions"):
        m.muse_rope_axes(x, pos.long(), [32])
    with pytest.raises(ValueError, match="positions"):
        m.muse_rope_axes(x, pos, [16, 16])
    with pytest.raises(ValueError, match="axes"):
        m.muse_rope_axes(x, pos, [1] * 5)
    with pytest.raises(ValueError, match="out: shape"):
        m.muse_rope_axes(x, pos, [32], out=x[:, :2])
    with pytest.raises(ValueError, match="K: shape|K: torch"):
        m.muse_rope_axes(x, pos, [32], K=x[:1])
    with pytest.raises(ValueError, match="Q: expected"):
        m.muse_rope_axes(x.half(), pos, [32])
    cache = torch.zeros(m.muse_cache_shape(4, 4, 64, 64, 64), dtype=torch.uint8)
    table = torch.zeros(2, 2, dtype=torch.int32)
    start = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="V: shape"):
        m.muse_cache_write(cache, x, x[..., :32], table, start)
    with pytest.raises(ValueError, match="K: shape"):
        m.muse_cache_write(cache, x[:, :2], x[:, :2], table, start)
    with pytest.raises(ValueError, match="do not hold"):
        m.muse_cache_write(cache[..., :2300].contiguous(), x, x, table, start)
    with pytest.raises(ValueError, match="page_table"):
        m.muse_cache_write(cache, x, x, table[:1], start)
    with pytest.raises(ValueError, match="cache: expected"):
        m.muse_cache_attend(x, cache.int(), table, start)
    with pytest.raises(ValueError, match="lse"):
        m.muse_cache_attend(x, cache, table, start, lse=torch.zeros(2, 4, 9))
    with pytest.raises(ValueError, match="K: shape"):
        m.muse_cache_read(cache, table, start, 8, 64, out=(x[:, :2], x))


def test_binding_refuses_overlapping_and_ragged_rows():
    """Geometry is refused before the device is looked at."""
    table, start = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cache = torch.zeros(m.muse_cache_shape(4, 4, 64, 64, 64), dtype=torch.uint8)
    buf = torch.zeros(1 << 16, dtype=torch.bfloat16)
    view = lambda stride, at=0, shape=(2, 4, 8, 64): torch.as_strided(buf, shape, stride, at)
    read = lambda k, v: m.muse_cache_read(cache, table, start, 8, 64, out=(k, v))
    good = view((2048, 512, 64, 1))
    for stride in ((2048, 512, 64, 2), (2048, 512, 68, 1)):
        with pytest.raises(ValueError, match="16-byte"):
            m.muse_cache_write(cache, view(stride), good, table, start)
    with pytest.raises(ValueError, match="16-byte"):
        m.muse_cache_write(cache, view((2048, 512, 64, 1), 1), good, table, start)
    # rows that are read may repeat, or lie as [B,N,H,D]; they get as far as the device
    for stride in ((0, 0, 64, 1), (2048, 64, 256, 1)):
        with pytest.raises(ValueError, match="CUDA"):
            m.muse_cache_write(cache, view(stride), good, table, start)
    one = view((7, 64, 3, 1), shape=(1, 4, 1, 64))       # sizes of one have no stride
    with pytest.raises(ValueError, match="CUDA"):
        m.muse_cache_write(cache, one, one, table[:1], start[:1])
    with pytest.raises(ValueError, match="CUDA"):
        read(good, good)


def test_binding_takes_nothing_but_what_it_names():
    x = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)
    pos = torch.zeros(1, 8, dtype=torch.int32)
    for bad in (None, 3, "x"):
        with pytest.raises(ValueError, match="Q: expected a tensor"):
            m.muse_rope_axes(bad, pos, [32])
    with pytest.raises(ValueError, match="sections"):
        m.muse_rope_axes(x, pos, [32.5])
    with pytest.raises(TypeError, match="sections"):
        m.muse_rope_axes(x, pos, 32)
    with pytest.raises(ValueError, match="base"):
        m.muse_rope_axes(x, pos, [32], base="a")
    with pytest.raises(ValueError, match="sections"):
        m.muse_rope_axes(x, pos, [2 ** 40])
    with pytest.raises(ValueError, match="dtype"):
        m.muse_cache_read(x, pos, pos, 8, 64, dtype=torch.float16)
    with pytest.raises(TypeError, match="arguments"):
        m._serving().rope_axes(x)


@pytest.mark.gpu
def test_binding_refuses_overlapping_rows_on_the_gpu():
    pos = torch.zeros(1, 8, dtype=torch.int32, device="cuda")
    buf = torch.zeros(1 << 16, dtype=torch.bfloat16, device="cuda")
    x = buf[:4096].view(2, 4, 8, 64)
    for stride in ((0, 512, 64, 1), (2048, 512, 32, 1), (1024, 512, 64, 1)):
        with pytest.raises(ValueError, match="overlapping"):
            m.muse_rope_axes(x, pos, [32], out=torch.as_strided(buf, (2, 4, 8, 64), stride, 8192))
    with pytest.raises(ValueError, match="in place"):
        m.muse_rope_axes(x, pos, [32], out=torch.as_strided(buf, (2, 4, 8, 64), (2048, 64, 256, 1)))
    with pytest.raises(ValueError, match="positions"):
        m.muse_rope_axes(x, pos.cpu(), [32])
    with pytest.raises(m.MuseError, match="INVALID_ARG"):
        m.muse_rope_axes(x, pos, [33])
    with pytest.raises(m.MuseError, match="SHAPE"):
        m.muse_rope_axes(x[..., :32].contiguous(), pos, [8])


@pytest.mark.parametrize("flags", [2 ** 32, 2 ** 32 + 1, -1, -2 ** 40])
def test_binding_does_not_cut_flags_short(flags):
    """2^32 is no flag, nor is it none."""
    x = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="flags"):
        m.muse_rope_axes(x, torch.zeros(1, 8, dtype=torch.int32), [32], flags=flags)


def test_the_hook_of_the_many_row_form_is_a_bit_of_its_own(lib):
    """Its value, and that bits beside it are refused before the device is touched."""
    assert m.MUSE_TEST_WITHHOLD_CACHE == 4 and m.MUSE_TEST_WITHHOLD_VALUES == 1
    for bits in (2, 6, 8, 4 | 8, 1 << 31):
        assert lib.muse_set_test_hooks(bits, 0) == 1


@pytest.mark.parametrize("pages,Hkv,page", [(10, 4, 96), (10, 4, 0), (10, 4, 16), (10, 4, 2048), (10, 4, -32),
                                            (0, 4, 64), (10, 0, 64), (-1, 4, 64)])
def test_no_shape_for_a_cache_that_every_call_refuses(lib, pages, Hkv, page):
    with pytest.raises(m.MuseError, match="SHAPE"):
        m.muse_cache_shape(pages, Hkv, page, 64, 64)
    c = _c(pages=pages, Hkv=Hkv, page=page)
    assert lib.muse_cache_write(_r(), _r(), _d(H=max(Hkv, 1)), c, FAKE, None, ST) == 2
    for good in (32, 64, 1024):
        assert m.muse_cache_shape(10, 4, good, 64, 64) == (10, 4, good // 32, 2304)


def test_the_binding_is_built_again_for_another_torch_or_interpreter(tmp_path, monkeypatch):
    from clustered_softmax_attention_b200 import build as b

    stamp = tmp_path / "binding.stamp"
    so = tmp_path / "_serving.so"
    so.write_bytes(b"")          # newer than its sources
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(b, "BINDING", str(so))
    assert b._binding_stale()    # nobody knows for what it was built
    stamp.write_text(b._binding_made_for())
    assert not b._binding_stale()
    for where, name, other in ((torch, "__version__", "0.0"), (b.sys, "version", "3.0")):
        with monkeypatch.context() as c:
            c.setattr(where, name, other)
            assert b._binding_stale()
    assert not b._binding_stale()
    so.unlink()
    assert b._binding_stale()
