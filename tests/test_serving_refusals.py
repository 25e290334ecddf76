"""What the operators on the device pages refuse: every case before anything is
enqueued, so this runs without a GPU.  Addresses are made up; nothing is read."""
import ctypes

import pytest

import tiered_kv_cache_gb300 as hc

A = 1 << 20      # an aligned address


@pytest.fixture(scope="module", autouse=True)
def built():
    from tiered_kv_cache_gb300 import build
    build.build()


def desc(**kw):
    d = dict(num_layers=2, num_buffers=2, page_size=16, elem_bytes=2, row_elems=256, host_num_pages=1, layout=0,
             launch_ctas=0, flags=0, reserved=0)
    d.update(kw)
    return hc.PoolDesc(*d.values())


def call(fn, packer, fields, d, layer=0, kv=None, pages=10):
    kv = kv or hc.DeviceKV([A] * (d.num_buffers * d.num_layers), pages)
    before = hc.launch_count()
    rc = getattr(hc.library(), fn)(kv.ref, ctypes.byref(d), layer, packer.pack(*fields.values()), None)
    assert hc.launch_count() == before
    return hc.STATUS[rc]


APPEND = dict(q=A, q_out=A, k=A, v=A, qw=A, kw=A, slots=A, positions=A, cos_sin=A, qst=512, qsh=128, ost=512, osh=128,
              kst=256, ksh=128, vst=256, vsh=128, n=3, rows=100, dtype=0, hq=4, hk=2, d=128, qn=128, kn=128, rot=128,
              off=0, il=0, eps=1e-6, ks=1.0, vs=1.0)
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("change,status", [
    (dict(q=0), "INVALID_ARG"), (dict(q_out=0), "INVALID_ARG"), (dict(k=0), "INVALID_ARG"), (dict(v=0), "INVALID_ARG"),
    (dict(slots=0), "INVALID_ARG"), (dict(positions=0), "INVALID_ARG"), (dict(cos_sin=0), "INVALID_ARG"),
    (dict(qw=0), "INVALID_ARG"), (dict(kw=0), "INVALID_ARG"), (dict(qw=A + 2), "ALIGNMENT"),
    (dict(q=A + 8), "ALIGNMENT"), (dict(q_out=A + 2), "ALIGNMENT"), (dict(k=A + 4), "ALIGNMENT"),
    (dict(v=A + 8), "ALIGNMENT"), (dict(qst=516), "ALIGNMENT"), (dict(ksh=132), "ALIGNMENT"),
    (dict(slots=A + 4), "ALIGNMENT"), (dict(positions=A + 4), "ALIGNMENT"), (dict(cos_sin=A + 2), "ALIGNMENT"),
    (dict(qst=-512), "INVALID_ARG"), (dict(vst=1 << 40), "INVALID_ARG"),
    (dict(ost=0), "INVALID_ARG"), (dict(osh=0), "INVALID_ARG"), (dict(osh=64), "INVALID_ARG"),
    (dict(ost=256), "INVALID_ARG"), (dict(ost=1024), "INVALID_ARG"),
    (dict(ost=128, osh=256, q_out=2 * A), "INVALID_ARG"),
    (dict(n=-1), "INVALID_ARG"), (dict(n=1 << 29), "INVALID_ARG"), (dict(n=1 << 62), "INVALID_ARG"),
    (dict(rows=0), "INVALID_ARG"), (dict(rows=1 << 40), "INVALID_ARG"),
    (dict(dtype=2), "INVALID_ARG"), (dict(hq=0, hk=0), "INVALID_ARG"), (dict(hq=-1), "INVALID_ARG"),
    (dict(hk=-1), "INVALID_ARG"), (dict(hk=3), "INVALID_ARG"), (dict(d=120), "INVALID_ARG"), (dict(d=4), "INVALID_ARG"),
    (dict(d=0), "INVALID_ARG"), (dict(d=776), "INVALID_ARG"), (dict(hk=64, d=4), "INVALID_ARG"),
    (dict(qn=136), "INVALID_ARG"), (dict(qn=4), "INVALID_ARG"), (dict(kn=-8), "INVALID_ARG"),
    (dict(rot=63), "INVALID_ARG"), (dict(rot=-2), "INVALID_ARG"), (dict(off=2), "INVALID_ARG"),
    (dict(rot=64, off=63), "INVALID_ARG"), (dict(rot=64, off=-2), "INVALID_ARG"), (dict(rot=64, off=66), "INVALID_ARG"),
    (dict(rot=2, off=2 ** 31 - 2), "INVALID_ARG"),
    (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=NAN), "INVALID_ARG"), (dict(ks=0.0), "INVALID_ARG"),
    (dict(vs=-1.0), "INVALID_ARG"), (dict(ks=INF), "INVALID_ARG"), (dict(ks=2.0), "INVALID_ARG"),
])
def test_append_refuses(change, status):
    assert call("hicache_append_kv", hc._APPEND_DESC, {**APPEND, **change}, desc()) == status


def test_append_accepts_nothing_to_do():
    assert call("hicache_append_kv", hc._APPEND_DESC, {**APPEND, "n": 0, "q": 0, "slots": 0}, desc()) == "OK"


DECODE = dict(q=A, out=A, table=A, lens=A, lse=A, weights=A, ws=A, ws_bytes=1 << 30, qb=512, qh=128, ob=512, oh=128,
              tb=20, lb=4, wb=20, dtype=0, batch=3, hq=4, d=128, dv=128, width=20, window=0, reserved=0, scale=0.1,
              ks=1.0, vs=1.0, decay=1.0)


@pytest.mark.parametrize("change,status", [
    (dict(q=0), "INVALID_ARG"), (dict(out=0), "INVALID_ARG"), (dict(table=0), "INVALID_ARG"),
    (dict(lens=0), "INVALID_ARG"), (dict(ws=0), "INVALID_ARG"), (dict(ws=A + 128), "ALIGNMENT"),
    (dict(ws_bytes=0), "INVALID_ARG"), (dict(ws_bytes=255), "INVALID_ARG"), (dict(ws_bytes=-1), "INVALID_ARG"),
    (dict(q=A + 8), "ALIGNMENT"), (dict(out=A + 8), "ALIGNMENT"), (dict(qb=510), "ALIGNMENT"), (dict(oh=132), "ALIGNMENT"),
    (dict(table=A + 2), "ALIGNMENT"), (dict(lens=A + 1), "ALIGNMENT"), (dict(lse=A + 2), "ALIGNMENT"),
    (dict(weights=A + 2), "ALIGNMENT"),
    (dict(qb=-8), "INVALID_ARG"), (dict(ob=0), "INVALID_ARG"), (dict(oh=120), "INVALID_ARG"),
    (dict(tb=-1), "INVALID_ARG"), (dict(lb=3), "INVALID_ARG"), (dict(wb=19), "INVALID_ARG"),
    (dict(dtype=-1), "INVALID_ARG"), (dict(batch=-1), "INVALID_ARG"), (dict(batch=65536), "INVALID_ARG"),
    (dict(hq=0), "INVALID_ARG"), (dict(hq=5), "INVALID_ARG"), (dict(hq=4098), "INVALID_ARG"),
    (dict(d=0), "INVALID_ARG"), (dict(d=96, dv=96), "INVALID_ARG"), (dict(d=4, dv=4), "INVALID_ARG"),
    (dict(dv=64), "INVALID_ARG"), (dict(width=0), "INVALID_ARG"), (dict(width=1 << 27), "INVALID_ARG"),
    (dict(window=-1), "INVALID_ARG"), (dict(reserved=1), "INVALID_ARG"), (dict(scale=NAN), "INVALID_ARG"),
    (dict(scale=INF), "INVALID_ARG"), (dict(decay=NAN), "INVALID_ARG"), (dict(ks=0.5), "INVALID_ARG"),
    (dict(vs=0.0), "INVALID_ARG"),
])
def test_decode_refuses(change, status):
    assert call("hicache_decode_attention", hc._DECODE_DESC, {**DECODE, **change}, desc()) == status


@pytest.mark.parametrize("d,change,layer,status", [
    (desc(num_buffers=3), {}, 0, "INVALID_ARG"), (desc(elem_bytes=4), {}, 0, "INVALID_ARG"),
    (desc(), {}, 2, "INVALID_ARG"), (desc(), {}, -1, "INVALID_ARG"), (desc(page_size=0), {}, 0, "INVALID_ARG"),
    (desc(row_elems=260), {}, 0, "ALIGNMENT"),
    (desc(elem_bytes=1, row_elems=240), dict(d=120, dv=120), 0, "INVALID_ARG"),
    (desc(row_elems=1024), dict(d=512, dv=512, hq=2), 0, "INVALID_ARG"),
    (desc(num_buffers=1, row_elems=576), dict(d=576, dv=576), 0, "INVALID_ARG"),
    (desc(num_buffers=1, row_elems=512), dict(d=512, dv=512), 0, "INVALID_ARG"),
    (desc(num_buffers=1, row_elems=576, elem_bytes=1), dict(d=576, dv=512), 0, "INVALID_ARG"),
])
def test_decode_refuses_pools(d, change, layer, status):
    assert call("hicache_decode_attention", hc._DECODE_DESC, {**DECODE, **change}, d, layer) == status


def test_decode_refuses_scales_that_overflow_together():
    """Each in range of 32 bits, their product (times log2 e) is not."""
    d = desc(elem_bytes=1)
    for scale, ks, status in ((1e38, 1e38, "INVALID_ARG"), (-3e38, 1.0, "INVALID_ARG"), (1e30, 1e9, "INVALID_ARG")):
        assert call("hicache_decode_attention", hc._DECODE_DESC, {**DECODE, "scale": scale, "ks": ks}, d) == status
        assert "scale" in hc.library().hicache_last_error().decode()


def test_caches_are_checked():
    for fn, packer, f in (("hicache_append_kv", hc._APPEND_DESC, APPEND),
                          ("hicache_decode_attention", hc._DECODE_DESC, DECODE)):
        for bufs, pages, status in (([0] * 4, 10, "INVALID_ARG"), ([A + 8] * 4, 10, "ALIGNMENT"),
                                    ([A, A, 0, A], 10, "INVALID_ARG"), ([A] * 4, 0, "INVALID_ARG"),
                                    ([A] * 4, 1 << 31, "INVALID_ARG")):
            assert call(fn, packer, f, desc(), kv=hc.DeviceKV(bufs, pages)) == status
        lib = hc.library()
        kv = hc.DeviceKV([A] * 4, 10)
        d = desc()
        assert getattr(lib, fn)(None, ctypes.byref(d), 0, packer.pack(*f.values()), None) == -1
        assert getattr(lib, fn)(kv.ref, None, 0, packer.pack(*f.values()), None) == -1
        assert getattr(lib, fn)(kv.ref, ctypes.byref(d), 0, None, None) == -1
        assert "NULL" in lib.hicache_last_error().decode()


EVICT = dict(table=A, weights=A, lens=A, keep=A, victims=A, num=A, out_table=2 * A, out_weights=2 * A, out_lens=2 * A,
             tb=20, wb=20, vb=20, otb=20, owb=20, P=16, batch=3, width=20, cap=20, sink=0, recent=1)


@pytest.mark.parametrize("change,status", [
    *[({k: 0}, "INVALID_ARG") for k in ("table", "weights", "lens", "keep", "victims", "num", "out_table",
                                        "out_weights", "out_lens")],
    *[({k: A + 2}, "ALIGNMENT") for k in ("table", "weights", "lens", "keep", "victims", "num", "out_table",
                                          "out_weights", "out_lens")],
    (dict(tb=-1), "INVALID_ARG"), (dict(wb=1 << 40), "INVALID_ARG"), (dict(vb=19), "INVALID_ARG"),
    (dict(otb=0), "INVALID_ARG"), (dict(owb=19), "INVALID_ARG"), (dict(P=0), "INVALID_ARG"),
    (dict(batch=-1), "INVALID_ARG"), (dict(width=0), "INVALID_ARG"), (dict(width=1 << 28), "INVALID_ARG"),
    (dict(cap=-1), "INVALID_ARG"), (dict(sink=-1), "INVALID_ARG"), (dict(recent=0), "INVALID_ARG"),
    (dict(out_table=A, otb=24), "INVALID_ARG"), (dict(out_weights=A, owb=24), "INVALID_ARG"),
])
def test_evict_refuses(change, status):
    before = hc.launch_count()
    rc = hc.library().hicache_evict_pages(hc._EVICT_DESC.pack(*{**EVICT, **change}.values()), None)
    assert hc.STATUS[rc] == status and hc.launch_count() == before
    assert hc.library().hicache_evict_pages(None, None) == -1


def test_workspace_sizes():
    out = ctypes.c_int64()
    lib = hc.library()

    def ask(d, *sizes):
        return lib.hicache_decode_workspace(ctypes.byref(d), *sizes, ctypes.byref(out))
    assert ask(desc(), 3, 4, 128, 128, 20, 0) == 0 and out.value > 0
    plain = out.value
    assert ask(desc(), 3, 4, 128, 128, 20, 1) == 0 and out.value >= plain + 3 * 4 * 20 * 16 * 4
    assert ask(desc(), 3, 5, 128, 128, 20, 0) == -1 and ask(desc(), 3, 4, 128, 128, 0, 0) == -1
    assert lib.hicache_decode_workspace(None, 3, 4, 128, 128, 20, 0, ctypes.byref(out)) == -1
    assert lib.hicache_decode_workspace(ctypes.byref(desc()), 3, 4, 128, 128, 20, 0, None) == -1
    with pytest.raises(hc.HiCacheError):
        hc.decode_workspace(desc(), 3, 4, 128, 64, 20)


def test_tensors_are_checked():
    """The binding's own checks: types, shapes, and tensors that are not on the
    current CUDA device."""
    torch = pytest.importorskip("torch")
    q = torch.zeros((3, 4, 128), dtype=torch.bfloat16)
    kv = hc.DeviceKV([A] * 4, 10)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="current CUDA device"):
        hc.decode_attention(kv, desc(), 0, q, i32(3, 5), i32(3), q, i32(64))
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        hc.decode_attention(kv, desc(), 0, q.float(), i32(3, 5), i32(3), q, i32(64))
    with pytest.raises(ValueError, match="current CUDA device"):
        hc.append_kv(kv, desc(), 0, q, q[:, :2], q[:, :2], torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="both None"):
        hc.append_kv(kv, desc(), 0, None, None, None, None)
    with pytest.raises(ValueError, match="current CUDA device"):
        hc.evict_pages(16, i32(3, 5), i32(3), torch.zeros((3, 5)), i32(3), i32(3, 5), i32(3))
    b16, cpu = torch.bfloat16, -1
    assert hc._tensor("t", q, b16, (3, 4, 128), cpu) == (512, 128, 1)
    for t, dtype, shape, device in ((q, torch.float16, (3, 4, 128), cpu), (q, b16, (3, 4, 64), cpu),
                                    (q, b16, (3, 512), cpu), (q, b16, (3, 4, 128), 0),
                                    (q.transpose(1, 2), b16, (3, 128, 4), cpu)):
        with pytest.raises(ValueError):
            hc._tensor("t", t, dtype, shape, device)
    with pytest.raises(ValueError, match="buffers"):
        hc._check_cache(hc.DeviceKV([A] * 3, 10), desc(), 0, cpu)
    small = torch.zeros((10 * 16, 255), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="bytes"):
        hc._check_cache(hc.DeviceKV([small] * 4, 10), desc(), 0, cpu)
    with pytest.raises(ValueError, match="expected device 0"):
        hc._check_cache(hc.DeviceKV([small] * 4, 1), desc(), 0, 0)
    with pytest.raises(ValueError, match="contiguous"):
        hc._check_cache(hc.DeviceKV([torch.zeros((320, 512), dtype=b16)[:, ::2]] * 4, 10), desc(), 0, cpu)
    with pytest.raises(hc.HiCacheError, match="aligned"):
        hc.decode_gave_up(q.view(-1)[1:])


def test_page_predicate(tmp_path):
    """The kernels' test of a page table's entry, at and around every edge."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "p.cpp"
    src.write_text("""
#include <cstdio>
#include <climits>
#include "hicache_serving.h"
using namespace hicache;
int main() {
  const long long n[] = {1, 7, INT32_MAX - 1, INT32_MAX};
  const int e[] = {INT32_MIN, -1, 0, 1, 6, 7, 8, INT32_MAX - 2, INT32_MAX - 1, INT32_MAX};
  for (long long k : n)
    for (int x : e)
      if (page_present(x, k) != ((long long)x >= 0 && (long long)x < k)) return 1;
  for (int g = 1; g <= 40; ++g) if (decode_rows(g) != (g <= 8 ? 8 : 16)) return 2;
  for (int h = 1; h <= 300; ++h) { const int r = latent_rows(h); if (r != 16 && r != 32 && r != 64) return 3; if (h <= 64 && r < h) return 4; }
  std::puts("ok");
}
""")
    exe = tmp_path / "p"
    subprocess.check_call(["g++", "-std=c++17", f"-I{root}/tiered_kv_cache_gb300/csrc", f"-I{root}/include",
                           "-I/usr/local/cuda/include", str(src), "-o", str(exe)])
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout.strip() == "ok"


def test_cache_types_are_checked():
    """A cache of another floating-point type than the call's; storage without one is taken."""
    torch = pytest.importorskip("torch")
    bf, fp, e4, e5 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.float8_e5m2
    for cache, dtype, es, ok in ((bf, bf, 2, True), (fp, fp, 2, True), (bf, fp, 2, False), (fp, bf, 2, False),
                                 (torch.int16, bf, 2, True), (torch.uint8, fp, 2, True), (torch.float32, bf, 2, False),
                                 (e4, bf, 1, True), (e4, fp, 1, True), (e5, bf, 1, False), (torch.uint8, bf, 1, True),
                                 (bf, bf, 1, False)):
        kv = hc.DeviceKV([torch.zeros((160, 256 * 4), dtype=cache)] * 4, 10)
        for _ in range(2):
            if ok:
                assert hc._check_cache(kv, desc(elem_bytes=es), 0, -1, dtype) == 2
            else:
                with pytest.raises(ValueError, match="expected torch"):
                    hc._check_cache(kv, desc(elem_bytes=es), 0, -1, dtype)
    # one cache, calls of both types
    kv = hc.DeviceKV([torch.zeros((160, 256), dtype=bf)] * 4, 10)
    assert hc._check_cache(kv, desc(), 0, -1, bf) == 2
    with pytest.raises(ValueError, match="expected torch.float16"):
        hc._check_cache(kv, desc(), 0, -1, fp)
    # and of one-byte elements in rows of as many bytes
    with pytest.raises(ValueError, match="expected torch.float8_e4m3fn"):
        hc._check_cache(kv, desc(elem_bytes=1, row_elems=512), 0, -1, bf)
