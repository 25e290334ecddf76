"""What query, prefix and merge attention refuse, before anything is enqueued, and the
geometry of their units against brute force: all without a GPU.  Addresses are made up;
nothing is read."""
import ctypes
import os
import subprocess

import pytest

import tiered_kv_cache_gb300 as hc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20      # an aligned address
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    from tiered_kv_cache_gb300 import build
    build.build()


def desc(**kw):
    d = dict(num_layers=2, num_buffers=2, page_size=16, elem_bytes=2, row_elems=256, host_num_pages=1, layout=0,
             launch_ctas=0, flags=0, reserved=0)
    d.update(kw)
    return hc.PoolDesc(*d.values())


def call(fn, packer, fields, d, layer=0, kv=None):
    kv = kv or hc.DeviceKV([A] * (d.num_buffers * d.num_layers), 10)
    before = hc.launch_count()
    rc = getattr(hc.library(), fn)(kv.ref, ctypes.byref(d), layer, packer.pack(*fields.values()), None)
    assert hc.launch_count() == before
    return hc.STATUS[rc]


QUERY = dict(q=A, out=2 * A, starts=A, table=A, lens=A, lse=A, ws=A, ws_bytes=1 << 40, qt=512, qh=128, ot=512, oh=128,
             tb=20, lt=4, n=7, dtype=0, batch=3, hq=4, d=128, width=20, window=0, causal=0, reserved=0, scale=0.1, ks=1.0,
             vs=1.0)


@pytest.mark.parametrize("change,status", [
    (dict(q=0), "INVALID_ARG"), (dict(out=0), "INVALID_ARG"), (dict(starts=0), "INVALID_ARG"),
    (dict(table=0), "INVALID_ARG"), (dict(lens=0), "INVALID_ARG"), (dict(ws=0), "INVALID_ARG"),
    (dict(ws=A + 128), "ALIGNMENT"), (dict(ws_bytes=0), "INVALID_ARG"), (dict(ws_bytes=-1), "INVALID_ARG"),
    (dict(q=A + 8), "ALIGNMENT"), (dict(out=A + 2), "ALIGNMENT"), (dict(qt=516), "ALIGNMENT"), (dict(oh=132), "ALIGNMENT"),
    (dict(starts=A + 2), "ALIGNMENT"), (dict(table=A + 1), "ALIGNMENT"), (dict(lens=A + 3), "ALIGNMENT"),
    (dict(lse=A + 2), "ALIGNMENT"), (dict(qt=-8), "INVALID_ARG"), (dict(ot=0), "INVALID_ARG"), (dict(oh=120), "INVALID_ARG"),
    (dict(tb=-1), "INVALID_ARG"), (dict(tb=1 << 40), "INVALID_ARG"), (dict(lt=3), "INVALID_ARG"),
    (dict(n=-1), "INVALID_ARG"), (dict(n=1 << 29), "INVALID_ARG"), (dict(n=1 << 62), "INVALID_ARG"),
    (dict(dtype=2), "INVALID_ARG"), (dict(batch=-1), "INVALID_ARG"), (dict(batch=65536), "INVALID_ARG"),
    (dict(hq=0), "INVALID_ARG"), (dict(hq=5), "INVALID_ARG"), (dict(hq=4098), "INVALID_ARG"),
    (dict(d=0), "INVALID_ARG"), (dict(d=96), "INVALID_ARG"), (dict(d=4), "INVALID_ARG"), (dict(d=-128), "INVALID_ARG"),
    (dict(width=0), "INVALID_ARG"), (dict(width=1 << 27), "INVALID_ARG"), (dict(window=-1, causal=1), "INVALID_ARG"),
    (dict(window=5), "INVALID_ARG"), (dict(reserved=1), "INVALID_ARG"), (dict(scale=NAN), "INVALID_ARG"),
    (dict(scale=-INF), "INVALID_ARG"), (dict(ks=0.5), "INVALID_ARG"), (dict(vs=0.0), "INVALID_ARG"),
])
def test_query_refuses(change, status):
    assert call("hicache_query_attention", hc._QUERY_DESC, {**QUERY, **change}, desc()) == status


def test_query_accepts_nothing_to_do():
    for change in (dict(n=0), dict(batch=0)):
        assert call("hicache_query_attention", hc._QUERY_DESC, {**QUERY, "q": 0, "starts": 0, **change}, desc()) == "OK"


PREFIX = dict(q=A, out=2 * A, starts=A, shared=A, prefix=A, table=A, lens=A, lse=A, ws=A, ws_bytes=1 << 40, qb=512, qh=128,
              ob=512, oh=128, pb=30, tb=20, lb=4, dtype=0, batch=3, groups=2, hq=4, d=128, wide=30, width=20, reserved=0,
              scale=0.1, ks=1.0, vs=1.0)


@pytest.mark.parametrize("change,status", [
    *[({k: 0}, "INVALID_ARG") for k in ("q", "out", "starts", "shared", "prefix", "table", "lens", "ws", "ws_bytes")],
    *[({k: A + 2}, "ALIGNMENT") for k in ("q", "out", "starts", "shared", "prefix", "table", "lens", "lse", "ws")],
    (dict(qb=510), "ALIGNMENT"), (dict(qh=-128), "INVALID_ARG"), (dict(ob=0), "INVALID_ARG"), (dict(oh=64), "INVALID_ARG"),
    (dict(pb=-1), "INVALID_ARG"), (dict(tb=1 << 40), "INVALID_ARG"), (dict(lb=3), "INVALID_ARG"),
    (dict(dtype=-1), "INVALID_ARG"), (dict(batch=-1), "INVALID_ARG"), (dict(batch=65536), "INVALID_ARG"),
    (dict(groups=-1), "INVALID_ARG"), (dict(groups=65536), "INVALID_ARG"), (dict(hq=3), "INVALID_ARG"),
    (dict(d=264), "INVALID_ARG"), (dict(wide=0), "INVALID_ARG"), (dict(width=0), "INVALID_ARG"),
    (dict(wide=1 << 28), "INVALID_ARG"), (dict(reserved=3), "INVALID_ARG"), (dict(scale=INF), "INVALID_ARG"),
    (dict(ks=2.0), "INVALID_ARG"), (dict(vs=-1.0), "INVALID_ARG"),
])
def test_prefix_refuses(change, status):
    assert call("hicache_prefix_attention", hc._PREFIX_DESC, {**PREFIX, **change}, desc()) == status


def test_prefix_accepts_nothing_to_do():
    assert call("hicache_prefix_attention", hc._PREFIX_DESC, {**PREFIX, "batch": 0, "q": 0}, desc()) == "OK"


@pytest.mark.parametrize("d,change,layer,status", [
    (desc(num_buffers=1, row_elems=128), {}, 0, "INVALID_ARG"), (desc(num_buffers=1, row_elems=576), dict(d=576), 0, "INVALID_ARG"),
    (desc(elem_bytes=4), {}, 0, "INVALID_ARG"), (desc(), {}, 2, "INVALID_ARG"), (desc(), {}, -1, "INVALID_ARG"),
    (desc(elem_bytes=1, row_elems=240), dict(d=120), 0, "INVALID_ARG"),
    (desc(elem_bytes=1), dict(ks=1e38, scale=1e38), 0, "INVALID_ARG"),
])
def test_pools_are_checked(d, change, layer, status):
    assert call("hicache_query_attention", hc._QUERY_DESC, {**QUERY, **change}, d, layer) == status
    assert call("hicache_prefix_attention", hc._PREFIX_DESC, {**PREFIX, **change}, d, layer) == status


def test_caches_and_descriptors_are_checked():
    lib = hc.library()
    for fn, packer, f in (("hicache_query_attention", hc._QUERY_DESC, QUERY),
                          ("hicache_prefix_attention", hc._PREFIX_DESC, PREFIX)):
        for bufs, status in (([0] * 4, "INVALID_ARG"), ([A + 8] * 4, "ALIGNMENT")):
            assert call(fn, packer, f, desc(), kv=hc.DeviceKV(bufs, 10)) == status
        kv, d = hc.DeviceKV([A] * 4, 10), desc()
        assert getattr(lib, fn)(None, ctypes.byref(d), 0, packer.pack(*f.values()), None) == -1
        assert getattr(lib, fn)(kv.ref, None, 0, packer.pack(*f.values()), None) == -1
        assert getattr(lib, fn)(kv.ref, ctypes.byref(d), 0, None, None) == -1
    assert lib.hicache_merge_attention(None, None) == -1


MERGE = dict(outs=[A, 2 * A, 3 * A], lses=[A, 2 * A, 3 * A], out=4 * A, lse=4 * A, ot=[512] * 3, oh=[128] * 3, lt=[4] * 3,
             out_t=512, out_h=128, lse_t=4, n=5, dtype=0, parts=3, heads=4, d=128)


def merge(**change):
    f = {**MERGE, **change}
    pad = lambda x: list(x) + [0] * (hc.MERGE_PARTS - len(x))  # noqa: E731
    args = [*pad(f["outs"]), *pad(f["lses"]), f["out"], f["lse"], *pad(f["ot"]), *pad(f["oh"]), *pad(f["lt"]), f["out_t"],
            f["out_h"], f["lse_t"], f["n"], f["dtype"], f["parts"], f["heads"], f["d"]]
    before = hc.launch_count()
    rc = hc.library().hicache_merge_attention(hc._MERGE_DESC.pack(*args), None)
    assert hc.launch_count() == before
    return hc.STATUS[rc]


@pytest.mark.parametrize("change,status", [
    (dict(outs=[A, 0, 3 * A]), "INVALID_ARG"), (dict(lses=[A, 2 * A, 0]), "INVALID_ARG"), (dict(out=0), "INVALID_ARG"),
    (dict(outs=[A, 2 * A + 8, 3 * A]), "ALIGNMENT"), (dict(lses=[A + 2, 2 * A, 3 * A]), "ALIGNMENT"),
    (dict(out=4 * A + 8), "ALIGNMENT"), (dict(lse=4 * A + 1), "ALIGNMENT"), (dict(ot=[512, 510, 512]), "ALIGNMENT"),
    (dict(oh=[128, -128, 128]), "INVALID_ARG"), (dict(lt=[4, 4, -4]), "INVALID_ARG"), (dict(out_t=0), "INVALID_ARG"),
    (dict(out_h=120), "INVALID_ARG"), (dict(lse_t=3), "INVALID_ARG"), (dict(parts=0), "INVALID_ARG"),
    (dict(parts=9), "INVALID_ARG"), (dict(parts=-1), "INVALID_ARG"), (dict(heads=0), "INVALID_ARG"),
    (dict(d=0), "INVALID_ARG"), (dict(d=12), "INVALID_ARG"), (dict(d=1 << 21), "INVALID_ARG"), (dict(dtype=2), "INVALID_ARG"),
    (dict(n=-1), "INVALID_ARG"), (dict(n=1 << 40), "INVALID_ARG"), (dict(n=1 << 62), "INVALID_ARG"),
    (dict(out=A, out_t=1024), "INVALID_ARG"), (dict(lse=2 * A), "INVALID_ARG"),
])
def test_merge_refuses(change, status):
    assert merge(**change) == status


def test_merge_accepts_nothing_to_do():
    assert merge(n=0, out=0) == "OK"


def test_workspace_sizes():
    out = ctypes.c_int64()
    lib, d = hc.library(), desc()
    ask = lambda f, *x: getattr(lib, f)(ctypes.byref(d), *x, ctypes.byref(out))  # noqa: E731
    assert ask("hicache_query_workspace", 3, 7, 4, 128, 20) == 0 and out.value > 0
    for bad in ((-1, 7, 4, 128, 20), (3, -1, 4, 128, 20), (3, 1 << 40, 4, 128, 20), (3, 7, 5, 128, 20), (3, 7, 4, 128, 0)):
        assert ask("hicache_query_workspace", *bad) == -1
    assert ask("hicache_prefix_workspace", 3, 2, 4, 128, 30, 20) == 0 and out.value > 0
    one = out.value
    assert ask("hicache_prefix_workspace", 3, 2, 4, 128, 30, 5000) == 0 and out.value > one
    for bad in ((-1, 2, 4, 128, 30, 20), (3, -1, 4, 128, 30, 20), (3, 2, 4, 64 + 4, 30, 20), (3, 2, 4, 128, 0, 20),
                (3, 2, 4, 128, 30, 0)):
        assert ask("hicache_prefix_workspace", *bad) == -1
    assert lib.hicache_query_workspace(None, 3, 7, 4, 128, 20, ctypes.byref(out)) == -1
    assert lib.hicache_prefix_workspace(ctypes.byref(d), 3, 2, 4, 128, 30, 20, None) == -1
    with pytest.raises(hc.HiCacheError):
        hc.query_workspace(desc(num_buffers=1, row_elems=576), 1, 1, 16, 576, 4)


def test_tensors_are_checked():
    """The binding's own checks: types, shapes, and tensors that are not on the current
    CUDA device."""
    torch = pytest.importorskip("torch")
    q = torch.zeros((3, 4, 128), dtype=torch.bfloat16)
    kv = hc.DeviceKV([A] * 4, 10)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    f32 = torch.zeros((3, 4))
    with pytest.raises(ValueError, match="current CUDA device"):
        hc.query_attention(kv, desc(), 0, q, i32(4), i32(3, 5), i32(3), q, i32(64))
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        hc.query_attention(kv, desc(), 0, q.float(), i32(4), i32(3, 5), i32(3), q, i32(64))
    with pytest.raises(ValueError, match="3"):
        hc.prefix_attention(kv, desc(), 0, q[0], i32(3), i32(2, 5), i32(2), i32(3, 5), i32(3), q, i32(64))
    with pytest.raises(ValueError, match="current CUDA device"):
        hc.prefix_attention(kv, desc(), 0, q, i32(3), i32(2, 5), i32(2), i32(3, 5), i32(3), q, i32(64))
    with pytest.raises(ValueError, match="current CUDA device"):
        hc.merge_attention([q, q], [f32, f32], q)
    for outs, lses in (([], []), ([q] * 9, [f32] * 9), ([q, q], [f32])):
        with pytest.raises(ValueError, match="of each"):
            hc.merge_attention(outs, lses, q)


def run_host(tmp_path, body):
    """Compiles and runs a program over the kernels' header; its output."""
    src, exe = tmp_path / "h.cpp", tmp_path / "h"
    src.write_text('#include <climits>\n#include <cstdio>\n#include <initializer_list>\n#include "hicache_serving.h"\n'
                   "using namespace hicache;\nint main() {\n" + body + '\n  std::puts("ok");\n}\n')
    subprocess.check_call(["g++", "-std=c++17", f"-I{ROOT}/tiered_kv_cache_gb300/csrc", f"-I{ROOT}/include",
                           "-I/usr/local/cuda/include", str(src), "-o", str(exe)])
    return subprocess.run([str(exe)], capture_output=True, text=True).stdout.strip()


def test_units_cover_what_their_rows_see(tmp_path):
    """Every row in one unit, every token that a row sees in its unit's blocks, no block
    that none of its rows sees; with more queries than tokens, windows, odd groups."""
    assert run_host(tmp_path, """
  for (int G : {1, 3, 4, 7, 16})
    for (int nq : {1, 2, 5, 63, 64, 65, 130})
      for (int kv : {0, 1, 5, 64, 65, 128, 300, 517})
        for (int causal : {0, 1})
          for (int window : {0, 1, 30, 200})
            for (int rows : {128, 256})
              for (int block : {64, 128}) {
                if (window && !causal) continue;
                const FastDiv group = make_fastdiv(G);
                const int units = query_units(nq, G, rows);
                int next = 0;
                for (int m = 0; m < units; ++m) {
                  const QueryUnit u = query_unit(m, nq, kv, group, rows, block, causal, window);
                  if (u.row0 != next || u.rows < 1 || u.rows > rows) return 1;
                  next += u.rows;
                  bool first = false, last = false;
                  for (int r = u.row0; r < u.row0 + u.rows; ++r) {
                    int lo, hi;
                    const int i = r / G;
                    query_sees(i, nq, kv, causal, window, &lo, &hi);
                    const int pos = kv - nq + i, end = causal ? (pos + 1 > 0 ? pos + 1 : 0) : kv;
                    const int begin = window && end > window ? end - window : 0;
                    if (hi != end || (end > 0 && lo != begin) || lo > hi) return 2;
                    if (hi > lo && (lo < u.blk0 * block || hi > (u.blk0 + u.blocks) * block)) return 3;
                    first |= hi > lo && lo < (u.blk0 + 1) * block;
                    last |= hi > lo && hi > (u.blk0 + u.blocks - 1) * block;
                  }
                  if (u.blocks > 0 && !(first && last)) return 4;
                  if (query_cost(u.blocks) != (u.blocks ? u.blocks + kQueryStart : 0)) return 5;
                }
                if (next != nq * G) return 6;
              }
  // the largest: no step leaves 32 bits
  const FastDiv one = make_fastdiv(1);
  const int most = INT_MAX - 5000;
  const QueryUnit u = query_unit(query_units(most, 1, 256) - 1, most, INT_MAX - 2000, one, 256, 128, 1, 0);
  if (u.row0 + u.rows != most || u.blk0 != 0 || u.blocks != (INT_MAX - 2000) / 128 + 1) return 7;
  int lo, hi;
  query_sees(0, most, 0, 1, 100, &lo, &hi);
  if (lo != 0 || hi != 0) return 8;""") == "ok"


def test_open_records_stay_in_the_call(tmp_path):
    """Every piece that a join reads lies in the workspace, whatever a record holds."""
    assert run_host(tmp_path, """
  const int e[] = {INT_MIN, -1, 0, 1, 2, 3, 75, 150, 151, 152, 153, 0x3f800000, INT_MAX};
  for (int chunk : e)
    for (int pieces : e) {
      const bool want = chunk >= 0 && chunk < kQueryCtas && pieces >= 2 && (long long)chunk + pieces <= kQueryCtas;
      if (query_open(chunk, pieces, kQueryCtas) != want) return 1;
    }
  static_assert(kOwnTokens % 128 == 0, "whole blocks");""") == "ok"
