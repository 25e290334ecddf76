"""What hicache_append_kv hands its kernel, read on the CPU: the library's own
objects, with a stand-in for the launch that prints the parameters.  Addresses
are made up; nothing is read."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include "hicache.h"
#include "hicache_serving.h"
namespace hicache {
int launch_append(const AppendParams &p, void *) {
  std::printf("q_norm=%d k_norm=%d q_st=%lld q_sh=%lld o_st=%lld o_sh=%lld k_st=%lld k_sh=%lld v_st=%lld v_sh=%lld ",
              p.q_norm, p.k_norm, (long long)p.q_st, (long long)p.q_sh, (long long)p.o_st, (long long)p.o_sh,
              (long long)p.k_st, (long long)p.k_sh, (long long)p.v_st, (long long)p.v_sh);
  return 0;
}
}  // namespace hicache
// arguments: name=value, over a plain call of 3 tokens, 4 query and 2 kv heads of 128
int main(int argc, char **argv) {
  const long long A = 1 << 20;
  char *const base = reinterpret_cast<char *>(A);
  hicache_pool_desc d{};
  d.num_layers = 1, d.num_buffers = 2, d.page_size = 16, d.elem_bytes = 2, d.row_elems = 256, d.host_num_pages = 1;
  void *bufs[2] = {base, base};
  hicache_device_kv kv{};
  kv.buf_ptrs = bufs, kv.device_num_pages = 10;
  hicache_append_desc a{};
  a.q = a.q_out = base, a.k = a.v = a.q_weight = a.k_weight = base;
  a.slots = reinterpret_cast<int64_t *>(base);
  a.q_token_stride = a.q_out_token_stride = 512, a.q_head_stride = a.q_out_head_stride = 128;
  a.k_token_stride = a.v_token_stride = 256, a.k_head_stride = a.v_head_stride = 128;
  a.num_tokens = 3, a.q_heads = 4, a.kv_heads = 2, a.head_dim = 128, a.q_norm_dim = a.k_norm_dim = 128;
  a.eps = 1e-6f, a.k_scale = a.v_scale = 1.f;
  for (int i = 1; i < argc; ++i) {
    const char *eq = std::strchr(argv[i], '=');
    const size_t n = size_t(eq - argv[i]);
    const long long x = std::atoll(eq + 1);
    auto is = [&](const char *s) { return std::strlen(s) == n && !std::strncmp(argv[i], s, n); };
    if (is("q_heads")) a.q_heads = int(x);
    else if (is("kv_heads")) a.kv_heads = int(x);
    else if (is("row")) d.row_elems = x;
    else if (is("n")) a.num_tokens = x;
    else if (is("q_weight")) a.q_weight = reinterpret_cast<void *>(x);
    else if (is("k_weight")) a.k_weight = reinterpret_cast<void *>(x);
    else if (is("qst")) a.q_token_stride = x;
    else if (is("qsh")) a.q_head_stride = x;
    else if (is("ost")) a.q_out_token_stride = x;
    else if (is("osh")) a.q_out_head_stride = x;
    else if (is("kst")) a.k_token_stride = x;
    else if (is("ksh")) a.k_head_stride = x;
    else if (is("vst")) a.v_token_stride = x;
    else if (is("vsh")) a.v_head_stride = x;
    else return 1;
  }
  std::printf("rc=%d\n", hicache_append_kv(&kv, &d, 0, &a, nullptr));
  return 0;
}
"""


@pytest.fixture(scope="module")
def params(tmp_path_factory):
    """Runs a call with some arguments changed: its return code and the kernel's parameters."""
    from tiered_kv_cache_gb300 import build as b
    b.build()
    d = tmp_path_factory.mktemp("params")
    (d / "m.cpp").write_text(MAIN)
    cuda = "/usr/local/cuda"
    objs = [os.path.join(b.BUILD, s + ".o") for s in b.SOURCES if s != "hicache_append.cu"]
    subprocess.check_call(["g++", "-std=c++17", f"-I{ROOT}/tiered_kv_cache_gb300/csrc", f"-I{ROOT}/include",
                           f"-I{cuda}/include", str(d / "m.cpp"), *objs, f"-L{cuda}/lib64", "-lcudart_static", "-ldl",
                           "-lrt", "-lpthread", "-o", str(d / "m")])

    def run(**change):
        r = subprocess.run([str(d / "m")] + [f"{k}={v}" for k, v in change.items()], capture_output=True, text=True,
                           check=True)
        return {k: int(v) for k, v in (x.split("=") for x in r.stdout.split())}
    return run


def test_plain_call(params):
    p = params()
    assert (p["rc"], p["q_norm"], p["k_norm"]) == (0, 128, 128)


@pytest.mark.parametrize("weight", [0, (1 << 20) + 2])
def test_weights_of_absent_heads_are_not_read(params, weight):
    """A call of queries alone, or of keys and values alone: the norm of the
    other kind, whose weight may be NULL or at any address, is left out."""
    p = params(kv_heads=0, k_weight=weight)
    assert (p["rc"], p["q_norm"], p["k_norm"]) == (0, 128, 0)
    p = params(q_heads=0, q_weight=weight)
    assert (p["rc"], p["q_norm"], p["k_norm"]) == (0, 0, 128)


def run_host(tmp_path, body):
    """Compiles and runs a program over the kernels' header; its output."""
    src, exe = tmp_path / "h.cpp", tmp_path / "h"
    src.write_text('#include <climits>\n#include <cstdio>\n#include <initializer_list>\n#include "hicache_serving.h"\nusing namespace hicache;\n'
                   "int main() {\n" + body + '\n  std::puts("ok");\n}\n')
    subprocess.check_call(["g++", "-std=c++17", f"-I{ROOT}/tiered_kv_cache_gb300/csrc", f"-I{ROOT}/include",
                           "-I/usr/local/cuda/include", str(src), "-o", str(exe)])
    return subprocess.run([str(exe)], capture_output=True, text=True).stdout.strip()


def test_idle_sequences_are_counted_to_the_largest_batch(tmp_path):
    """Strips and idle sequences of one sum, at and around 2^15 idle ones and at
    the largest batch."""
    assert run_host(tmp_path, """
  const uint64_t idle[] = {0, 1, 2, 32767, 32768, 32769, 40000, 65534, 65535};
  const int64_t strips[] = {0, 1, 5, (int64_t(1) << 42) + 3, (int64_t(1) << 48) - 1};
  for (uint64_t i : idle)
    for (int64_t s : strips) {
      uint64_t sum = uint64_t(s);
      for (uint64_t k = 0; k < i; ++k) sum += kIdleSeq;
      if (idle_seqs(sum) != i || strips_in(sum) != s) return 1;
    }""") == "ok"


def test_pieces_to_join(tmp_path):
    """Every piece that a join reads lies in the workspace, whatever the words say."""
    assert run_host(tmp_path, """
  const int e[] = {INT_MIN, INT_MIN + 1, -153, -152, -1, 0, 1, 2, 3, 37, 38, 75, 76, 77, 150, 151, 152, 153,
                   0x3f800000, 0x7f800000, INT_MAX - 1, INT_MAX};
  for (int QB = 1; QB <= 64; ++QB) {
    const long long groups = kDecodeCtas / QB;
    for (int x : e)
      for (int y : e) {
        const bool want = y >= 2 && x >= 0 && (long long)x + y <= groups;
        if (pieces_to_join(x, y, QB) != want) return 1;
        if (want && (((long long)x + y - 1) * QB + QB - 1) >= kDecodeCtas) return 2;
      }
  }""") == "ok"


def test_evict_count_at_the_ends_of_the_range(tmp_path):
    """Pages that leave, against 128 bits, for sinks, recent pages and budgets up
    to the largest; the first page that is too recent stays in 32 bits."""
    assert run_host(tmp_path, """
  const int e[] = {0, 1, 2, 3, 7, 100, 4096, INT_MAX / 2, INT_MAX - 1025, INT_MAX - 1, INT_MAX};
  for (int n : e)
    for (int sink : e)
      for (int recent : e)
        for (int keep : {INT_MIN, -1, 0, 1, 2, 3, 100, INT_MAX})
          for (int cap : e) {
            if (recent < 1) continue;
            __int128 may = 0, over = (__int128)n - (keep > 0 ? keep : 0), want;
            if ((__int128)n - recent > sink) may = (__int128)n - recent - sink;
            want = over < 0 ? 0 : over;
            if (may < want) want = may;
            if (cap < want) want = cap;
            if (evict_count(n, sink, recent, keep, cap) != want) return 1;
            if ((__int128)n - recent < INT_MIN) return 2;
          }""") == "ok"


def test_strides_of_single_tokens_and_heads_are_not_used(params):
    """A dimension of one may have any stride, odd, negative or huge; of several it is
    checked and passed on."""
    strides = ["qst", "qsh", "ost", "osh", "kst", "ksh", "vst", "vsh"]
    names = ["q_st", "q_sh", "o_st", "o_sh", "k_st", "k_sh", "v_st", "v_sh"]
    given = [512, 128, 512, 128, 256, 128, 256, 128]
    p = params()
    assert p["rc"] == 0 and [p[x] for x in names] == given
    for odd in (1, 3, -7, 2 ** 50, 132):
        p = params(n=1, q_heads=1, kv_heads=1, row=128, **{x: odd for x in strides})
        assert p["rc"] == 0 and [p[x] for x in names] == [0] * 8
        p = params(n=1, **{x: odd for x in strides[::2]})
        assert p["rc"] == 0 and [p[x] for x in names] == [0, 128] * 4
        p = params(q_heads=1, kv_heads=1, row=128, **{x: odd for x in strides[1::2]})
        assert p["rc"] == 0 and [p[x] for x in names] == [512, 0, 512, 0, 256, 0, 256, 0]
        for x in strides:
            assert params(**{x: odd})["rc"] != 0
