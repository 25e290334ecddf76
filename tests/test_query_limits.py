"""The arithmetic of query, prefix and merge attention at the limits of the sizes that the
calls accept, without a GPU."""
import ctypes

import pytest

import tiered_kv_cache_gb300 as hc
from test_query_refusals import PREFIX, call, desc, merge, run_host


@pytest.fixture(scope="module", autouse=True)
def built():
    from tiered_kv_cache_gb300 import build
    build.build()


def test_parts_of_own_tokens(tmp_path):
    """A sequence's own tokens lie in parts of kOwnTokens, each token in one, up to the longest
    table; the workspace holds as many."""
    assert run_host(tmp_path, """
  const long long most = INT_MAX - 1024ll;            // max_pages * page_size
  for (long long n : {0ll, 1ll, 4095ll, 4096ll, 4097ll, 8192ll, 1000000007ll, most - 4096, most + 1024 - kOwnTokens, most + 1025 - kOwnTokens, most - 1, most}) {
    const long long want = (n + kOwnTokens - 1) / kOwnTokens;
    if (own_parts(int32_t(n)) != want) return 1;
    long long next = 0;
    for (long long i = want > 3 ? want - 3 : 0; i < want; ++i) {
      const int32_t lo = int32_t(i) * kOwnTokens;
      if (i == (want > 3 ? want - 3 : 0)) next = lo;
      const int32_t hi = own_end(lo, int32_t(n));
      if (lo != next || hi <= lo || hi - lo > kOwnTokens || hi > n) return 2;
      next = hi;
    }
    if (next != n) return 3;
  }""") == "ok"


def test_workspace_of_the_longest_tables():
    out = ctypes.c_int64()
    d = desc(page_size=1000)
    ask = lambda own: hc.library().hicache_prefix_workspace(ctypes.byref(d), 1, 1, 4, 128, 1, own, ctypes.byref(out))  # noqa: E731
    sizes = []
    for pages in (2_147_480, 2_147_482):
        assert ask(pages) == 0
        sizes.append(out.value)
    # 524,288 parts and the prefix's, each of 4 rows of 128 elements and a log-sum in 32 bits
    assert sizes[0] <= sizes[1] and sizes[1] >= 524_289 * 4 * 129 * 4
    assert ask(2_147_483) == -1


def test_counters_of_units_do_not_wrap(tmp_path):
    """A call may have more units than 32 bits count: behind 2^32 the counter would begin anew, with
    units whose place in their sequence is negative."""
    assert run_host(tmp_path, """
  const long long parts = own_parts(INT_MAX - 1024), units = 65535ll * parts * query_units(1, 1, 256);
  QueryParams p{};
  if (units <= (1ll << 32)) return 1;
  if (sizeof(*p.next) * CHAR_BIT < 64) return 2;""") == "ok"


@pytest.mark.parametrize("heads,stride", [((1 << 25) + 1, 1 << 39), ((1 << 27) - 300, 1 << 38), ((1 << 24) + 1, 1 << 39)])
def test_merge_refuses_heads_that_overlap(heads, stride):
    """Rows that lie on one another, of strides that leave 64 bits times the number of heads."""
    change = dict(n=2, heads=heads, d=8, out_t=stride, out_h=stride, ot=[stride] * 3, oh=[stride] * 3, lt=[heads] * 3, lse_t=heads)
    assert merge(**change) == "INVALID_ARG"
    # apart, the call goes on to what is checked next
    assert merge(**{**change, "out_h": 8, "lse": 4 << 20 | 2}) == "ALIGNMENT"
    assert merge(**{**change, "out_t": 8, "out_h": 16, "lse": 4 << 20 | 2}) == "ALIGNMENT"


def test_prefix_without_a_table():
    """Without groups there is no prefix table: its width may be 0."""
    out, d = ctypes.c_int64(), desc()
    ask = lambda groups, wide: hc.library().hicache_prefix_workspace(ctypes.byref(d), 3, groups, 4, 128, wide, 20, ctypes.byref(out))  # noqa: E731
    assert ask(0, 1) == 0
    one = out.value
    assert ask(0, 0) == 0 and out.value == one
    assert ask(1, 0) == -1 and ask(0, -1) == -1
    none = {**PREFIX, "groups": 0, "starts": 0, "shared": 0, "prefix": 0, "wide": 0, "pb": 0}
    # the sizes pass: what is checked behind them refuses
    assert call("hicache_prefix_attention", hc._PREFIX_DESC, {**none, "lse": PREFIX["lse"] + 2}, d) == "ALIGNMENT"
    assert call("hicache_prefix_attention", hc._PREFIX_DESC, {**none, "groups": 1}, d) == "INVALID_ARG"
