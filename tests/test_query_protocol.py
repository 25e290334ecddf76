"""The barriers of query attention's kernel under many random schedules (see query_protocol), with the
constants of its header; and mistakes that the simulation must find."""
import pytest

from query_protocol import Kernel, Sizes, pieces_of
from test_query_refusals import run_host


@pytest.fixture(scope="module")
def header(tmp_path_factory):
    """Stages by head_dim, and the other constants."""
    out = run_host(tmp_path_factory.mktemp("h"), """
  std::printf("%d %d %d %d %d %d\\n", query_stages(64), query_stages(128), query_stages(256), kQueryInfo, kQueryTurns, kQueryPieces);
""").split()
    return [int(x) for x in out[:6]]


def sizes(header, dim, **change):
    s64, s128, s256, info, turns, ring = header
    tiles, parts, stages = {64: (2, 2, s64), 128: (2, 2, s128), 256: (1, 1, s256)}[dim]
    return Sizes(**{**dict(tiles=tiles, parts=parts, stages=stages, info=info, turns=turns, ring=ring), **change})


def try_all(z, mode, seeds, **kw):
    for seed in seeds:
        Kernel(seed, z, mode, pieces_of(seed, z.tiles), **kw).run()


@pytest.mark.parametrize("mode", ["boxes", "rows", "registers"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_any_schedule(header, dim, mode):
    try_all(sizes(header, dim), mode, range(25))


@pytest.mark.parametrize("dim,mode,change,without", [
    (128, "boxes", dict(turns=4), ()),            # a parity wait two phases early
    (128, "boxes", dict(info=4), ()),             # what is present overwritten before it is read
    (128, "rows", {}, ("group",)),                # copying warps apart
    (128, "boxes", {}, ("added",)),               # the next Q over sums that are still to be read
    (128, "boxes", {}, ("exps",)), (64, "registers", {}, ("empty",)), (256, "boxes", {}, ("scores",)),
    (64, "boxes", {}, ("taken",)), (256, "rows", {}, ("pv",)), (128, "boxes", {}, ("q",)),
])
def test_mistakes_are_found(header, dim, mode, change, without):
    with pytest.raises(AssertionError):
        try_all(sizes(header, dim, **change), mode, range(150), without=without)


def test_the_headers_conditions(tmp_path):
    """What the kernel asserts of its constants, at their limits."""
    assert run_host(tmp_path, """
  static_assert(query_turns_hold(3, 5) && !query_turns_hold(4, 5) && query_turns_hold(4, 8) && !query_turns_hold(5, 8), "");
  static_assert(query_info_holds(7, 3, 5) && !query_info_holds(6, 3, 5) && query_info_holds(7, 3, 8), "");
""") == "ok"
