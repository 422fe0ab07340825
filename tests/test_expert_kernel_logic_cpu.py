"""Logic of the expert layer's kernels that can be followed without a GPU, taken from their
source: the hand-over of shared-memory slots between warps, and loops at the ends of their
index types."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from combine_mp_layout_gb300 import _build, binding as B


def source(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        return f.read()


def wgrad_roles():
    """The weights' gradient's code per role (converting warps, storing warps, and so on)."""
    text = source("mp_expert_wgrad.cu")
    parts = re.split(r"\n  (?:if|\} else if) \(((?:warp|rank) [^\n]*)\) \{\n", text)
    return {cond: body for cond, body in zip(parts[1::2], parts[2::2])}


def constant(text, name):
    return int(re.search(r"constexpr int %s = (\d+);" % name, text).group(1))


def test_wgrad_powers_of_two_are_given_back_by_every_reader():
    """A slot is refilled when every warp that waits for it and reads it has said so."""
    text = source("mp_expert_wgrad.cu")
    conv = constant(text, "kConvWarps")
    count = re.search(r"mbar_init\(&tail->nempty\[i\], ([^)]*)\);", text).group(1)
    warps = {"warp < kConvWarps": conv, "warp < kConvWarps + 4": 4}
    readers = [c for c, body in wgrad_roles().items() if "&tail->nfull[" in body
               and "bounded_wait" in body.split("&tail->nfull[")[0].splitlines()[-1]]
    assert sorted(readers) == sorted(warps)
    assert eval(count, {"kConvWarps": conv}) == sum(warps.values())
    for c in readers:
        assert "mbar_arrive(&tail->nempty[" in wgrad_roles()[c], c


def test_wgrad_late_warp_never_misses_a_phase():
    """Tiles of one stage, which the two groups of converting warps take in turn: in every order
    of events a converting warp that is late still finds the phase that it waits for (a barrier's
    parity tells one phase from the next, not from the one after that)."""
    text = source("mp_expert_wgrad.cu")
    slots, tiles = constant(text, "kNorms"), 12
    gives_back = "mbar_arrive(&tail->nempty[" in wgrad_roles()["warp < kConvWarps"]
    todo, known = [(0, 0, 0)], {(0, 0, 0)}  # tiles looked up, stored, passed by the late warp
    while todo:
        filled, stored, passed = todo.pop()
        if passed < tiles:
            phases = len(range(passed % slots, filled, slots))  # completed on its slot
            assert phases <= passed // slots + 1, (filled, stored, passed)
        steps = []
        if filled < tiles and (filled < slots or (
                stored > filled - slots and (not gives_back or passed > filled - slots))):
            steps.append((filled + 1, stored, passed))
        # a tile is finished once its one stage is converted: the late warp's in every other tile
        if stored < filled and (stored % 2 == 0 or passed > stored):
            steps.append((filled, stored + 1, passed))
        if passed < filled and passed < tiles:
            steps.append((filled, stored, passed + 1))
        for s in steps:
            if s not in known:
                known.add(s)
                todo.append(s)
    assert (tiles, tiles, tiles) in known


def run_c(tmp_path, body):
    """What a C++ program with this main prints; integers wrap around as on the GPU."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "a.cpp", tmp_path / "a"
    src.write_text("""#include <cstdint>
#include <cstdio>
struct Dim { unsigned x, y; };
struct Args { int N, I, K, E, rows, out_cols; };
int main() {
  Dim blockIdx = {}, gridDim = {};
  Args p = {};
  (void)blockIdx; (void)gridDim; (void)p;
%s
}
""" % body)
    subprocess.run([cxx, "-O1", "-fwrapv", str(src), "-o", str(exe)], check=True,
                   capture_output=True, text=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True,
                          timeout=60).stdout


def assignments(names):
    return "\n".join("  %s = %s;" % kv for kv in names.items())


def run_loop(tmp_path, header, index, names, limit, turns):
    """Runs one of the kernels' loops on the CPU (its `for (...)` as it stands, with the given
    values for what it names): every index lies in [0, limit), and there are so many of them."""
    out = run_c(tmp_path, assignments(names) + """
  long long turns = 0;
  for (%s) {
    if ((long long)(%s) < 0 || (long long)(%s) >= %dLL) { std::puts("out of range"); return 0; }
    if (++turns > %dLL) { std::puts("does not end"); return 0; }
  }
  std::printf("%%lld", turns);""" % (header, index, index, limit, turns + 2))
    assert out.strip() == str(turns), (header, names, out)


def loops(text, containing):
    """What stands in the parentheses of the `for` loops that name `containing`."""
    found = []
    for m in re.finditer(r"\bfor \(", text):
        end, depth = m.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(text[end], 0)
            end += 1
        found.append(" ".join(text[m.end():end - 1].split()))
    return [h for h in found if containing in h]


@pytest.mark.parametrize("N", [0, 1, 4863, 2 ** 31 - 4864, 2 ** 31 - 4000, 2 ** 31 - 1])
def test_router_token_loops_stay_within_the_tokens(tmp_path, N):
    """Up to the largest number of tokens that is accepted, for the first and the last warp."""
    heads = loops(source("mp_route.cu"), "gridDim.x * kTeams")
    assert len(heads) == 2
    blocks, teams = 608, 8
    for header in heads:
        for block, team in ((0, 0), (blocks - 1, teams - 1)):
            at = block * teams + team
            run_loop(tmp_path, header, "n",
                     {"blockIdx.x": block, "gridDim.x": blocks, "p.N": N,
                      "const int kTeams": teams, "const int team": team},
                     N, max(0, -(-(N - at) // (blocks * teams))))


LONGEST = 2 ** 31 - 128


def statement(text, pattern):
    """The one statement that matches, as it stands."""
    found = set(" ".join(m.split()) for m in re.findall(pattern + r"[^;]*;", text))
    assert len(found) == 1, (pattern, found)
    return found.pop()


@pytest.mark.parametrize("I", [128, 512, 640, 2 ** 30, LONGEST - 1024, LONGEST])
def test_activation_channels_stay_within_the_row(tmp_path, I):
    """Up to the largest inner size that is accepted."""
    text = source("mp_swiglu.cu")
    forward, backward = text[:text.index("mp_k_swiglu_backward(")], text[
        text.index("mp_k_swiglu_backward("):]
    spans = statement(forward, r"const int spans = ")
    names = {"p.I": I, "const int kSpan": 512, "const int kCPL": 16}
    assert int(run_c(tmp_path, assignments(names) + """
  %s
  std::printf("%%d", spans);""" % spans)) == -(-I // 512)
    for host in re.findall(r"int64_t\(rows\) \* (\([^;]*\));", text):
        assert int(run_c(tmp_path, assignments(dict(names, **{"const int I": I})) + """
  std::printf("%%lld", (long long)(%s));""" % host)) == -(-I // 512)
    # the forward kernel's last span of a row: the lanes that have channels
    left = I - (-(-I // 512) - 1) * 512
    assert int(run_c(tmp_path, assignments(names) + """
  const int64_t row = 3;
  %s
  const int64_t unit = row * spans + spans - 1;
  int lanes = 0;
  for (int lane = 0; lane < 32; ++lane) {
    %s
    %s
    lanes += valid;
  }
  std::printf("%%d", lanes);""" % (spans, statement(forward, r"const (?:int|uint32_t) ch = "),
                                 statement(forward, r"const bool valid = ")))) == left // 16
    # the gradient's walk over a row
    heads = loops(backward, "WPR * kSpan")
    assert len(heads) == 1
    for warp in (0, 3):
        run_loop(tmp_path, heads[0], "c0",
                 dict(names, **{"const int warp": warp, "const int WPR": 4, "const bool live": 1}),
                 I, max(0, -(-(I - warp * 512) // 2048)))
    at = (I - 1) // 512 * 512
    assert int(run_c(tmp_path, assignments(dict(names, **{"const unsigned c0": at})) + """
  int lanes = 0;
  for (int lane = 0; lane < 32; ++lane) {
    %s
    %s
    lanes += valid;
  }
  std::printf("%%d", lanes);""" % (statement(backward, r"const (?:int|uint32_t) ch = "),
                                 statement(backward, r"const bool valid = ")))) == left // 16


@pytest.mark.skipif(torch.cuda.is_available(),
                    reason="fake-pointer argument checks run only on a host without a visible GPU")
@pytest.mark.parametrize("call", ["mp_expert_matmul_e4m3", "mp_expert_matmul_dgrad_e4m3",
                                  "mp_expert_matmul_wgrad_e4m3"])
@pytest.mark.parametrize("rows", [2 ** 31 - 1024, 2 ** 31 - 1])
def test_products_refuse_rows_whose_tiles_pass_32_bits(call, rows):
    _build.build()
    p = ctypes.c_void_p(0x10000)  # never dereferenced
    assert getattr(B.lib(), call)(1, rows, 128, 128, p, p, p, p, None, p, p,
                                  None) == B.MP_ERR_INVALID_ARG


@pytest.mark.parametrize("n", [128, 256, 272, 7168, 2 ** 31 - 384, 2 ** 31 - 256, 2 ** 31 - 128,
                               2 ** 31 - 16])
def test_products_column_tiles_of_the_largest_sizes(tmp_path, n):
    """The numbers of column tiles and of scale blocks, as the kernels and launchers work them
    out, for output channels up to the largest that are accepted."""
    helper = re.search(r"constexpr int ceil_div\(int a, int b\) (\{[^}]*\})",
                       source("mp_internal.h"))
    names = {"p.out_cols": n, "p.N": n, "p.K": n, "p.E": 1, "const int N": n, "const int K": n,
             "const int E": 1, "const int kBN": 256, "const int kWC": 128,
             "const int MP_SCALE_BLOCK": 128, "const int64_t row_tiles": 1}
    if helper:
        names["const auto ceil_div"] = "[](int a, int b) " + helper.group(1)

    def value(text, pattern, name):
        return int(run_c(tmp_path, assignments(names) + """
  %s
  std::printf("%%lld", (long long)%s);""" % (statement(text, pattern), name)))
    mm, wg = source("mp_expert_matmul.cu"), source("mp_expert_wgrad.cu")
    tiles = -(-n // 256)
    assert value(mm, r"const int ncol = ", "ncol") == tiles
    assert value(mm, r"const int64_t tiles = ", "tiles") == tiles
    assert value(mm, r"const int kb = ", "nb") == -(-n // 128)
    assert value(wg, r"const int kt = ", "kt") == tiles
    assert value(wg, r"const int kt = ", "nt") == tiles
