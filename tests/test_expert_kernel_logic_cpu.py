"""Logic of the expert layer's kernels that can be followed without a GPU, taken from their
source: the hand-over of shared-memory slots between warps."""
import os
import re

from combine_mp_layout_gb300 import _build


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
