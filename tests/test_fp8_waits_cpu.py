"""The 256 x 256 tiles of 8-bit products wait for a number of their own vector memory operations, counted by hand: all
but the newest n have ended.  What a wait is for has to have n operations behind it, so a load that the compiler moves or
leaves out makes the wait too short (one it adds only makes it longer).  This reads the compiled kernel's order:
per turn up to five loads of scales, then eight loads to LDS; a wait for all but four, eight, or those and the sixteen
stores of the item before; nothing else in between."""
import os
import re
import subprocess


def _events():
    from preconditioned_optimizer_matrix_amd import build
    r = subprocess.run([build.hipcc()] + build.COMMON + ["--cuda-device-only", "-S", os.path.join(build.CSRC, "pmx_fp8.hip"), "-o", "-"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    start = re.search(r"^\S*fp8_large_kernel\S*:", r.stdout, re.M).end()
    body = r.stdout[start:r.stdout.index(".section", start)]
    by_hand, out = False, []
    for line in body.splitlines():
        t = line.strip()
        if t.startswith((";;#ASMSTART", ";;#ASMEND")):
            by_hand = t.startswith(";;#ASMSTART")
        elif by_hand and t.startswith("s_waitcnt vmcnt"):
            out.append("wait" + re.search(r"vmcnt\((\d+)\)", t).group(1))
        elif t.startswith("buffer_load") and t.endswith(" lds"):
            out.append("lds")
        elif t.startswith("buffer_store_dwordx4"):
            out.append("store")
        elif re.match(r"(buffer|global|flat|scratch)_", t):
            out.append(t.split()[0])
    return out


def test_counted_waits_have_their_operations_behind_them():
    ev = _events()
    assert not [e for e in ev if e.startswith(("scratch", "flat"))]
    text = " ".join(ev) + " "
    scales, loads = "(?:global_load_dword ){5}", "(?:lds ){8}"
    # the group that waits for all of B: an item's first turn behind up to 16 stores, then the others
    assert len(re.findall("wait16 " + scales + loads + "wait0 " + scales + loads, text)) == 1
    # the other: half of A's loads may stay under way, then the turn's own eight, and 16 stores
    assert len(re.findall("wait20 " + scales + loads + "wait24 wait4 " + scales + loads + "wait8 ", text)) == 1
    # an item's results: 16 stores, four at a time, or of another number and then a wait for all
    assert ev.count("store") == 2 * 16 and ev.count("lds") == 14 + 4 * 8
