"""The waits in the products of the mixture-of-experts layer, in the code that the compiler made of
them. A wave keeps a ring of steps on their way from HBM to LDS and, before it reads one, waits until
no more loads than the later steps' are out. That is right only if each of those steps has as many
loads as the source counts: a load whose result the compiler can show to be unused is not issued, and
the wait then ends before what is to be read has arrived. On a GPU such a read gives an earlier
step's codes only now and then; here every wait of every kernel is counted."""
import re
import subprocess

import pytest

from microscaling_precision_quantization_amd import build

DEPTH = 4  # steps of the ring: one that is read, the others on their way


def parse(text):
    """name -> "L" (a buffer load) and ints (the counts of the source's own waits) in order, of each product."""
    parts = re.split(r"^(_ZN2mx\S*moe_(?:up|down)_kernel\S*):.*$", text, flags=re.M)
    out = {}
    for name, body in zip(parts[1::2], parts[2::2]):
        body = re.split(r"^\s*\.section", body, flags=re.M)[0]
        ops, own = [], False
        for line in map(str.strip, body.splitlines()):
            if "#ASMSTART" in line or "#ASMEND" in line:
                own = "START" in line
            elif line.startswith("buffer_load"):
                ops.append("L")
            elif own and (m := re.match(r"s_waitcnt vmcnt\((\d+)\)", line)):
                ops.append(int(m.group(1)))
        out[name] = ops
    return out


def places(ops):
    """(loads, wait) of each place of the unrolled group of tiles: what it loads, then waits for. From the
    wait for the first steps of all to the last wait that leaves loads out."""
    waits = [i for i, o in enumerate(ops) if o != "L" and o > 0]
    first = max(i for i in range(waits[0]) if ops[i] == 0)
    out, loads = [], 0
    for o in ops[first + 1:waits[-1] + 1]:
        if o == "L":
            loads += 1
        else:
            out.append((loads, o))
            loads = 0
    return out


def early(group, runs_on):
    """Places whose wait may end before their next step has arrived. Place k loads step k + DEPTH - 1 and
    then needs step k + 1. runs_on: the first places of a group follow the last ones of the one before;
    else every load is waited for in between. (The compiler's own waits, and other accesses that are out
    as well, can only make a wait longer.)"""
    bad, out = [], []  # out: the step of each load on its way, the oldest first
    for k in range(len(group) * (2 if runs_on else 1)):
        loads, wait = group[k % len(group)]
        out += [k + DEPTH - 1] * loads
        out = out[max(0, len(out) - wait):]
        if any(step <= k + 1 for step in out):
            bad.append(k)
    return bad


def test_the_count_itself():
    three = [(3, 6)] * 16
    assert early(three, True) == [] and early(three, False) == []
    assert early([(2, 6)] * 16, True)[0] == 2           # fewer loads than are counted
    assert early(three[:-1] + [(2, 6)], True) != []      # ... in the last place alone: seen by the next group
    assert early(three[:13] + [(2, 6)] * 3, False) == [13, 14, 15]
    assert early(three[:13] + [(0, 3), (0, 0)], False) == []
    assert parse("_ZN2mx13moe_up_kernelX:\n buffer_load_dword v0 lds\n ;;#ASMSTART\n s_waitcnt vmcnt(6)\n ;;#ASMEND\n"
                 " s_waitcnt vmcnt(1)\n .section x\n buffer_load_dword") == {"_ZN2mx13moe_up_kernelX": ["L", 6]}
    assert places(["L", 0, "L", "L", 0, "L", 1, "L", "L", 2, 0, "L"]) == [(1, 1), (2, 2)]


@pytest.fixture(scope="module")
def products(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("moe") / "moe.s")
    flags = [f for f in build.COMMON if f != "-fPIC"] + build.EXTRA["moe.hip"]
    r = subprocess.run([build.HIPCC, *flags, "-x", "hip", "--offload-device-only", "-S", f"{build.CSRC}/moe.hip", "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    with open(out) as f:
        return parse(f.read())


def test_every_wait_covers_what_is_read_next(products):
    assert len(products) >= 30
    bad = {}
    for name, ops in products.items():
        steps, several = re.search(r"kernelILi\d+ELb[01]ELi(\d)ELb([01])", name).groups()
        group = places(ops)
        tiles = 4 if steps == "4" else 8
        assert len(group) >= tiles * int(steps) - DEPTH, name  # (the unrolled group, once)
        # Rows of several rounds of loads: each round ends with none out.
        bad[name] = early(group, runs_on=several == "0")
    assert not any(bad.values()), {n: b for n, b in bad.items() if b}
