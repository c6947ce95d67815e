"""What the products of the feed-forward block launch for operands of any
alignment and stride, on the CPU: the library's host code over a stub launch.
Tiles that go straight to LDS need whole aligned units, 32-bit offsets over a
tile and, for the gradient of the input, one stride for both summed operands;
every operand that is not so has to be copied to the workspace first, where the
copies and the parts of split tiles have to fit."""
import itertools
import os
import subprocess

import pytest

from sharded_optimizer_step_amd import _build

HERE = os.path.dirname(os.path.abspath(__file__))
FORWARD, INPUT, WEIGHT = 0, 1, 2
FAR = 1 << 22  # the longest stride whose offsets over 256 rows stay under 2^31


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("launch")
    flags = [f for f in _build.HIPCC_FLAGS if f.startswith(("-std", "--offload", "-ffp"))]
    cmd = ["hipcc", "-O1", *flags, "-Wno-everything", "--cuda-host-only", "-I", os.path.join(_build.ROOT, "include"), "-I", _build.CSRC,
           "-c", "-o", str(d / "host.o"), os.path.join(HERE, "ffn_launch_host.hip")]
    for c in (cmd, ["g++", "-no-pie", "-o", str(d / "host"), str(d / "host.o"), "-Wl,--unresolved-symbols=ignore-all"]):
        r = subprocess.run(c, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]

    def run(kind, outputs, rows, cols, hidden, operands):
        """(workspace address, its size, copies, (direct, [(address, ld)] of d, d, h, w, w, where the parts begin))"""
        args = [kind, outputs, rows, cols, hidden, *itertools.chain(*operands)]
        r = subprocess.run([str(d / "host"), *map(str, args)], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, (args, r.returncode, r.stderr)
        lines = [line.split() for line in r.stdout.splitlines()]
        space, size = map(int, lines[0][1:])
        copies, product = [], None
        for what, *v in lines[1:]:
            v = list(map(int, v))
            if what == "copy":
                copies += [v[i:i + 5] for i in range(0, len(v), 5)]
            else:
                assert product is None
                product = what == "direct", [tuple(v[i:i + 2]) for i in range(0, 10, 2)], v[10]
        assert product is not None
        return space, size, copies, product

    return run


def whole(n):
    return (n + 7) // 8 * 8


def used(kind, outputs):
    """The operands that a product reads, among d, d, h, w, w."""
    return {FORWARD: [2, 3, 4], INPUT: [0, 1, 3, 4], WEIGHT: [0, 1, 2] if outputs == 2 else [0, 2]}[kind]


def check(host, kind, outputs, rows, cols, hidden, operands):
    where = (kind, outputs, rows, cols, hidden, operands)
    space, size, copies, (direct, factors, parts) = host(kind, outputs, rows, cols, hidden, operands)
    assert space <= parts <= space + size, where
    held = {}
    end = space
    for address, ld, r, c, to in sorted(copies, key=lambda v: v[4]):
        assert to % 16 == 0 and to >= end, where
        end = to + r * whole(c) * 2
        held[to] = address, ld, r, c
    assert end <= parts, where
    shapes = [(rows, hidden)] * 2 + [(rows, cols)] + [(hidden, cols)] * 2
    for i in used(kind, outputs):
        at, ld = factors[i]
        if at in held:
            assert held[at] == (*operands[i], *shapes[i]) and ld == whole(shapes[i][1]), (where, i)
        else:
            assert (at, ld) == operands[i], (where, i)
            assert not direct or shapes[i][1] % 8 == 0, (where, i)
        if direct:
            assert at % 16 == 0 and ld % 8 == 0 and ld <= FAR, (where, i)
    if direct and kind == INPUT:
        assert factors[0][1] == factors[1][1] and factors[3][1] == factors[4][1], where
    return direct, copies


# columns that are a multiple of 8 or not, of one operand, both or none
SIZES = [(300, 767, 520), (2011, 1003, 2736), (900, 1003, 1024), (2011, 1000, 2731), (2011, 1024, 2731), (8192, 4096, 11003), (640, 767, 1001),
         (300, 264, 520), (16, 1003, 2731), (5, 7, 9), (64, 4091, 11003), (700, 8, 11)]
PLACES = [(0, 0), (0, 8), (0, 16), (0, 3), (2, 0), (2, 8), (0, FAR), (0, 8 * FAR)]  # address, columns more than there are


@pytest.mark.parametrize("kind,outputs", [(FORWARD, 1), (INPUT, 1), (WEIGHT, 1), (WEIGHT, 2)])
@pytest.mark.parametrize("rows,cols,hidden", SIZES)
def test_factors_are_what_their_tiles_take(host, kind, outputs, rows, cols, hidden):
    widths = [hidden, hidden, cols, cols, cols]
    base = [((i + 1) << 44, whole(w)) for i, w in enumerate(widths)]
    for a, b in ((0, 1), (2, 2), (3, 4)):
        if a not in used(kind, outputs):
            continue
        for p, q in itertools.product(PLACES, PLACES):
            operands = list(base)
            operands[a] = base[a][0] + p[0], base[a][1] + p[1]
            if b != a:
                operands[b] = base[b][0] + q[0], base[b][1] + q[1]
            check(host, kind, outputs, rows, cols, hidden, operands)


@pytest.mark.parametrize("rows,cols,hidden,stay", [(300, 767, 520, [0, 1]), (2011, 1024, 2731, [3, 4])])
def test_operands_that_their_tiles_take_stay_where_they_are(host, rows, cols, hidden, stay):
    """A pair of whole aligned units and one stride is not copied; one whose strides differ is, both of it."""
    operands = [((i + 1) << 44, whole(w) + 64) for i, w in enumerate([hidden, hidden, cols, cols, cols])]
    direct, copies = check(host, INPUT, 1, rows, cols, hidden, operands)
    assert direct and {c[0] for c in copies} == {operands[i][0] for i in {0, 1, 3, 4} - set(stay)}
    operands[stay[1]] = operands[stay[1]][0], operands[stay[1]][1] + 8
    direct, copies = check(host, INPUT, 1, rows, cols, hidden, operands)
    assert direct and {c[0] for c in copies} == {operands[i][0] for i in (0, 1, 3, 4)}
