"""Host-side sizing of the loss head and of Muon (csrc/plan_xent.h, csrc/plan_muon.h), built
with g++ and checked on the CPU: the regions of the caller's workspace hold what the kernels
write and do not overlap, pieces and ranges cover the vocabulary once, grids and buffer
windows stay within their limits, and the tile choices agree with the products measured on
the card with each tile."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_layer_backward_bwd_amd", "csrc")
TILE = {0: (32, 128), 1: (64, 128), 2: (128, 128), 3: (256, 256), 4: (64, 64), 5: (64, 256)}
BOTH = {0: (0, 5), 1: (1, 5), 2: (2, 2), 3: (3, 3), 4: (4, 4), 5: (1, 2)}


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path_factory.mktemp("plan") / "plan_probe")
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "native", "plan_probe.cpp"), "-o", exe], check=True)

    def ask(lines):
        out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        return [list(map(int, l.split())) for l in out.stdout.strip().splitlines()]
    return ask


def up(x, m):
    return -(-x // m) * m


def log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def head_shapes():
    rng = random.Random(3)
    got = [(1, 1, 1), (1, 1, (1 << 22) - 1), (1, (1 << 22) - 1, 1), ((1 << 27) - 1, 1, 1), (16384, 4096, 131072),
           (1 << 20, 64, 1 << 20), (256, 4096, 50257), (257, 4096, 50257), (2559, 64, 50257), (2560, 64, 50257)]
    for _ in range(300):
        got.append((log_int(rng, 1, 1 << 17), log_int(rng, 1, 1 << 14), log_int(rng, 1, 1 << 18)))
    return got


def regions(offsets, sizes, total):
    """Each region inside the workspace, 256-byte aligned, none over another."""
    at = sorted((o, n) for o, n in zip(offsets, sizes) if n)
    for o, n in at:
        assert o % 256 == 0 and o + n <= total
    for (o, n), (p, _) in zip(at, at[1:]):
        assert o + n <= p


@pytest.mark.parametrize("pack", [0, 1])
def test_forward_plan(probe, pack):
    shapes = head_shapes()
    got = probe(["fwd %d %d %d %d" % (*s, pack) for s in shapes])
    need = probe(["bytes %d %d %d" % s for s in shapes])
    for (M, K, V), g, b in zip(shapes, got, need):
        rows, Kp, Vc, parts, join, ox, ow, op, orun, oz, osum, total = g
        ti, tj = TILE[rows]
        assert Kp >= K and Kp % 8 == 0 and Vc % 256 == 0 and Vc * -(-V // Vc) >= V
        assert parts == -(-Vc // tj) and join in (1, 2, 4, 8, 16, 32, 64)
        if M <= 32:
            assert join >= M                      # one block joins all rows and writes the mean
        regions((ox, ow, op, orun, oz, osum),
                (2 * M * Kp, 2 * K * Vc if pack else 0, 8 * M * parts, 8 * M, 4 * M, 16 * -(-M // join)), total)
        if not pack or M >= 2560:                 # what a call of any alignment may use
            assert total <= b[0]
        assert -(-M // ti) * parts < 1 << 31      # blocks


@pytest.mark.parametrize("pack", [0, 1])
def test_backward_plan(probe, pack):
    shapes = head_shapes()
    got = probe(["bwd %d %d %d %d" % (*s, pack) for s in shapes])
    need = probe(["bytes %d %d %d" % s for s in shapes])
    for (M, K, V), g, b in zip(shapes, got, need):
        rows, both, Kp, Vc, splits, length, acc, orow, ox, ow, og, oacc, total = g
        assert Vc % 256 == 0 and Vc * -(-V // Vc) >= V
        assert 1 <= splits <= 64 and length % 64 == 0
        assert splits * length >= Vc and (splits - 1) * length < Vc      # ranges cover a piece once
        assert acc == int(splits > 1 or Vc < V)
        regions((orow, ox, ow, og, oacc),
                (16 * M + 8, 2 * M * Kp, 2 * K * Vc if pack else 0, 2 * M * up(min(Vc, V), 64),
                 4 * M * Kp * splits if acc else 0), total)
        if not pack or M > 256:
            assert total <= b[1]
        if M <= 256:                              # these tiles read W at any alignment
            assert both != 3
        if both in (0, 1):                        # dW's whole reduction at once
            assert M <= 64
        assert 2 * M * Vc <= (512 << 20) or Vc == 256
        (xi, xj), (wi, wj) = TILE[BOTH[both][0]], TILE[BOTH[both][1]]
        blocks = splits * -(-M // xi) * -(-Kp // xj) + -(-K // wi) * -(-Vc // wj)
        assert blocks < 1 << 31


def test_buffer_windows():
    """A descriptor's window stays below 2^31 bytes at the largest widths accepted."""
    width = (1 << 22) - 1
    assert 2 * 256 * width < 1 << 31              # RC: 256 rows of W or G
    assert 2 * 64 * up(width, 64) < 1 << 31       # OC: 64 rows
    assert 2 * 256 * up((1 << 20) - 1, 64) < 1 << 31


def muon_shapes():
    rng = random.Random(4)
    got = [(1, 1, 1), (65535, 1, 1), (1, (1 << 20) - 1, 1), (1, 1, (1 << 20) - 1), (1, 64, 4096), (1, 65, 4096)]
    for _ in range(300):
        got.append((log_int(rng, 1, 200), log_int(rng, 1, 1 << 14), log_int(rng, 1, 1 << 14)))
    return got


def test_muon_plan(probe):
    shapes = muon_shapes()
    for (B, K, N), g in zip(shapes, probe(["muon %d %d %d" % s for s in shapes])):
        s, sp, Np, tall, parts, one, splits, x0, x1, oa, ob, op, osum, total = g
        assert s == min(K, N) and sp == up(s, 64) and Np == up(N, 64) and tall == int(K > N)
        assert 1 <= parts <= 1024 and one in (0, 64, 128) and 1 <= splits <= 16
        if s <= 64:
            assert one == 64
        assert not one or s <= one
        regions((x0, x1, oa, ob, op, osum),
                (2 * B * K * Np, 2 * B * K * Np, 2 * B * s * sp, 2 * B * s * sp, 8 * B * parts,
                 4 * B * splits * one * one if splits > 1 else 0), total)


def test_muon_grids(probe):
    rng = random.Random(5)
    cases = [(log_int(rng, 1, 65535), log_int(rng, 1, (1 << 20) - 1), log_int(rng, 1, (1 << 20) - 1)) for _ in range(300)]
    cases = [(b, i, j) for b, i, j in cases if b * i * j < 1 << 40]     # 2 TB of weights
    for (b, i, j), (tile, lower) in zip(cases, probe(["tile %d %d %d %d 0" % (*c, min(c[1:])) for c in cases])):
        T = {0: 256, 1: 128, 2: 128, 3: 64}[tile]
        assert not lower and b * -(-i // T) * -(-j // T) < 1 << 31


# products timed on the card with every tile (microseconds per launch: 256, 128, 128 deep, 64; of
# symmetric ones the full grid's and the lower tiles'): the choice is within a tenth of the fastest
@pytest.mark.parametrize("batch,I,J,R,full,lower", [
    (12, 1024, 1024, 1024, (30.0, 30.3, 35.2, 52.8), (33.6, 22.4, 26.2, 32.8)),
    (4, 1144, 1144, 3160, (63.9, 40.8, 50.2, 60.0), (65.2, 33.9, 28.0, 35.5)),
    (3, 515, 515, 2050, (43.5, 21.9, 17.5, 12.6), (48.0, 17.8, 18.7, 12.3)),
    (1, 2048, 2048, 8192, (143.0, 79.7, 73.0, 107.6), (148.3, 77.6, 58.6, 84.9)),
    (1, 4096, 4096, 4096, (101.3, 120.2, 141.5, 211.8), (89.4, 99.6, 104.0, 158.6)),
    (1, 4096, 4096, 12288, (280.2, 341.8, 382.6, 620.9), (221.5, 292.9, 277.3, 486.1)),
    (1, 256, 256, 256, (12.1, 7.5, 6.0, 4.5), (13.6, 6.7, 7.2, 4.9)),
    (1, 4096, 12288, 4096, (318.3, 384.6, 456.4, 668.1), None),
    (1, 2048, 8192, 2048, (61.5, 72.7, 93.7, 128.4), None),
    (4, 744, 800, 744, (26.2, 10.8, 11.6, 14.1), None),
    (8, 134, 395, 134, (14.4, 6.9, 7.1, 4.7), None),
    (2, 1248, 1720, 1248, (36.0, 22.8, 28.9, 29.0), None),
])
def test_muon_tile_choice_near_the_fastest_measured(probe, batch, I, J, R, full, lower):
    (tile, low), = probe(["tile %d %d %d %d %d" % (batch, I, J, R, lower is not None)])
    took = (lower if low else full)[tile]
    assert took <= 1.1 * min(full + (lower or ()))
