"""The handshake of the gated block's products on pairs of SMs (csrc/ffn_gemm.cu), on the CPU.

Model.  Each SM has a producer that waits for its own `empty` barrier of a stage and copies its share
of a step; the copies of both count on the leader's `full` barrier, which the leader's producer arms
with the bytes of both.  The leader's MMA warp waits for `full` and commits to both SMs' `empty`.  A
wait on a parity passes while the barrier's latest completed phase has it, so a producer that falls two
phases behind waits for ever.  Only its own copies, which the leader waits for, hold the leader back:
an SM without a copy in a step can fall behind by any number of steps."""

import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Barrier:
    def __init__(self):
        self.pending, self.bytes, self.completed = 1, 0, 0

    def _step(self):
        if self.pending == 0 and self.bytes == 0:
            self.pending, self.completed = 1, self.completed + 1

    def arrive(self, bytes_=0):
        assert self.pending == 1, "arrives twice in a phase"
        self.bytes += bytes_
        self.pending -= 1
        self._step()

    def land(self, bytes_):
        self.bytes -= bytes_
        self._step()

    def passes(self, parity):
        return ((self.completed - 1) & 1) == parity


def run(stages, tiles, slow, seed):
    """tiles: of each its steps and whether the second SM copies in them; slow: how seldom that SM's
    producer gets a turn.  The number of steps done; raises where nothing can go on."""
    rng = random.Random(seed)
    full = [Barrier() for _ in range(stages)]
    empty = [[Barrier() for _ in range(stages)] for _ in range(2)]
    steps = [copies for n, copies in tiles for _ in range(n)]
    holds = [[None] * stages, [None] * stages]  # the step whose data a stage has
    landing = []

    def producer(rank):
        for i, copies in enumerate(steps):
            s = i % stages
            while not empty[rank][s].passes(((i // stages) & 1) ^ 1):
                yield False
            if rank == 0:
                full[s].arrive(1 + copies)
            if rank == 0 or copies:
                landing.append((rank, s, i))
            yield True

    def mma():
        for i, copies in enumerate(steps):
            s = i % stages
            while not full[s].passes((i // stages) & 1):
                yield False
            assert holds[0][s] == i and (not copies or holds[1][s] == i), "another step's data"
            for rank in range(2):
                empty[rank][s].arrive()
            yield True
    roles = {"p0": producer(0), "p1": producer(1), "mma": mma()}
    stuck = set()  # the roles that wait, since anything last moved
    while roles:
        if not landing and stuck == set(roles):
            raise RuntimeError("nothing goes on")
        name = rng.choice(sorted(roles) + ["land"])
        if name == "p1" and rng.random() < slow:
            continue
        moved = False
        if name == "land":
            if landing:
                rank, s, i = landing.pop(rng.randrange(len(landing)))
                holds[rank][s] = i
                full[s].land(1)
                moved = True
        else:
            try:
                moved = next(roles[name])
                stuck.add(name)
            except StopIteration:
                del roles[name]
                moved = True
        if moved:
            stuck = set()
    return len(steps)


@pytest.mark.parametrize("stages", [5, 6, 8])
@pytest.mark.parametrize("slow", [0.0, 0.8, 0.99])
def test_both_sms_copy(stages, slow):
    for seed in range(20):
        assert run(stages, [(17, 1), (65, 1), (3, 1), (37, 1)], slow, seed) == 122


def test_an_sm_without_copies_falls_behind():
    """Why each SM has a share of every step: in a tile of more than two rounds of the ring an SM
    that copies nothing stalls on some schedule."""
    with pytest.raises(RuntimeError):
        for seed in range(20):
            run(6, [(17, 1), (65, 0), (37, 1)], 0.99, seed)


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_every_sm_has_a_share_of_every_step(tmp_path):
    exe = str(tmp_path / "ffn_tiles")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "quantized_moe_grouped_route_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "c", "ffn_tiles.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
