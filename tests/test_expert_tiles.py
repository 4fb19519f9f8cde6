"""The experts' table of tiles: counts at the largest sizes, groups that overlap,
and more experts than a block has threads."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from row_wise_softmax_warp_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))
MOST = 1 << 30  # tiles


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("tile_probe") / "tile_probe.so")
    subprocess.run([build._nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-I", build.CSRC, "-shared", "-o", out,
                    os.path.join(HERE, "csrc", "tile_probe.cu")], check=True, capture_output=True)
    lib = ctypes.CDLL(out)
    lib.host_tiles_of.restype = ctypes.c_uint
    lib.host_cut_tiles.argtypes = [ctypes.c_uint]
    lib.run_tile_probe.argtypes = [ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                   ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]
    return lib


def alternating(experts, slots):
    """Offsets 0, slots, 0, slots, ...: half of the groups have all rows."""
    return np.where(np.arange(experts + 1) % 2, slots, 0).astype(np.int32)


def counts_of(offsets, slots):
    lo = np.clip(offsets[:-1].astype(np.int64), 0, slots)
    return lo, np.maximum(np.clip(offsets[1:].astype(np.int64), 0, slots), lo) - lo


def test_counts_stay_in_range(probe):
    """Every sum of tiles that 1024 experts can reach, however their groups overlap."""
    assert [probe.host_tiles_of(n, 256) for n in (0, 1, 256, 257, 1 << 30)] == [0, 1, 1, 2, 1 << 22]
    for slots in (1 << 29, (1 << 30) - 255, 1 << 30):
        _, counts = counts_of(alternating(1024, slots), slots)
        tiles = sum(probe.host_tiles_of(int(c), 256) for c in counts)
        assert tiles < 1 << 32  # the unsigned sum does not wrap
        row_tiles = probe.host_cut_tiles(tiles)
        assert row_tiles == min(tiles, MOST)
        for across in (1, 2, 3, 1 << 23):  # (2^31 - 1) / 256 columns of tiles at most
            every = probe.host_all_tiles(row_tiles, across)
            assert every == min(row_tiles * across, MOST)
            assert 0 < every + 4096 < 1 << 31  # the last tile's number plus a grid
    assert probe.host_all_tiles(0, 1 << 23) == 0 and probe.host_all_tiles(5, 7) == 35


def run(probe, threads, offsets, slots, asked):
    experts = len(offsets) - 1
    at, want = torch.from_numpy(offsets).cuda(), torch.from_numpy(np.asarray(asked, np.int32)).cuda()
    table = torch.full((experts + 1,), -7, dtype=torch.int32, device="cuda")
    out = torch.full((len(asked), 3), -7, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert probe.run_tile_probe(threads, at.data_ptr(), experts, slots, table.data_ptr(), want.data_ptr(), len(asked),
                                out.data_ptr()) == 0
    return table.cpu().numpy(), out.cpu().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("threads", [224, 384])
@pytest.mark.parametrize("slots", [1 << 20, 1 << 29, 1 << 30])
@pytest.mark.parametrize("experts", [2, 7, 1023, 1024])
def test_overlapping_groups(probe, experts, slots, threads):
    offsets = alternating(experts, slots)
    asked = np.unique(np.linspace(0, min(MOST, (experts + 1) // 2 * (slots // 256)) - 1, 200).astype(np.int64))
    table, out = run(probe, threads, offsets, slots, asked)
    _, counts = counts_of(offsets, slots)
    want = np.minimum(np.concatenate([[0], np.cumsum(-(-counts // 256))]), MOST)
    assert (table == want).all()
    expert, first, count = out.T.astype(np.int64)
    assert (expert == np.searchsorted(want[1:], asked, side="right")).all()
    assert (first == (asked - want[expert]) * 256).all() and (count == 256).all() and (first + 256 <= slots).all()


@pytest.mark.gpu
@pytest.mark.parametrize("threads", [224, 384])
@pytest.mark.parametrize("experts", [1, 224, 225, 385, 449, 770, 1024])
def test_tiles_cover_the_groups(probe, experts, threads):
    """Runs of up to five experts a thread: every row of every group in one tile of at most 256."""
    rng = np.random.default_rng(experts)
    sizes = rng.choice([0, 0, 1, 31, 255, 256, 257, 513, 1793], experts)
    sizes[-1] = 3
    offsets = np.cumsum([5, *sizes]).astype(np.int32)  # five rows before the first group
    tiles = int((-(-sizes // 256)).sum())
    table, out = run(probe, threads, offsets, int(offsets[-1]) + 9, np.arange(tiles))
    assert table[-1] == tiles
    seen = np.zeros(int(offsets[-1]) + 9, np.int64)
    for expert, first, count in out:
        assert 0 < count <= 256 and offsets[expert] <= first and first + count <= offsets[expert + 1]
        seen[first:first + count] += 1
    assert (seen[5:offsets[-1]] == 1).all() and seen[:5].sum() == 0 and seen[offsets[-1]:].sum() == 0
