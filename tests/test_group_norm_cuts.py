"""CPU: how the group norm's calls are cut up: rules that every cut keeps (its workspace holds what its kernel
leaves, its CTAs are resident where they wait for one another), and the kernels that the GPU tests' sizes get."""

import ctypes
import json
import math
import os
import shutil
import subprocess

import pytest
import torch

import test_gpu_group_norm_clusters as clusters
import test_gpu_group_norm_layouts as layouts
import test_gpu_group_norm_no_numbers as no_numbers

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "adamw_optimizer_step_tensor_gb300", "csrc")
KINDS = ("lanes", "row", "small", "cluster", "fused")
SIZE = {torch.float32: 4, torch.float16: 2, torch.bfloat16: 2}


class Cut(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("kind", "piece", "tiles", "wide", "cluster", "part_rows", "parts", "batch", "aligned", "ctas")]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    inc = next((os.path.join(d, "include") for d in (os.environ.get("CUDA_HOME"), "/usr/local/cuda")
                if d and os.path.exists(os.path.join(d, "include", "cuda_runtime.h"))), None)
    if cxx is None or inc is None:
        pytest.skip("needs a host C++ compiler and the CUDA headers")
    so = str(tmp_path_factory.mktemp("host") / "cuts.so")
    subprocess.run([cxx, "-std=c++17", "-O2", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", inc,
                    os.path.join(CSRC, "group_norm_cut.cpp"), os.path.join(ROOT, "tests", "host", "group_norm_cuts.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    L.group_norm_cut.restype, L.group_norm_cut.argtypes = Cut, [ctypes.c_int64] * 2 + [ctypes.c_int] * 7
    L.group_norm_cluster_ns.restype, L.group_norm_cluster_ns.argtypes = ctypes.c_double, [ctypes.c_int64] * 2 + [ctypes.c_int] * 6
    L.group_norm_parts_ns.restype, L.group_norm_parts_ns.argtypes = ctypes.c_double, [ctypes.c_int64] * 2 + [ctypes.c_int] * 5
    L.group_norm_check.restype = ctypes.c_int64
    L.group_norm_check.argtypes = [ctypes.c_uint64, ctypes.c_int64, ctypes.POINTER(ctypes.c_int64), ctypes.c_char_p, ctypes.c_int]
    return L


def cut(lib, shape, groups, size, backward, layout=(0, 0, False)):
    return lib.group_norm_cut(*shape[:2], shape[2], groups, size, backward, *layout)


@pytest.mark.parametrize("seed", range(4))
def test_every_cut_keeps_the_rules(lib, seed):
    kinds, why = (ctypes.c_int64 * 5)(), ctypes.create_string_buffer(400)
    assert lib.group_norm_check(seed, 400_000, kinds, why, 400) == 0, why.value.decode()
    assert min(kinds) > 10_000                  # of every kernel


def test_sizes_of_the_layout_tests_reach_the_kernels_they_name(lib):
    for shape, groups, names in layouts.CASES:
        want = iter(names.split())
        for dtype, size in layouts.DTYPES.items():
            for backward in (0, 1):
                name = next(want)
                for layout in ((0, 0, False), layouts.LAYOUTS["padded"], layouts.LAYOUTS["swapped"], (8, 8, True)):
                    assert KINDS[cut(lib, shape, groups, size, backward, layout).kind] == name, (shape, dtype, backward, layout)
    # samples in parts: tiles of whole groups, a group over several tiles, several batches and one
    fused = [cut(lib, s, g, size, b) for s, g, _ in layouts.CASES for size in (2, 4) for b in (0, 1)]
    several = [(c.aligned, c.batch < s[0]) for (s, g, _), c in zip([x for x in layouts.CASES for _ in range(4)], fused) if c.kind == 4]
    assert set(several) == {(1, False), (0, False), (0, True), (1, True)}


def test_off_the_grid_a_piece_is_one_element(lib):
    for shape, groups, _ in layouts.SMALL:
        kinds = {KINDS[cut(lib, shape, groups, size, b, layouts.LAYOUTS[n]).kind] for size in (2, 4) for b in (0, 1) for n in ("odd", "shifted", "all")}
        assert kinds <= set(KINDS) and all(cut(lib, shape, groups, 2, b, layouts.LAYOUTS["all"]).piece == 1 for b in (0, 1))


def test_sizes_of_the_other_tests_reach_every_kernel(lib):
    kinds = {(KINDS[c.kind], b) for s, g in no_numbers.SHAPES for size in (2, 4) for b in (0, 1) for c in [cut(lib, s, g, size, b)]}
    assert kinds == {(k, b) for k in KINDS for b in (0, 1)}
    assert {cut(lib, s, g, size, 0).cluster for s, g in no_numbers.SHAPES for size in (2, 4)} >= {1, 2, 8}
    for dtype, shapes in clusters.SHAPES.items():
        got = {(c.cluster, c.piece, b) for s, g in shapes for b in (0, 1) for c in [cut(lib, s, g, SIZE[dtype], b)]}
        assert got >= {(n, p, b) for n in (2, 4, 8) for p in {torch.float32: (1, 4), torch.bfloat16: (1, 2, 8)}[dtype] for b in (0, 1)}


def measured():
    """The choices that were measured: (sizes, groups, bytes of an element, backward), us of the kernel for parts,
    and us of the clusters by (groups a tile, CTAs)."""
    with open(os.path.join(ROOT, "tests", "golden", "group_norm_cuts.json")) as f:
        for c in json.load(f)["calls"]:
            yield (tuple(c["sizes"]), c["groups"], {"f32": 4, "f16": 2, "bf16": 2}[c["type"]], int(c["direction"] == "bwd")), c["parts_us"], {
                tuple(map(int, k.split(","))): us for k, us in c["clusters_us"].items()}


def test_the_models_are_as_near_to_the_measured_choices_as_they_are_said_to_be(lib):
    off = []
    for (shape, groups, size, back), parts, choices in measured():
        for (m, ctas), us in choices.items():
            ns = lib.group_norm_cluster_ns(*shape[:2], shape[2], groups, size, back, m, ctas)
            assert ns > 0, (shape, m, ctas)
            off.append(math.log(ns / 1e3 / us))
        c = cut(lib, shape, groups, size, back)
        model = lib.group_norm_parts_ns(*shape[:2], shape[2], groups, size, back, c.batch) / 1e3
        assert 0.8 < model / parts < 3, (shape, model, parts)
        mine = parts if KINDS[c.kind] == "fused" else choices[c.wide * c.piece * groups // shape[2], c.cluster]
        most = 1.45 if (shape, back) == ((112, 3589, 58), 1) else 1.26
        assert mine <= most * min(parts, *choices.values()), (shape, mine)
    assert len(off) == 251 and math.sqrt(sum(x * x for x in off) / len(off)) < 0.26
