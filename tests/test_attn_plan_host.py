"""Host side of the attention over the 4-bit cache: which sizes a call takes, and which
launch (CPU only)."""
import ctypes
import os
import random
import subprocess

import pytest

from attn_forms import FORMS, sizes

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "ternary_weight_i2_amd", "csrc")
SHIM = """#include "attn_plan.h"
extern "C" void plan(const int64_t *a, int bf16, int64_t *out) {
    const bitnet::Attn4Plan p = bitnet::attn4_plan(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], bf16);
    const int64_t r[] = {p.prompt, p.wide, p.splits, p.per_cu, p.tiles, p.workgroups};
    for (int i = 0; i < 6; ++i) out[i] = r[i];
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    (at / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(at / "shim.cpp"),
                    "-o", str(at / "shim.so")], check=True)
    f = ctypes.CDLL(str(at / "shim.so")).plan

    def call(args, bf16):
        out = (ctypes.c_int64 * 6)()
        f((ctypes.c_int64 * 8)(*args), int(bf16), out)
        return dict(zip(("prompt", "wide", "splits", "per_cu", "tiles", "workgroups"), out))
    return call


@pytest.fixture(scope="module")
def L():
    from ternary_weight_i2_amd import _binding
    return _binding.load()


def test_workspace_query_refuses_what_the_call_refuses(L):
    w = L.bitnet_attn_kv4_workspace
    assert w(1 << 20, 1 << 20, 16, 16, 64, 64, 0, 0) == -1
    assert "too many" in L.bitnet_last_error().decode()
    assert w(1, 1 << 21, 128, 128, 256, 64, 0, 0) == -1
    # below the stated limit every call is taken, however long its histories: splits are
    # given up first
    assert w(1 << 20, 1, 8, 8, 64, 1 << 30, 0, 0) == 0
    assert w((1 << 20) - 1, 1, 15, 15, 256, 1 << 30, 0, 0) == 0
    rng = random.Random(1)
    for _ in range(3000):
        kv = rng.choice([1, 2, 5, 8, 16, 100])
        heads = kv * rng.choice([1, 2, 4, 8])
        n_seqs, n = (int(2 ** rng.uniform(0, 20.5)) for _ in range(2))
        sizes = (min(n_seqs, 1 << 20), n, heads, kv, rng.choice([64, 128, 256]),
                 64 * int(2 ** rng.uniform(0, 24)), rng.choice([0, 1000]), 4)
        if n * heads // 16 + sizes[0] * kv < 1 << 24:
            assert w(*sizes) >= 0, sizes


@pytest.mark.parametrize("form", FORMS)
def test_every_form_is_reached_by_its_sizes(plan, form):
    f = FORMS[form]
    for dim in f["dims"]:
        for window in (False, True):
            for bf16 in (False, True):
                p = plan(sizes(f, dim, window), bf16)
                assert (p["prompt"], p["wide"], p["splits"] > 1) == f["plan"], (dim, window, bf16, p)


def test_plan_has_room_for_every_row_and_the_query_for_its_splits(L, plan):
    rng = random.Random(2)
    for _ in range(3000):
        kv = rng.choice([1, 2, 5, 8])
        heads = kv * rng.choice([1, 2, 4, 8])
        n_seqs, n = int(2 ** rng.uniform(0, 12)), int(2 ** rng.uniform(0, 13))
        a = (n_seqs, n, heads, kv, rng.choice([64, 128, 256]), int(2 ** rng.uniform(0, 20)),
             rng.choice([0, 500]), rng.choice([0, 4]))
        rows, most = n * heads // kv, 1
        for bf16 in (False, True):
            p = plan(a, bf16)
            high = 32 if p["prompt"] else 16
            # the last tile that a sequence's rows can reach, and all of them launched
            assert p["tiles"] >= rows // high + n_seqs
            assert p["workgroups"] * max(p["prompt"], 1) == p["tiles"] * kv * p["splits"]
            assert p["splits"] == 1 or not (p["prompt"] or p["wide"])
            most = max(most, p["splits"])
        assert L.bitnet_attn_kv4_workspace(*a) == (most * n * heads * (a[4] + 4) * 4 if most > 1 else 0)
