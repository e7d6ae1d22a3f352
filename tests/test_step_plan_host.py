"""Host side of the operators around a decode step: which launches a call takes, over the range
of its sizes (CPU only)."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "ternary_weight_i2_amd", "csrc")
SHIM = """#include "attn_plan.h"
#include "w4_plan.h"
extern "C" void w4(const int64_t *a, int64_t *r) {
    const bitnet::W4Plan p = bitnet::w4_plan(a[0], a[1], a[2]);
    const int64_t v[] = {p.tt, p.rt, p.wk, p.rows, p.tokens, p.shares};
    for (int i = 0; i < 6; ++i) r[i] = v[i];
}
extern "C" void weigh(const int64_t *a, int64_t *r) {
    const bitnet::WeighPlan p = bitnet::weigh_plan(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8]);
    const int64_t v[] = {p.tiles, p.splits, p.chunks, p.many, p.parts, p.kept_at, p.sums_at, p.bytes};
    for (int i = 0; i < 8; ++i) r[i] = v[i];
}
extern "C" void evict(const int64_t *a, int64_t *r) {
    const bitnet::EvictPlan p = bitnet::evict_plan(a[0], a[1], a[2]);
    const int64_t v[] = {p.slices, p.search_at, p.slices_at, p.bytes};
    for (int i = 0; i < 4; ++i) r[i] = v[i];
}
extern "C" void slice(const int64_t *a, int64_t *r) {
    const bitnet::EvictSlice s = bitnet::evict_slice((int)a[0], (int)a[1], (int)a[2]);
    r[0] = s.from;
    r[1] = s.to;
}
extern "C" void tile(const int64_t *a, int64_t *r) {
    r[0] = bitnet::first_tile<16, 1>((int)a[0], (uint32_t)a[1], (int)a[2]);
    r[1] = bitnet::first_tile<4, 2>((int)a[0], 1, (int)a[2]);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    (at / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(at / "shim.cpp"),
                    "-o", str(at / "shim.so")], check=True)
    lib = ctypes.CDLL(str(at / "shim.so"))

    def call(name, *args):
        names = {"w4": "tt rt wk rows tokens shares", "weigh": "tiles splits chunks many parts kept_at sums_at bytes",
                 "evict": "slices search_at slices_at bytes", "slice": "from to", "tile": "rows16 block4"}[name].split()
        out = (ctypes.c_int64 * len(names))()
        getattr(lib, name)((ctypes.c_int64 * len(args))(*args), out)
        return dict(zip(names, out))
    return call


def spread(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def test_products_are_covered_whole(plan):
    """Every row and token has a workgroup, every share a block, and there is no launch beyond
    what the hardware takes; few rows do not leave one wave alone with many blocks."""
    rng, forms = random.Random(1), set()
    for i in range(4000):
        N = rng.choice([1, 2, 16, 17, 32, 33, 64, 65, 2 ** 21, spread(rng, 1, 2 ** 21)])
        M = rng.choice([1, 15, 16, 17, 2 ** 24, spread(rng, 1, 2 ** 24)])
        K = 128 * rng.choice([1, 2, 256, spread(rng, 1, 256)])
        p = plan("w4", N, M, K)
        tiles, blocks = -(-M // 16), K // 128
        assert p["tt"] in (1, 2, 4) and p["rt"] in (1, 2) and p["wk"] in (1, 2, 4)
        assert p["wk"] == 1 or (p["tt"] == 1 and p["rt"] == 1)
        assert (p["tt"] == 1) == (N <= 16) and p["rt"] == 1 or p["tt"] > 1
        assert p["tokens"] * 16 * p["tt"] >= N > (p["tokens"] - 1) * 16 * p["tt"]
        per = 8 * p["rt"] // p["wk"]
        assert p["rows"] * per >= tiles > (p["rows"] - 1) * per
        assert 1 <= p["shares"] <= min(blocks, 32) and p["wk"] <= blocks
        assert p["rows"] * 512 < 2 ** 32 and p["tokens"] < 2 ** 16 and p["shares"] < 2 ** 16
        if tiles < 64 and N <= 16:
            assert p["shares"] * p["wk"] >= min(blocks // 8, 16)
        forms.add((p["tt"], p["rt"], p["wk"], p["shares"] > 1))
    assert len(forms) >= 12


def test_weights_of_tokens_have_room(plan):
    """Shares, parts and the workspace's three areas, over sizes from one token to the largest."""
    rng, forms = random.Random(2), set()
    for i in range(4000):
        seqs = rng.choice([1, 1, spread(rng, 1, 2 ** 20)])
        N = rng.choice([seqs if seqs <= 2 ** 21 else 1, spread(rng, 1, 2 ** 21)])
        kv = rng.choice([1, 5, 8, 1024])
        heads = kv * rng.choice([x for x in (1, 4, 8, 128) if kv * x <= 1024])
        dim, window = rng.choice([64, 128, 256]), rng.choice([0, 0, spread(rng, 1, 2 ** 30)])
        sinks, bf16 = rng.choice([0, 4, 1000]), rng.randrange(2)
        max_kv = rng.choice([0, 1, 64, 65, spread(rng, 1, 2 ** 30)])
        p = plan("weigh", seqs, N, heads, kv, dim, max_kv, window, sinks, bf16)
        rows, pages = N * (heads // kv), max(-(-max_kv // 64), 1)
        assert p["tiles"] == rows // 16 + seqs
        assert 1 <= p["splits"] <= 128 and 1 <= p["chunks"] <= pages and 1 <= p["parts"] <= 2048
        assert p["splits"] == 1 or p["splits"] * p["tiles"] * kv <= 2 ** 22
        assert p["chunks"] == 1 or p["chunks"] * seqs * kv <= 2 ** 22
        assert p["parts"] == 1 or (p["many"] and p["parts"] * p["chunks"] * seqs * kv <= 2048)
        assert p["kept_at"] % 16 == 0 and p["sums_at"] % 16 == 0
        assert p["kept_at"] >= p["splits"] * N * heads * 8
        per = {64: 2, 128: 4, 256: 8}[dim] * (1 if bf16 else 2) + (2 if dim == 256 else 1)
        assert p["sums_at"] - p["kept_at"] == (p["tiles"] * kv * per * 1024 if p["many"] else 0)
        assert p["bytes"] - p["sums_at"] == (seqs * p["chunks"] * kv * p["parts"] * 256 if p["parts"] > 1 else 0)
        forms.add((p["many"], p["parts"] > 1, p["splits"] > 1))
        # fp32's workspace serves both types
        assert plan("weigh", seqs, N, heads, kv, dim, max_kv, window, sinks, 0)["bytes"] >= p["bytes"]
    assert len(forms) >= 5


def test_tiles_lie_where_the_second_launch_looks_for_them():
    """The tiles of a sequence begin at begin * G / 16 + its number and are none of another's."""
    rng = random.Random(3)
    for i in range(300):
        G, new = rng.choice([1, 3, 4, 8]), [rng.choice([0, 1, 2, 30, 100]) for _ in range(rng.randint(1, 20))]
        start, taken = 0, []
        for b, n in enumerate(new):
            taken += [start * G // 16 + b + r for r in range(-(-n * G // 16))]
            start += n
        assert len(set(taken)) == len(taken) and (not taken or max(taken) < start * G // 16 + len(new))


def test_long_histories_are_chosen_from_by_several(plan):
    rng = random.Random(4)
    for i in range(2000):
        seqs, kv = spread(rng, 1, 2 ** 20), rng.choice([1, 5, 8, 1024])
        pages = rng.choice([1, 319, 320, spread(rng, 1, 2 ** 24)])
        p = plan("evict", seqs, kv, pages)
        assert 1 <= p["slices"] <= 32
        if p["slices"] == 1:
            assert p["bytes"] == 0
        else:
            assert pages >= 320 and p["slices"] * seqs * kv <= 512
            assert p["search_at"] == 3 * seqs * kv * p["slices"] * 8192
            assert p["slices_at"] == p["search_at"] + 3 * seqs * kv * 8
            assert p["bytes"] == p["slices_at"] + seqs * kv * p["slices"] * 8
    assert plan("evict", 1, 5, 2048)["slices"] > 8


def test_slices_of_a_history_load_inside_a_page(plan):
    """Every token is in one slice, and the four weights that each of a slice's threads loads at
    once lie in one page and on 16 bytes, also where the slice has no token."""
    rng = random.Random(5)
    helds = list(range(0, 400)) + [spread(rng, 400, 2 ** 30) for _ in range(300)] + [2 ** 30 - i for i in range(4)]
    for held in helds:
        for slices in (range(2, 17) if held < 400 else (rng.randint(2, 16), 16)):
            at = 0
            for k in range(slices):
                s = plan("slice", held, slices, k)
                assert s["from"] % 4 == 0, (held, slices, k)
                for t in (s["from"], s["from"] + 4 * 1023, s["from"] + 4 * 1024 * 7 + 60):
                    assert t % 64 + 4 <= 64 and t < 2 ** 31
                if s["from"] < s["to"]:
                    assert s["from"] == at and s["to"] <= held
                    at = s["to"]
                else:
                    assert s["from"] >= held
            assert at == held


def test_forms_of_a_product_go_by_the_tokens(plan):
    """The kernels of up to 16 tokens are those that the planner means, and so are the others."""
    rng = random.Random(6)
    for i in range(4000):
        N, M = rng.choice([1, 4, 16, 17, 32, 33, spread(rng, 1, 2 ** 21)]), spread(rng, 1, 2 ** 24)
        p = plan("w4", N, M, 128 * spread(rng, 1, 256))
        assert p["tt"] == (1 if N <= 16 else 2 if N <= 32 else 4)
        assert p["rt"] == 1 if N <= 16 else p["wk"] == 1


def test_a_history_has_sixteen_workgroups_at_most(plan):
    rng = random.Random(7)
    for i in range(2000):
        p = plan("evict", spread(rng, 1, 2 ** 20), rng.choice([1, 5, 8, 1024]), spread(rng, 1, 2 ** 24))
        assert 1 <= p["slices"] <= 16


def test_first_tiles_leave_each_sequence_its_own(plan):
    """Where the launches look for a sequence's tiles of 16 rows, or blocks of four positions, is
    another's place for none of them, and none lies behind those that the planner counts."""
    rng = random.Random(8)
    for i in range(300):
        G, new = rng.choice([1, 3, 4, 8]), [rng.choice([0, 1, 2, 30, 100]) for _ in range(rng.randint(1, 20))]
        start, tiles, blocks = 0, [], []
        for b, n in enumerate(new):
            at = plan("tile", start, G, b)
            tiles += [at["rows16"] + r for r in range(-(-n * G // 16))]
            # from any place in a page on, n positions touch up to (n + 3) // 4 + 1 blocks of four
            blocks += [at["block4"] + r for r in range((n + 3 + 3) // 4 if n else 0)]
            start += n
        for taken in (tiles, blocks):
            assert len(set(taken)) == len(taken)
        if start:
            assert max(tiles) < plan("weigh", len(new), start, G, 1, 64, 4096, 0, 0, 1)["tiles"]
            assert max(blocks) < start // 4 + 2 * len(new)
