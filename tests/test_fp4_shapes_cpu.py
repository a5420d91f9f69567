"""Launches of the 4-bit products for few tokens, without a GPU: csrc/fp4_shape.h
over tokens, groups, rows and widths.  Two CTAs fit an SM wherever there are more
CTAs than SMs and none walks; shared and tensor memory hold every layout; the sums
that a cluster exchanges stay in their region."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "post_weight_quantization_accum_b200", "csrc")
SM_SMEM, CTA_RESERVED, CTA_SMEM, TMEM = 228 * 1024, 1024, 227 * 1024, 512  # of sm_100
SMS = 148

SHIM = """
#include "fp4_shape.h"
using namespace gptq;
// (raw taken or not, width, stages, splits, accs, raw stages, smem, apart, ring, tmem, tiles)
extern "C" void shape(int raw, int64_t tokens, int groups, int ragged, int64_t rows, int n, int sms, int64_t* r) {
  StreamShape s = {};
  r[0] = 1;
  if (raw) r[0] = raw_shape(tokens, groups, ragged, rows, n, sms, &s);
  else s = stream_shape(tokens, groups, ragged, rows, n, sms);
  r[1] = s.width; r[2] = s.stages; r[3] = s.splits; r[4] = s.accs; r[5] = s.raw_stages;
  if (r[0] == 0) return;
  r[6] = stream_smem(s, raw, groups); r[7] = stream_apart_bytes(s.width, s.splits);
  r[8] = int64_t(s.stages) * stream_stage_bytes(s.width, raw); r[9] = stream_tmem_cols(s.width, s.accs, s.stages);
  r[10] = stream_tiles(s, tokens, groups, ragged, rows);
}
"""


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    where = tmp_path_factory.mktemp("shape")
    src, so = where / "shim.cpp", where / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.shape.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                          ctypes.POINTER(ctypes.c_int64)]

    def call(raw, tokens, groups, ragged, rows, n):
        r = (ctypes.c_int64 * 11)()
        lib.shape(raw, tokens, groups, ragged, rows, n, SMS, r)
        return dict(zip(("taken", "width", "stages", "splits", "accs", "raw_stages", "smem", "apart", "ring", "tmem", "tiles"), r))
    return call


ROWS = [1, 128, 129, 640, 1024, 2048, 4096, 5120, 9216, 11008, 14336, 16384, 18944, 20000, 65536]
WIDTHS = [32, 256, 257, 512, 1000, 2048, 4096, 4097, 5120, 7168, 8192, 11008, 14336, 16384, 20000, 65535]


def _layers(raw):
    """Every call that reaches the kernel for few tokens (or, RAW, could)."""
    for rows in ROWS:
        for n in WIDTHS:
            for tokens in ([1, 2, 3, 4, 7, 8, 15, 16] if raw else [1, 2, 16, 17, 31, 32, 33, 48, 64, 65, 100, 128]):
                yield tokens, 1, 0, rows, n
            for groups in (1, 2, 8, 32, 60, 128, 350, 512):
                for tokens in ((1, 4, 8, 16) if raw else (1, 4, 16, 17, 64, 32 * groups)):
                    if tokens <= 32 * groups:
                        yield tokens, groups, 1, rows, n


@pytest.mark.parametrize("raw", [0, 1])
def test_layouts_fit_and_share_an_sm(shape, raw):
    seen, tight = set(), 0
    for layer in _layers(raw):
        s = shape(raw, *layer)
        if not s["taken"]:
            continue
        seen.add((s["splits"], s["raw_stages"]) if raw else (s["width"], s["splits"], s["accs"]))
        assert s["smem"] <= CTA_SMEM and s["tmem"] <= TMEM and 1 <= s["splits"] <= 8 and s["stages"] >= 2, (layer, s)
        if s["accs"] == 2:
            continue
        if s["tiles"] * s["splits"] > SMS:
            assert 2 * (s["smem"] + CTA_RESERVED) <= SM_SMEM and 2 * s["tmem"] <= TMEM, (layer, s)
            tight += s["stages"] == 3 and raw
    if raw:
        assert tight > 0 and max(r for _, r in seen) == 8 and {k for k, _ in seen} == {2, 3, 4, 6, 7, 8}
    else:
        assert {w for w, _, _ in seen} == {16, 32, 64, 128}


def test_few_tokens_keep_the_ring_where_a_cta_has_the_sm(shape):
    assert shape(1, 1, 1, 0, 4096, 4096)["stages"] == 4
    assert shape(1, 1, 1, 0, 2048, 14336)["stages"] == 4
    for rows, n in ((14336, 4096), (16384, 4096), (5120, 14336)):
        s = shape(1, 1, 1, 0, rows, n)
        assert (s["raw_stages"], s["stages"]) == (8, 3)


@pytest.mark.parametrize("raw", [0, 1])
def test_exchanged_sums_stay_in_their_region(shape, raw):
    """The rows of 128 floats that a cluster's CTAs write and read for every
    number of tokens: sent ones at rank * ceil(count / splits) + token / splits
    of the owner token % splits, the others at their token."""
    layouts = {}
    for layer in _layers(raw):
        s = shape(raw, *layer)
        if s["taken"] and s["splits"] > 1:
            layouts[s["width"], s["splits"], s["apart"] or s["ring"]] = s
    assert len(layouts) >= 6
    for (width, splits, region), s in layouts.items():
        for count in range(1, width + 1):
            if count <= 16:
                each = -(-count // splits)
                rows = [rank * each + token // splits for rank in range(splits) for token in range(count)]
                mine = [-(-(count - rank) // splits) for rank in range(splits)]
                rows += [p * each + j for p in range(splits) for m in mine for j in range(m)]
                # two sources' rows for one owner do not meet
                for owner in range(splits):
                    own = [rank * each + token // splits for rank in range(splits) for token in range(owner, count, splits)]
                    assert len(set(own)) == len(own) == mine[owner] * splits
            else:
                rows = range(count)
            assert (max(rows) + 1) * 512 <= region, (s, count)


def test_groups_take_tiles_of_64(shape):
    """Up to 32 tokens a group on average, which is as many as come here."""
    for groups in (1, 2, 8, 60, 512):
        for tokens in (1, groups, 16 * groups, 32 * groups):
            for rows, n in ((64, 64), (2048, 4096), (20000, 1000)):
                assert shape(0, tokens, groups, 1, rows, n)["width"] == 64
