"""Which way attention's work is cut (host sizes only, no GPU): the plan itself is asked, through a few
lines of C++ linked against the library."""
import ctypes
import os
import subprocess

import pytest

from fp4_sparse_attention_gb300 import build

SMS = 152
ASK = r"""
#include <cstring>
#include "attention.h"
extern "C" int ask(int latent, int listed, int seqs, int rows, int heads, int kv_heads, int max_q, int max_k, int sms, int* out) {
  fp4idx::AttnParams p;
  std::memset(&p, 0, sizeof(p));
  static const uint16_t v = 0;
  static const int32_t list = 0;
  p.v = latent ? nullptr : &v;
  p.indices = listed ? &list : nullptr;
  p.num_indices = listed;
  p.num_seqs = seqs;
  p.num_rows = rows;
  p.num_heads = heads;
  p.num_kv_heads = kv_heads;
  p.group = heads / kv_heads;
  p.max_seqlen_q = max_q;
  p.max_seqlen_k = max_k;
  if (!fp4idx::plan_attention(&p, sms)) return 0;
  out[0] = p.whole_items;
  out[1] = p.groups;
  out[2] = p.members;
  out[3] = p.items;
  return 1;
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    lib = build.build()
    where = tmp_path_factory.mktemp("plan")
    src, so = str(where / "ask.cu"), str(where / "ask.so")
    with open(src, "w") as f:
        f.write(ASK)
    subprocess.run([build._nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-shared", "-o", so, src, lib, "-Xlinker", "-rpath",
                    "-Xlinker", os.path.dirname(lib)], check=True, capture_output=True)
    f = ctypes.CDLL(so).ask

    def call(kind, seqs, heads, kv_heads=1, rows=None, max_q=1, max_k=0, listed=0):
        out = (ctypes.c_int * 4)()
        assert f(int(kind == "latent"), listed, seqs, seqs if rows is None else rows, heads, kv_heads, max_q, max_k, SMS, out)
        return dict(zip(("whole", "groups", "members", "items"), out))

    return call


@pytest.mark.parametrize("reqs", [33, 36, 37, 38, 39, 76, 114, 152, 304])
@pytest.mark.parametrize("keys", [4096, 32768, 131072])
def test_long_prefixes_are_cut_whatever_the_batch_size(ask, reqs, keys):
    # a whole item would leave the longest request to one CTA, whatever the others' lengths are
    for kind, heads, kv in (("paged", 32, 4), ("paged", 32, 8), ("latent", 16, 1), ("latent", 64, 1), ("latent", 128, 1)):
        p = ask(kind, reqs, heads, kv, max_k=keys)
        tiles = p["items"] * keys // (64 if kind == "latent" else 128)
        # (groups are left out only to cut items evenly, for less than the five tiles of a crossing)
        assert not p["whole"] and tiles / p["groups"] <= tiles / (SMS // p["members"]) + 5, (kind, heads, kv, p)


def test_prompt_among_decodes_is_cut(ask):
    p = ask("latent", 19, 128, rows=1024 + 18, max_q=1024, max_k=4096)
    assert not p["whole"] and p["groups"] == SMS // p["members"]


@pytest.mark.parametrize("reqs", range(1, 400, 7))
@pytest.mark.parametrize("keys", [64, 500, 1000, 3000, 9000, 100000])
def test_no_whole_prefix_takes_longer_than_cutting_could_cost(ask, reqs, keys):
    for kind, heads, kv, tile in (("paged", 8, 1, 128), ("paged", 64, 8, 128), ("latent", 16, 1, 64), ("latent", 128, 1, 64)):
        p = ask(kind, reqs, heads, kv, max_k=keys)
        if p["whole"]:
            assert -(-keys // tile) * -(-p["items"] // p["groups"]) <= 12


def test_short_prefixes_and_lists_stay_whole(ask):
    assert ask("paged", 40, 32, 4, max_k=4 * 128)["whole"] and ask("paged", 38, 32, 4, max_k=12 * 128)["whole"]
    assert ask("latent", 1, 16, max_k=64)["whole"] and ask("latent", 64, 16, max_k=3 * 64)["whole"]
    assert ask("paged", 64, 32, 4, max_k=8192, listed=16)["whole"]
    assert ask("latent", 1, 64, rows=100, max_q=100, max_k=32768, listed=2048)["whole"]
    assert not ask("latent", 1, 64, rows=4, max_q=4, max_k=16384, listed=2048)["whole"]
