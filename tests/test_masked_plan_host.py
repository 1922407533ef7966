"""How masked attention lays its calls over CTAs, asked from the plan itself on the host: the GPU tests'
calls reach the kernel with two query tiles per CTA, the split of keys over a cluster, and both grid orders."""
import os
import shutil
import subprocess

import pytest

import patch_attention_b200 as pa
from patch_attention_b200 import build
from tests._two_tiles import HEAD_BY_HEAD, LAYOUT, SPLIT, TWO_TILES

SMS = 148

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include "pf_internal.h"
int main() {
  int batch, n_q, n_k, heads_q, heads_kv, d, causal, docs, sms;
  while (std::scanf("%d %d %d %d %d %d %d %d %d", &batch, &n_q, &n_k, &heads_q, &heads_kv, &d, &causal, &docs, &sms) == 9) {
    pf::MaskedFwdParams p;
    std::memset(&p, 0, sizeof(p));
    int id = 0;
    p.batch = batch; p.heads_q = heads_q; p.heads_kv = heads_kv; p.head_dim = d;
    p.m.n_q = n_q; p.m.n_k = n_k; p.m.causal = causal;
    p.m.doc_q = p.m.doc_k = docs ? &id : nullptr;
    pf::masked_fwd_plan(p, sms);
    std::printf("%d %d %d %d\n", p.pack, p.n_groups, p.n_split, p.heads_first);
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """plan(cases): [(heads per tile, query tiles, CTAs' groups of them, key split, longest first over all heads)]"""
    compiler = shutil.which("g++") or shutil.which("c++")
    assert compiler and os.path.exists(pa.LIB_PATH)
    at = tmp_path_factory.mktemp("plan")
    src, exe = at / "plan.cpp", at / "plan"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.NVCC)), "include")
    here = os.path.dirname(os.path.abspath(pa.LIB_PATH))
    subprocess.run([compiler, "-std=c++17", "-O1", "-I", build.INCLUDE, "-I", build.CSRC, "-I", cuda, str(src),
                    os.path.abspath(pa.LIB_PATH), f"-Wl,-rpath,{here}", "-Wl,--allow-shlib-undefined", "-o", str(exe)],
                   check=True, capture_output=True, text=True)

    def ask(cases):
        text = "".join(f"{b} {nq} {nk} {hq} {hk} {d} {int('c' in r)} {int('d' in r)} {SMS}\n"
                       for b, nq, nk, hq, hk, d, r in cases)
        out = subprocess.run([str(exe)], input=text, check=True, capture_output=True, text=True).stdout.split()
        rows = [tuple(int(x) for x in out[i:i + 4]) for i in range(0, len(out), 4)]
        assert len(rows) == len(cases)
        return [(pack, -(-c[1] // (128 // pack)), groups, split, first)
                for c, (pack, groups, split, first) in zip(cases, rows)]

    return ask


def test_two_query_tiles_per_cta(plan):
    for name, (pack, tiles, groups, split, _) in zip(TWO_TILES, plan(list(TWO_TILES.values()))):
        assert split == 1 and tiles > 1 and groups == (tiles + 1) // 2, name
        assert (pack, tiles) == LAYOUT[name], name


def test_grid_orders(plan):
    for name, (_, tiles, groups, split, first) in zip(HEAD_BY_HEAD, plan(list(HEAD_BY_HEAD.values()))):
        assert not first and groups < tiles, name
    causal = [c for c in TWO_TILES.values() if "c" in c[6]]
    assert causal and all(first for *_, first in plan(causal))


def test_split_keys(plan):
    for name, (_, tiles, groups, split, _) in zip(SPLIT, plan(list(SPLIT.values()))):
        assert split > 1 and groups == tiles, name
