"""The pieces that both tensor-core sources have (gemm_tc.cu, and tc.cuh of the operators' kernels) say the same (CPU)."""

import os
import re

import pytest

from muon_newton_schulz_expert_gb300.build import CSRC


def pieces(name):
    """{name: text without comments and spacing} of the wrappers, waits and structs before a file's first kernel."""
    src = open(os.path.join(CSRC, name)).read()
    src = re.sub(r"//[^\n]*", "", src.split("PTX wrappers")[1])
    found = {}
    for m in re.finditer(r"^(?:__device__|struct)[^\n;{]*?(\w+)\s*(?:\((?:[^{]*?)\))?\s*\{", src, re.M):
        depth, end = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(src[end], 0)
            end += 1
        found.setdefault(m.group(1), re.sub(r"\s+", "", src[m.start():end]))
    return found


# each is one function of the hardware's, or a wait whose limit must hold in both
SHARED = ["smem_u32", "mbar_init", "mbar_expect_tx", "mbar_try_wait", "mbar_test_wait", "global_ns", "Watch",
          "wait_bounded", "wait_polled", "dcheck", "tma_load_3d", "tma_load_3d_pair", "cluster_rank", "map_to_rank",
          "mbar_arrive_cluster", "cluster_sync_all", "tma_store_3d", "bulk_commit", "bulk_wait_read_all",
          "bulk_wait_all", "fence_proxy_async_smem", "tma_prefetch_desc", "tc_fence_before", "tc_fence_after",
          "tc_commit_mc", "tc_mma", "tmem_ld16", "smem_desc", "drain_wait"]


@pytest.mark.parametrize("name", SHARED)
def test_both_say_the_same(name):
    ours, theirs = pieces("tc.cuh"), pieces("gemm_tc.cu")
    assert len(ours[name]) > 20 and ours[name] == theirs[name]


def test_nothing_else_is_in_both_under_one_name():
    both = set(pieces("tc.cuh")) & set(pieces("gemm_tc.cu"))
    # 32 columns are waited for in one instruction there and apart here, so that 64 can be waited for at once
    assert both - {"tmem_ld32"} == set(SHARED)
