"""Rules on the kernels' sources that no run on one device shows."""

import os
import re

from token_sparse_denoising_layer_b200 import build


def _sources():
    for name in sorted(os.listdir(build.CSRC)):
        with open(os.path.join(build.CSRC, name)) as f:
            yield name, f.read()


def test_arrivals_at_another_ctas_barrier_name_the_clusters_scope():
    """Without a scope an arrive orders nothing beyond its own CTA."""
    found = 0
    for name, text in _sources():
        for op in re.findall(r"mbarrier\.arrive[\w.:]*\.shared::cluster[\w.:]*", text):
            found += 1
            assert re.search(r"\.(release|relaxed)\.cluster\.shared::cluster", op), f"{name}: {op}"
    assert found >= 2


def test_the_wait_for_both_ctas_of_a_pair_names_the_clusters_scope():
    text = dict(_sources())["k_gemm.cu"]
    pair = text[text.index("k_gemm_pair(const __grid_constant__"):]
    waits = re.findall(r"mbar_wait(<true>)?\(&acc_empty", pair[:pair.index("lead_empty0")])
    assert waits == ["<true>"]
