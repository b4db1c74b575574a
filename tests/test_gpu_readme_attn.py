"""The README's example of the softmax layers' operators runs as written, and its
output is the attention of its normalised, rotated queries over the keys and
values that the cache holds, evaluated here in float64."""
import os
import re

import pytest

import attn_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu


def test_readme_softmax_example_runs():
    import numpy as np
    import torch
    assert torch.cuda.is_available()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    blocks = re.findall(r"```py\n(.*?)```", open(os.path.join(root, "README.md")).read(), re.S)
    assert len(blocks) == 1
    say("case README example of the softmax layers")
    ns = {}
    exec(compile(blocks[0], "README.md", "exec"), ns)
    q, o, kc, vc = (ns[x].double().cpu().numpy() for x in ("qn", "o", "kc", "vc"))
    start = ns["tok_start"].cpu().numpy()
    assert list(start) == [0, 100, 101, 108] and list(ns["lens"].cpu().numpy()) == [100, 1, 7]
    assert int(ns["used"]) == 4 and ns["kv"].desc.n_blocks == 32
    for a, b in zip(start, start[1:]):
        for h in range(8):
            want, bound = ref.attend(q[a:b, h], kc[a:b, h // 4], vc[a:b, h // 4], np.ones(b - a, bool), 0, 128 ** -0.5, 0, 0, "bf16")
            assert (np.abs(o[a:b, h] - want) <= bound).all()
