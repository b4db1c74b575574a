"""The README's example of long contexts runs as written; its outputs are the attention over the selected blocks and
over all of the context, evaluated here in float64 from what the cache holds."""
import os
import re

import pytest

import attn_ref as ref
import long_ref
from gpu_util import say

pytestmark = pytest.mark.gpu


def test_readme_long_contexts_example_runs():
    import numpy as np
    import torch
    assert torch.cuda.is_available()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    blocks = re.findall(r"```python3\n(.*?)```", open(os.path.join(root, "README.md")).read(), re.S)
    assert len(blocks) == 1
    say("case README example of long contexts")
    ns = {}
    exec(compile(blocks[0], "README.md", "exec"), ns)
    cache = ref.Cache(64, 64, 2, 128)
    img, table = ns["pages"].cpu().numpy(), ns["table"].cpu().numpy()
    q, o, full, score = (ns[x].double().cpu().numpy() for x in ("q", "o", "full", "score"))
    sel = ns["sel"].cpu().numpy()
    for i, n in enumerate((1201, 701)):
        K, V, there = cache.request(table[i], n, img)
        for h in range(8):
            assert sel[i, h // 4].tolist() == long_ref.select(score[i, h // 4], n - 1, 64, 8, 1, 2)
            for got, cols in ((o, sel[i, h // 4]), (full, range(24))):
                want, bound = long_ref.attend_listed(q[i, h], K[:, h // 4], V[:, h // 4], there, n - 1, cols, 64, 128 ** -0.5, "bf16")
                assert (np.abs(got[i, h] - want) <= bound).all()
