"""Commit of accepted drafts (pkv_commit_tree) where a CTA moves several layers, the last one fewer; bit for bit."""
import random

import pytest

from test_gpu_commit import Batch, trees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,layers", [(256, 32), (100, 37), (90, 128), (2000, 3), (152, 5), (153, 5)])
def test_layers_of_a_cta(n, layers):
    r = random.Random(n + layers)
    b = Batch(trees(n, [r.randrange(24) for _ in range(n)]), [r.randrange(20) for _ in range(n)], n, layers=layers, S=8, Hkv=1, D=64)
    b.device().run().verify(f"{n} sequences, {layers} layers")
    assert int(b.err) == 0
