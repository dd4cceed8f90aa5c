"""The README's serving example runs as written (parity itself is covered by
the packed and paged GPU tests)."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_serving_example(gpu):
    """The README's serving step: two requests through three steps of one paged cache."""
    text = open(os.path.join(ROOT, "README.md")).read()
    blocks = re.findall(r"```python\n(.*?)```", text, flags=re.S)
    scope = {}
    exec(compile(blocks[1], "README.md", "exec"), scope)  # noqa: S102 (the README's own example)
    torch.cuda.synchronize()
    assert gpu.attn_get_device_status() == gpu.ATTN_OK
    assert tuple(scope["o"].shape) == (2, 32, 128) and torch.isfinite(scope["o"].float()).all()
    assert scope["lens"].tolist() == [41, 19]
    assert scope["count"].item() == 64 - 3 - 2
