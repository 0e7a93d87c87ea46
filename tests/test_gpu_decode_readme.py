"""The README's decode loop runs as written on the GPU; what it leaves behind is consistent."""

import os
import re

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_decode_loop_runs():
    use = open(os.path.join(ROOT, "README.md")).read().split("## Use", 1)[1]
    block = re.findall(r"```python\n(.*?)```", use, re.S)[1]
    scope = {}
    exec(compile(block, "README.md", "exec"), scope)
    torch, lens, kept, weights = (scope[x] for x in ("torch", "lens", "kept", "weights"))
    # 515 + 8 tokens were cut to 512 once, four more followed; the other request never outgrew its budget
    assert lens.tolist() == [516, 312]
    assert bool((kept[:, 0] >= 0).all()) and bool((kept[:, 0].diff(dim=-1) > 0).all())
    assert kept[0, 1, 0, :308].tolist() == list(range(308)) and bool((kept[:, 1, :, 308:] == -1).all())
    assert torch.isfinite(scope["out"].float()).all() and float(weights.min()) >= 0
    # request 1 attended 12 times with 32 heads in every layer: that much weight lies in its slots
    assert weights[:, 40:].sum(dim=(1, 2, 3)).tolist() == pytest.approx([12 * 32] * 2, rel=1e-4)
