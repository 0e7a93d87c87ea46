"""The README's serving loop runs as written on the GPU; what it leaves behind is consistent."""

import os
import re

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_serving_loop_runs():
    use = open(os.path.join(ROOT, "README.md")).read().split("## Use", 1)[1]
    block = re.findall(r"```python\n(.*?)```", use, re.S)[2]
    scope = {}
    exec(compile(block, "README.md", "exec"), scope)
    torch, lens, tables, free, n_free, out = (scope[x] for x in ("torch", "lens", "tables", "free", "n_free", "out"))
    assert lens.tolist() == [2048 + n + 16 for n in (60, 200, 31)]
    assert bool(torch.isfinite(out.float()).all()) and float(out.float().abs().max()) > 0
    # every block is on the pile, in the shared document, or in one request's own part
    own = [tables[r, 128:-(-n // 16)].tolist() for r, n in enumerate(lens.tolist())]
    used = tables[0, :128].tolist() + sum(own, [])
    assert sorted(used + free[:int(n_free)].tolist()) == list(range(512))
