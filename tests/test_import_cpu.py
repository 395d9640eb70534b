"""What the binding needs to be imported: the entries that were there before the recurrence and the norm need the
library only, not the extension that fills tensor records."""
import subprocess
import sys

import pytest

RUN = """
import sys
sys.path.insert(0, {root!r})
import torch
{prepare}
from gated_deltaproduct_recurrence_amd import binding as b
assert b.gdp_descriptor_capacity(812, 4, 2) == (16, 29)
assert b.gdp_gated_scan_workspace_bytes(200, 3, 96) > 0
try:
    b.chunk_prefill(*[torch.zeros(4, 2, 64)] * 3, torch.zeros(2, 2), torch.zeros(4, 2), 2, torch.tensor([0, 2]))
except ImportError:
    raise
except Exception as e:
    print("prefill:", type(e).__name__, e)
x, cu = torch.zeros(4, 8), torch.tensor([0, 4], dtype=torch.int32)
for call in (lambda: b.gated_scan(x, x, cu), lambda: b.gated_scan_decode(x, x, x, cu),
             lambda: b.gated_scan_backward(x, x, cu, x), lambda: b.group_norm(x[None]),
             lambda: b.group_norm_backward(x[None], x[None])):
    try:
        call()
    except ImportError as e:
        assert "not built" in str(e) and {why!r} in str(e), e
    else:
        raise AssertionError("no ImportError")
print("done")
"""


@pytest.mark.parametrize("prepare,why", [
    ("sys.modules['gated_deltaproduct_recurrence_amd._records'] = None", "_records"),
    ("import types; m = types.ModuleType('_records'); m.record_bytes, m.records = 72, lambda *a: a\n"
     "sys.modules['gated_deltaproduct_recurrence_amd._records'] = m", "72 bytes"),
    ("torch.__version__ = '1.2.3+other'", "built for torch"),
])
def test_the_older_entries_need_no_extension(prepare, why):
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", RUN.format(root=root, prepare=prepare, why=why)], capture_output=True,
                         text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.rstrip().endswith("done"), res.stdout + res.stderr
