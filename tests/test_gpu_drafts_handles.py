"""The decoder of examples/drafts.py keeps one workspace of the delta rule for all of its layers."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import exact_online_amd as fi  # noqa: E402
from examples.drafts import DeltaDecoder, make_weights  # noqa: E402


def test_layers_share_a_handle(monkeypatch):
    made = []

    class Counted(fi.DeltaRule):
        def __init__(self, *a, **kw):
            made.append(a)
            super().__init__(*a, **kw)
    monkeypatch.setattr(fi, "DeltaRule", Counted)
    m = DeltaDecoder(make_weights(300, 64, 3, 2, 4, 32, 128, torch.float32), 2, 70, 2, 4, 32)
    assert len(made) == 1 and len(m.state) == 3
    z = m.run(torch.randint(300, (2, 70), device="cuda"), fresh=True)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(z).all())
    m.close()
