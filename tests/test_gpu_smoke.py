"""smoke() compares the norm and rotation outside the cache with the oracle (GPU): with a mistake
in the oracle for rows of that shape it fails, and there."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def test_smoke_compares_prompt_rows(gpu_lib, monkeypatch):
    import __graft_entry__ as entry
    from oracle import rows as R
    entry.smoke()
    rotate = R.rotate

    def wrong(x, *args, **kw):
        out, size = rotate(x, *args, **kw)
        if np.ndim(x) == 4:  # [batch, tokens, heads, d]
            out = out * 1.01
        return out, size

    monkeypatch.setattr(R, "rotate", wrong)
    with pytest.raises(AssertionError, match="of a prompt"):
        entry.smoke()
