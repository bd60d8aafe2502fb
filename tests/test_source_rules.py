"""Rules that the CUDA sources keep to, checked in their text (no GPU needed)."""
import glob
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def sources():
    found = [p for pattern in ("gated_pooling_gb300/csrc/*", "include/*") for p in glob.glob(os.path.join(ROOT, pattern))]
    assert len(found) > 10
    return found


def test_no_multicast():
    """No copy (nor commit) to several blocks of a cluster: every rank of a job on several GPUs loads this
    library, and a caller's workspace may be any memory."""
    for path in sources():
        assert "multicast" not in open(path, encoding="utf-8").read(), path
