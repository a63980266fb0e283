"""The library through its binding where torch is not installed: what needs no tensors."""
import subprocess
import sys

CODE = """
import sys
sys.modules["torch"] = None
import exact_means_clustering_flashassign_amd as fk
assert fk.fk_version() > 0
assert [fk.fk_status_string(i) for i in (0, 3)] == {names!r}
assert fk.load().fk_workspace_size(1, 2, 1000, 64, 10) >= 256
"""


def test_load_without_torch():
    import exact_means_clustering_flashassign_amd as fk
    from conftest import ROOT

    code = CODE.format(names=[fk.fk_status_string(i) for i in (0, 3)])
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
