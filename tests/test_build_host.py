"""The package without its extension module, and when that is built anew."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NO_BIND = """
import sys

class Block:
    def find_spec(self, name, path=None, target=None):
        if name == "ternary_weight_decoder_b200._bind":
            raise ImportError("not built")

sys.meta_path.insert(0, Block())
from ternary_weight_decoder_b200 import api, tp
assert api.tw_sweep_table_bytes(3) > 0
assert api.tw_residual_norm(None, None) == 1     # the C entry points are there
for call in (lambda: api.residual_norm(None), lambda: api.kv_assign(*[None] * 7),
             lambda: api._bind.paged_attention):
    try:
        call()
    except ImportError as e:
        assert "ternary_weight_decoder_b200.build" in str(e) and "not built" in str(e)
    else:
        raise AssertionError("no error")
print("fine")
"""


@pytest.fixture(scope="module")
def build():
    from ternary_weight_decoder_b200 import build
    build.build()
    return build


def test_other_operators_need_no_extension(build):
    r = subprocess.run([sys.executable, "-c", NO_BIND], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr


def test_library_is_built_without_the_extension(build, tmp_path, monkeypatch):
    def fails():
        raise RuntimeError("g++ failed")

    lib = tmp_path / "lib.so"
    monkeypatch.setattr(build, "build_bind", fails)
    monkeypatch.setattr(build, "LIB", str(lib))
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        build.build()
    assert lib.stat().st_size > 0


def test_extension_is_built_anew_for_another_torch(build, monkeypatch):
    assert build.bind_is_current()
    with monkeypatch.context() as m:
        m.setattr(build.importlib.metadata, "version", lambda name: "0.0.1")
        assert not build.bind_is_current()
    with monkeypatch.context() as m:
        m.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-0")
        assert not build.bind_is_current()
    with monkeypatch.context() as m:
        m.setattr(build, "BIND_MADE_FOR", build.BIND_MADE_FOR + ".none")
        assert not build.bind_is_current()
    assert build.bind_is_current()
