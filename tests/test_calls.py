"""The two ways from Python into the library (CPU only: each call is refused, or is an empty one): the module built for
this Python, and ctypes where there is none, with the same arguments, results and errors; what a build needs."""
import os
import subprocess
import sys

import pytest
import torch

import gated_pooling_gb300 as gp
from gated_pooling_gb300 import build as gb

FAKE = 1 << 20  # a 16-byte aligned non-null address; never dereferenced


@pytest.fixture(params=["module", "ctypes"])
def way(request, monkeypatch):
    gp.load()
    if request.param == "module":
        if not os.path.exists(gb.CALL):
            pytest.skip("the module is not built for this Python")
    else:
        monkeypatch.setattr(gb, "CALL", os.path.join(gb.LIBDIR, "of_another_python.so"))
    monkeypatch.setattr(gp, "_calls", None)
    return request.param


def append(**over):
    a = dict(x=FAKE, dtype=0, rows=0, heads=2, d=64, x_row_stride=128, x_head_stride=64, weight=None, norm=1, eps=1e-6, positions=FAKE,
             turns=FAKE, rot_dim=64, rot_start=0, layout=0, amplitude=1.0, slots=FAKE, num_slots=16, format=1, data=FAKE, scales=FAKE,
             dev_error=None, stream=0)
    a.update(over)
    gp.csa_cache_append(**a)


def test_arguments_and_errors(way):
    t = torch.zeros(64)
    append()
    assert isinstance(gp._calls, gp._CtypesCalls) == (way == "ctypes")
    append(x=t, weight=t, slots=t, norm=True, eps=0, amplitude=1)
    for over, code in ((dict(x=FAKE + 1), gp.CSA_ERR_INVALID_VALUE), (dict(d=72), gp.CSA_ERR_UNSUPPORTED), (dict(weight=FAKE + 2), 1)):
        with pytest.raises(gp.CsaError) as e:
            append(**over)
        assert e.value.status == code and "csa_cache_append" in str(e.value)
    for over, kind in ((dict(heads=1 << 31), OverflowError), (dict(rows=1 << 63), OverflowError), (dict(x=-1), OverflowError),
                       (dict(rows=-(1 << 63) - 1), OverflowError), (dict(x=1 << 64), OverflowError), (dict(x="x"), AttributeError),
                       (dict(d=1.5), TypeError), (dict(eps="1"), TypeError), (dict(slots=1.5), AttributeError)):
        with pytest.raises(kind):
            append(**over)
    with pytest.raises(TypeError):
        gp._calls.csa_cache_append(1, 2, 3)
    with pytest.raises(OverflowError):
        gp.csa_compressor_bwd(FAKE, FAKE, FAKE, FAKE, FAKE, 1, 4, 2, 64, 8, 2, FAKE, FAKE, FAKE, 0, FAKE, -1, None, 0)


@pytest.mark.parametrize("name,args", [
    ("csa_compressor_fwd", (0, 0, 0, 0, -1, 4, 2, 64, 8, 0, 2, None, 0)),
    ("csa_compressor_bwd", (0, 0, 0, 0, 0, -1, 4, 2, 64, 8, 2, 0, 0, 0, 0, 0, 0, None, 0)),
    ("csa_compressor_bwd_noalloc", (0, 0, 0, 0, 0, -1, 4, 2, 64, 8, 2, 0, 0, 0, 0, None, 0)),
    ("csa_compressor_map_blocks", (0, -1, 4, 8, 2, 0, None, 0)),
    ("csa_kpool_fwd", (0, 0, 0, 0, -1, 4, 64, 8, 0, 2, 0, None, 0)),
    ("csa_norm_rope_fwd", (0, 0, -1, 1, 64, 64, 64, 0, 1, 0.0, 0, 0, 0, 0, 0, 1.0, 0, 64, 64, 0)),
    ("csa_norm_rope_bwd", (0, 0, 0, -1, 1, 64, 64, 64, 64, 64, 0, 1, 0.0, 0, 0, 0, 0, 0, 1.0, 0, 64, 64, 0, 0, 0, 0, 0)),
    ("csa_cache_write", (0, 0, -1, 1, 64, 64, 64, 0, 1, 0, 0, 0, None, 0)),
    ("csa_cache_read", (0, 0, 0, 0, -1, 1, 1, 64, 0, 0, 64, 64, None, 0)),
    ("csa_cache_attn", (0, 1, 1, 0, -1, 1, 1, 1, 64, 0, 0, 0, 0, 1, 1, 1, 0, 0, 0, 1.0, 0, 0, 1, 1, 0, 0, 0, None, 0)),
    ("csa_compressor_step", (0, 0, 0, 0, -1, 4, 2, 64, 8, 0, 0, 0, 1, 0, 0, 0, 1, None, None, 0, 1, 0, None, None, None, None, 0)),
    ("csa_cache_append", (0, 0, -1, 1, 64, 64, 64, 0, 1, 0.0, 0, 0, 0, 0, 0, 1.0, 0, 1, 0, 0, 0, None, 0)),
    ("csa_cache_attn_prefix", (0, 1, 1, 0, -1, 1, 1, 1, 64, 0, 0, 0, 0, 1, 0, 1, 0, 0, 1, 1, 1, 0, 0, 0, 1.0, 0, 0, 1, 1, 0, 0, 0, None, 0)),
])
def test_every_function_goes_either_way(way, name, args):
    """A negative count is refused by each, so all of them take their arguments to the library."""
    with pytest.raises(gp.CsaError) as e:
        getattr(gp, name)(*args)
    assert e.value.status == gp.CSA_ERR_INVALID_VALUE and name in str(e.value)


def test_a_workspace_error_names_no_other_call(way):
    with pytest.raises(gp.CsaError) as e:
        gp.csa_cache_attn(FAKE, 64, 64, FAKE, 1, 1, 1, 1, 64, FAKE, None, 0, FAKE, 1, 1, 16, FAKE, None, 0, 1.0, None, FAKE, 64, 64, None,
                          None, 0, None, 0)
    assert e.value.status == gp.CSA_ERR_WORKSPACE and "csa_cache_attn: " in str(e.value) and "compressor_bwd" not in str(e.value)


def test_the_library_needs_no_python(monkeypatch, tmp_path):
    """Without g++, or without Python's headers, the library is what there is to build; a Python that the module was not
    built for takes the library as it is."""
    gb.build()
    assert gb.up_to_date() and gb.library_up_to_date()
    monkeypatch.setattr(gb, "CALL", str(tmp_path / "_csa_call.so"))
    monkeypatch.setattr(gb, "_build_library", lambda verbose: pytest.fail("the library is there"))
    for lacks in ("g++", "headers"):
        with monkeypatch.context() as m:
            if lacks == "g++":
                m.setattr(gb.shutil, "which", lambda name: None)
            else:
                m.setattr(gb.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
            assert not gb.can_build_call() and gb.up_to_date()
            assert gb.build() == gb.LIB and not os.path.exists(gb.CALL)
    if not gb.can_build_call():
        pytest.skip("no g++ or no headers here")
    assert not gb.up_to_date()  # a module of its own is built for this Python, and nothing else
    with monkeypatch.context() as m:
        m.setattr(gb, "_run", lambda cmd, what: open(cmd[cmd.index("-o") + 1], "w").close() or "")
        gb.build()
    assert os.path.exists(gb.CALL) and gb.up_to_date()


def test_a_module_of_an_older_header_is_not_called(monkeypatch, tmp_path):
    """One that cannot be built again, here for want of g++, may take other arguments than the library does by now."""
    gp.load()
    old = tmp_path / "_csa_call.so"
    old.write_bytes(b"")
    os.utime(old, (0, 0))
    monkeypatch.setattr(gb, "CALL", str(old))
    monkeypatch.setattr(gb, "can_build_call", lambda: False)
    monkeypatch.setattr(gp, "_calls", None)
    append()
    assert isinstance(gp._calls, gp._CtypesCalls)


def test_import_without_the_module():
    """A process of its own whose Python has no module: the package loads, calls and reports through ctypes."""
    code = ("import gated_pooling_gb300 as gp; from gated_pooling_gb300 import build as gb\n"
            "gb.CALL = gb.CALL + '.absent'; gb.can_build_call = lambda: False\n"
            "try:\n    gp.csa_kpool_fwd(0, 0, 0, 0, -1, 4, 64, 8, 0, 2, 0, None, 0)\n"
            "except gp.CsaError as e:\n    print(type(gp._calls).__name__, e.status)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root)
    assert res.returncode == 0 and res.stdout.split() == ["_CtypesCalls", "1"], res.stdout + res.stderr
