"""CPU: the binding's table of engines, kept by every way to create and destroy one."""
import ctypes

import pytest

from streaming_speaker_diarization_b200 import binding as b

HANDLE = 0x7ffffffe0000


@pytest.fixture
def destroyed(monkeypatch):
    """Library calls on a handle that no engine stands behind, and the handles destroyed."""
    got = []

    def metadata(handle, cfg):
        cfg._obj.precision = b.SF_FP32
        return 0
    monkeypatch.setattr(b.lib, "sf_get_metadata", metadata)
    monkeypatch.setattr(b.lib, "sf_destroy", lambda handle: got.append(handle) or 0)
    monkeypatch.setattr(b, "_current_device", lambda: 3)
    yield got
    b._engines.pop(HANDLE, None)


def test_engines_created_through_the_library_are_known():
    assert b.lib.sf_create.errcheck is b._created and b.lib.sf_create_from_file.errcheck is b._created
    assert b.lib.sf_destroy.errcheck is b._destroyed
    h = ctypes.c_void_p()
    assert b.lib.sf_create_from_file(b"/no/such/file", ctypes.byref(b.default_config()), ctypes.byref(h)) != 0
    assert None not in b._engines


@pytest.mark.parametrize("form", ["byref", "pointer", "array", "place"])
def test_the_handle_is_found_in_every_form_of_the_argument(destroyed, form):
    h = ctypes.c_void_p(HANDLE)
    out = {"byref": lambda: ctypes.byref(h), "pointer": lambda: ctypes.pointer(h), "place": lambda: h,
           "array": lambda: (ctypes.c_void_p * 1)(HANDLE)}[form]()
    assert b._created(0, None, (b"path", ctypes.byref(b.default_config()), out)) == 0
    assert b._engines[HANDLE] == (b.SF_FP32, 3)
    assert b._created(2, None, (b"path", None, ctypes.byref(ctypes.c_void_p()))) == 2
    b._destroyed(0, None, (h if form == "place" else HANDLE,))
    assert HANDLE not in b._engines and not destroyed


def test_an_engine_whose_device_is_not_found_is_destroyed(destroyed, monkeypatch):
    def no_device():
        raise b.SFError("SF_EDEVICE: none")
    monkeypatch.setattr(b, "_current_device", no_device)
    with pytest.raises(b.SFError, match="SF_EDEVICE"):
        b._created(0, None, (b"path", None, ctypes.byref(ctypes.c_void_p(HANDLE))))
    assert destroyed == [HANDLE] and HANDLE not in b._engines
