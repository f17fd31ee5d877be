"""A library that serves the NVFP4 calls is loaded whether or not it has the MXFP4 functions this
binding expects; only their calls refuse it.  The libraries are stubs of the exported names."""
import subprocess

import pytest

import nvfp4_block_scaled_quantize_amd as nv
from nvfp4_block_scaled_quantize_amd import mxfp4


@pytest.fixture(scope="module", params=["without", "another version", "with"])
def stub(request, tmp_path_factory):
    """Path of a library, and whether MXFP4 calls may use it."""
    version = {"without": None, "another version": mxfp4.MXFP4_ABI_VERSION + 1, "with": mxfp4.MXFP4_ABI_VERSION}[request.param]
    values = {name: 0 for name in nv.EXPORTED}
    values["nvfp4_abi_version"] = nv.ABI_VERSION
    if version is not None:
        values |= {name: 0 for name in mxfp4.MXFP4_EXPORTED}
        values["mxfp4_abi_version"] = version
    d = tmp_path_factory.mktemp("stub")
    (d / "stub.c").write_text("".join(f"long {n}(void) {{ return {v}; }}\n" for n, v in values.items()))
    subprocess.check_call(["gcc", "-shared", "-fPIC", str(d / "stub.c"), "-o", str(d / "stub.so")])
    return str(d / "stub.so"), request.param == "with"


def test_library_by_path(stub):
    assert nv.load_library(stub[0]).nvfp4_abi_version() == nv.ABI_VERSION


def test_own_library(stub, monkeypatch):
    path, usable = stub
    monkeypatch.setattr(nv, "LIB_PATH", path)
    monkeypatch.setattr(nv, "_lib", None)
    monkeypatch.setattr(mxfp4, "_bound", None)
    monkeypatch.setattr(mxfp4, "_unusable", None, raising=False)
    assert nv.load_library() is nv.load_library()
    if usable:
        assert nv.mxfp4_linear_workspace_bytes(1, 32, 32) == 0
    else:
        for _ in range(2):
            with pytest.raises(nv.Nvfp4Error, match="rebuild"):
                nv.mxfp4_linear_workspace_bytes(1, 32, 32)


def test_own_library_first_loaded_by_an_mxfp4_call(stub, monkeypatch):
    path, usable = stub
    monkeypatch.setattr(nv, "LIB_PATH", path)
    monkeypatch.setattr(nv, "_lib", None)
    monkeypatch.setattr(mxfp4, "_bound", None)
    monkeypatch.setattr(mxfp4, "_unusable", None, raising=False)
    if usable:
        assert nv.mxfp4_linear_workspace_bytes(1, 32, 32) == 0
    else:
        with pytest.raises(nv.Nvfp4Error, match="rebuild"):
            nv.mxfp4_linear_workspace_bytes(1, 32, 32)
    assert nv.load_library().nvfp4_abi_version() == nv.ABI_VERSION
