"""A library built before an entry point was added is refused with the advice to
rebuild it, whatever its version number says."""
import subprocess

import pytest

import selective_state_space_80_amd as mamba


def _stub(tmp_path, names):
    src = tmp_path / "stub.c"
    src.write_text(f"int mamba_abi_version(void) {{ return {mamba.ABI_VERSION}; }}\n" +
                   "".join(f"int {n}(void) {{ return 0; }}\n" for n in names if n != "mamba_abi_version"))
    out = tmp_path / "libstub.so"
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(out), str(src)], check=True)
    return str(out)


@pytest.mark.parametrize("lacks", ["mamba_rms_norm", "mamba_int8_matmul", "mamba_selective_scan_bwd", "mamba_status_string"])
def test_library_without_an_entry_point(tmp_path, monkeypatch, lacks):
    path = _stub(tmp_path, [n for n in mamba.EXPORTED if n != lacks])
    monkeypatch.setattr(mamba, "_lib", None)
    with pytest.raises(RuntimeError, match=f"(?s){lacks}.*rebuild it"):
        mamba.load_library(path)
    assert mamba._lib is None


def test_library_with_all_of_them(tmp_path, monkeypatch):
    monkeypatch.setattr(mamba, "_lib", None)
    assert mamba.load_library(_stub(tmp_path, mamba.EXPORTED)).mamba_abi_version() == mamba.ABI_VERSION


def test_library_without_a_version(tmp_path, monkeypatch):
    src = tmp_path / "none.c"
    src.write_text("int nothing(void) { return 0; }\n")
    out = tmp_path / "libnone.so"
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(out), str(src)], check=True)
    monkeypatch.setattr(mamba, "_lib", None)
    with pytest.raises(RuntimeError, match="rebuild it"):
        mamba.load_library(str(out))
