"""The build of the native host path, which the package can do without (no GPU needed)."""
import block_scaled_fp8_grouped_amd._build as build


def test_no_compiler_is_no_error(monkeypatch, tmp_path, capsys):
    """hipcc alone builds the library; what an older build left of the extension does not stay beside it."""
    path = tmp_path / "_native.so"
    monkeypatch.setattr(build, "BINDING_PATH", str(path))
    monkeypatch.setattr(build, "_compile", lambda src, obj: obj)
    monkeypatch.setattr(build, "_link", lambda objs, out: None)
    for compiler in ("/no/such/compiler", "false"):
        path.write_bytes(b"old")
        monkeypatch.setenv("CXX", compiler)
        build.build()
        assert not path.exists()
        err = capsys.readouterr().err
        assert "libbsfp8.so" in err and "is not built" in err
