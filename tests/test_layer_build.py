"""When the Python binding of the layer operators is built again, and that the library
needs neither it nor torch."""
import os

from blockwise_fp8_linear_fp8bw_b200 import build


def test_the_binding_follows_its_sources_the_header_and_torch(monkeypatch):
    build.build()
    assert not build._binding_stale()
    mtime = os.path.getmtime
    for path in (build.BINDING_SRC, build.HEADER, build.LAYER_HEADER):
        with monkeypatch.context() as m:
            newer = mtime(build.BINDING) + 1
            m.setattr(os.path, "getmtime", lambda p, path=path: newer if p == path else mtime(p))
            assert build._binding_stale(), path
    for version in ("0.0", build._torch_version() + "1", build._torch_version()[:-1]):
        with monkeypatch.context() as m:
            m.setattr(build, "_torch_version", lambda version=version: version)
            assert build._binding_stale(), version


def test_the_library_builds_without_torch(monkeypatch):
    made = []
    monkeypatch.setattr(build, "_torch_version", lambda: None)
    monkeypatch.setattr(build, "_build_lib", lambda verbose: made.append("library"))
    monkeypatch.setattr(build, "build_binding", lambda force=False: made.append("binding"))
    assert build.build(force=True) == build.LIB
    assert made == ["library"] and not build._binding_stale()
    monkeypatch.setattr(build, "_torch_version", lambda: "2")
    build.build(force=True)
    assert made == ["library", "library", "binding"]
