"""The build command makes everything that the package loads."""

from persistent_tile_scheduled_amd import _build


def test_build_command(monkeypatch):
    made = []
    for name in ("build_library", "build_torch_module", "build_stress_library"):
        monkeypatch.setattr(_build, name, lambda name=name: made.append(name))
    _build.main([])
    assert made == ["build_library", "build_torch_module"]
    made.clear()
    _build.main(["--stress"])
    assert made == ["build_stress_library"]
